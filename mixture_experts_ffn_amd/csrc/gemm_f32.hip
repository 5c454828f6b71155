// gemm_f32.hip — the fp32 grouped products, in their three contractions:
//
//   NN  y[m]  = x[m] . W[e]       W [E, K, N]
//   NT  y[m]  = x[m] . W[e]^T     W [E, N, K]
//   TN  dW[e] = sum_{m in e} a[m]^T b[m]
//
// Tiles of 64 x 64 outputs, 32 deep, four waves of 32 x 32, on the fp32 matrix
// instruction (16 x 16 x 4, products and sums in fp32).  Both operands lie in LDS
// with k outermost, so that a fragment is 16 consecutive values of four k rows,
// which a row length of 80 spreads over all banks; an operand that is contiguous
// along k is turned on the way in.  Two buffers, the next step's loads under the
// current one's products.  Bound by the matrix instruction: 256 flops a clock and
// CU, 32 clocks each, of which the four fragment reads of a step hide behind four.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace f32 {

constexpr int BT = 64, BK = 32, LD = BT + 16;

// A 64 x 32 operand tile on its way from memory to LDS: two 16-byte pieces a thread.
// KC: the operand is contiguous along k (piece: 4 k of a row), else along its
// rows (piece: 4 rows of a k).  What lies outside is zero.
template <bool KC> struct Stage {
    const float *p[2];
    bool ok[2];
    int r[2], k[2];
    f32x4 v[2];

    __device__ void place(const float *base, int64_t ld, int valid_r)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = threadIdx.x + i * 256;
            r[i] = KC ? u >> 3 : (u & 15) * 4;
            k[i] = KC ? (u & 7) * 4 : u >> 4;
            ok[i] = r[i] < valid_r; // a multiple of 4 rows where pieces run along them
            p[i] = base + (ok[i] ? KC ? r[i] * ld + k[i] : k[i] * ld + r[i] : 0);
        }
    }
    __device__ void load(int64_t ld, int k0, int K)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) // along k: K is a multiple of 8
            v[i] = ok[i] && k0 + k[i] < K
                       ? *reinterpret_cast<const f32x4 *>(p[i] + (KC ? k0 : k0 * ld))
                       : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ void store(float *s) const
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (KC) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[(k[i] + j) * LD + r[i]] = v[i][j];
            } else {
                *reinterpret_cast<f32x4 *>(s + k[i] * LD + r[i]) = v[i];
            }
        }
    }
};

template <int KIND> __global__ __launch_bounds__(256) void f32_grouped_kernel(F32Grouped a)
{
    constexpr bool TN = KIND == F32_TN;
    __shared__ __attribute__((aligned(16))) float sA[2][BK * LD], sB[2][BK * LD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    const int ntm = TN ? (a.M + BT - 1) / BT : 0, ntn = (a.N + BT - 1) / BT;
    const int64_t total = TN ? (int64_t)a.E * ntm * ntn : (int64_t)a.mtile_off[a.E] * ntn;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
        // group-major; inside a group column tiles outer, so that tiles in flight share weights
        int e, r0, rows, K;
        int64_t first; // first row of the group (TN), of the tile
        int n0;
        if constexpr (TN) {
            e = (int)(t / ((int64_t)ntm * ntn));
            const int local = (int)(t - (int64_t)e * ntm * ntn);
            n0 = local / ntm * BT;
            r0 = local % ntm * BT;
            rows = min(BT, a.M - r0);
            first = a.offsets[e];
            K = a.offsets[e + 1] - (int)first;
        } else {
            e = a.mtile_expert[t / ntn];
            const int mt0 = a.mtile_off[e], mts = a.mtile_off[e + 1] - mt0;
            const int64_t local = t - (int64_t)mt0 * ntn;
            n0 = (int)(local / mts) * BT;
            r0 = a.offsets[e] + (int)(local % mts) * BT;
            rows = min(BT, a.offsets[e + 1] - r0);
            first = r0;
            K = a.K;
        }
        const int cols = min(BT, a.N - n0);
        Stage<!TN> A;
        Stage<KIND == F32_NT> B;
        A.place(TN ? a.A + first * a.lda + r0 : a.A + first * a.lda, a.lda, rows);
        if constexpr (TN)
            B.place(a.B + first * a.ldb + n0, a.ldb, cols);
        else if constexpr (KIND == F32_NN)
            B.place(a.B + (int64_t)e * a.K * a.N + n0, a.ldb, cols);
        else
            B.place(a.B + (int64_t)e * a.K * a.N + (int64_t)n0 * a.ldb, a.ldb, cols);
        f32x4 acc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        A.load(a.lda, 0, K);
        B.load(a.ldb, 0, K);
        const int nk = (K + BK - 1) / BK;
        for (int s = 0; s < nk; ++s) {
            A.store(sA[s & 1]);
            B.store(sB[s & 1]);
            __syncthreads();
            if (s + 1 < nk) {
                A.load(a.lda, (s + 1) * BK, K);
                B.load(a.ldb, (s + 1) * BK, K);
            }
            const float *pa = sA[s & 1] + (lane >> 4) * LD + (lane & 15) + wm;
            const float *pb = sB[s & 1] + (lane >> 4) * LD + (lane & 15) + wn;
#pragma unroll
            for (int k = 0; k < BK; k += 4) {
                const float a0 = pa[k * LD], a1 = pa[k * LD + 16];
                const float b0 = pb[k * LD], b1 = pb[k * LD + 16];
                // the columns as the instruction's rows: a lane then holds four
                // neighbouring columns of one row
                acc[0][0] = Mfma<float>::mma(b0, a0, acc[0][0]);
                acc[0][1] = Mfma<float>::mma(b1, a0, acc[0][1]);
                acc[1][0] = Mfma<float>::mma(b0, a1, acc[1][0]);
                acc[1][1] = Mfma<float>::mma(b1, a1, acc[1][1]);
            }
        }
        // the buffer of step s is written again in step s + 2, after the barrier of s + 1
        float *C = TN ? a.C + (int64_t)e * a.M * a.N : a.C;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = wm + 16 * i + (lane & 15);
            if (r < rows)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = wn + 16 * j + (lane >> 4) * 4;
                    if (c < cols) // cols is a multiple of 8
                        *reinterpret_cast<f32x4 *>(C + (int64_t)(r0 + r) * a.N + n0 + c) = acc[i][j];
                }
        }
        __syncthreads(); // the next tile writes the buffers from the first on
    }
}

} // namespace f32

hipError_t launch_f32_grouped(int kind, const F32Grouped &a, hipStream_t s)
{
    const int64_t ntn = (a.N + f32::BT - 1) / f32::BT;
    const int64_t tiles =
        kind == F32_TN ? (int64_t)a.E * ((a.M + f32::BT - 1) / f32::BT) * ntn : a.max_mtiles * ntn;
    if (tiles <= 0)
        return hipSuccess;
    const dim3 grid((unsigned)(tiles < 65536 ? tiles : 65536));
    auto k = kind == F32_NN   ? f32::f32_grouped_kernel<F32_NN>
             : kind == F32_NT ? f32::f32_grouped_kernel<F32_NT>
                              : f32::f32_grouped_kernel<F32_TN>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe
