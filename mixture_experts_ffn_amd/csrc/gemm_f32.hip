// gemm_f32.hip — the fp32 grouped products, in their three contractions:
//
//   NN  y[m]  = x[m] . W[e]       W [E, K, N]
//   NT  y[m]  = x[m] . W[e]^T     W [E, N, K]
//   TN  dW[e] = sum_{m in e} a[m]^T b[m]
//
// Tiles of 64 x 64 outputs, 32 deep, four waves of 32 x 32, on the fp32 matrix
// instruction (16 x 16 x 4, products and sums in fp32); where these are too few for
// the CUs, tiles of 32 x 32 whose waves take a quarter of each step's k and are summed
// through LDS.  Both operands lie in LDS with k outermost, so that a fragment is 16
// consecutive values of four k rows; an operand that is contiguous along k is turned
// on the way in.  Two LDS buffers, and the loads of the next two steps in registers,
// since a step of a lone workgroup is shorter than a load.  Large problems keep the matrix
// cores (256 flops a clock and CU) busy 70 to 74 %, while the 64 x 64 tiles read 6.4 to 7.1
// TB/s through the L2s: 8192 rows of 4096 x 4096 over 8 groups 2420 us NN, 2500 NT, 2370 TN (110 to
// 116 TFLOP/s; a large library product reaches 154).  Small ones are bound by the length of the
// chain of steps: 1202 rows of 264 x 200 over 6 groups 9.2, 8.3 and 9.9 us.
#include <type_traits>

#include "common.h"
#include "group_view.h"
#include "kernels.h"

namespace moe {
namespace f32 {

constexpr int BK = 32;

// A BT x 32 operand tile on its way from memory to LDS, 16-byte pieces.  KC: the
// operand is contiguous along k (piece: 4 k of a row), else along its rows (piece: 4
// rows of a k).  What lies outside is zero.
template <bool KC, int BT> struct Stage {
    static constexpr int LD = BT + 20; // the turned pieces' rows fall in different banks
    static constexpr int NP = BT * BK / 4 / 256, RP = BT / 4;
    const float *p[NP];
    bool ok[NP];
    int r[NP], k[NP];
    f32x4 v[2][NP];

    __device__ void place(const float *base, int64_t ld, int valid_r)
    {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int u = threadIdx.x + i * 256;
            r[i] = KC ? u / (BK / 4) : u % RP * 4;
            k[i] = KC ? u % (BK / 4) * 4 : u / RP;
            ok[i] = r[i] < valid_r; // a multiple of 4 rows where pieces run along them
            p[i] = base + (ok[i] ? KC ? r[i] * ld + k[i] : k[i] * ld + r[i] : 0);
        }
    }
    __device__ void load(int slot, int64_t ld, int k0, int K)
    {
#pragma unroll
        for (int i = 0; i < NP; ++i) // along k: K is a multiple of 8
            v[slot][i] = ok[i] && k0 + k[i] < K
                             ? *reinterpret_cast<const f32x4 *>(p[i] + (KC ? k0 : k0 * ld))
                             : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ void store(int slot, float *s) const
    {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if constexpr (KC) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[(k[i] + j) * LD + r[i]] = v[slot][i][j];
            } else {
                *reinterpret_cast<f32x4 *>(s + k[i] * LD + r[i]) = v[slot][i];
            }
        }
    }
};

template <int KIND, int BT> __global__ __launch_bounds__(256) void f32_grouped_kernel(F32Grouped a)
{
    constexpr bool TN = KIND == F32_TN;
    constexpr int LD = BT + 20, MT = kF32Rows / BT; // tiles of an M-tile's rows
    __shared__ __attribute__((aligned(16))) float sA[2][BK * LD], sB[2][BK * LD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = BT == 64 ? (wave >> 1) * 32 : 0, wn = BT == 64 ? (wave & 1) * 32 : 0;
    const int wk = BT == 64 ? 0 : wave * 8; // 32: this wave's part of a step
    constexpr int KW = BT == 64 ? BK : 8;
    const int ntm = TN ? (a.M + BT - 1) / BT : 0, ntn = (a.N + BT - 1) / BT;
    GroupView view;
    if (!a.offsets) {
        view = group_view(a.src, kF32Rows);
        if (!TN)
            zero_ungrouped(view, a.src.M, a.C, (int64_t)a.N * 4);
    }
    auto at = [&](int x, int e) { return __builtin_amdgcn_readlane(x, e); };
    const int64_t total = TN            ? (int64_t)a.E * ntm * ntn
                          : a.offsets ? (int64_t)a.mtile_off[a.E] * MT * ntn
                                      : (int64_t)view.total * MT * ntn;
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
            first = a.offsets ? a.offsets[e] : at(view.start, e);
            K = (a.offsets ? a.offsets[e + 1] : at(view.end, e)) - (int)first;
        } else {
            const int m = __builtin_amdgcn_readfirstlane((int)(t / (MT * ntn)));
            int mt0, mts, end;
            if (a.offsets) {
                e = a.mtile_expert[m];
                mt0 = a.mtile_off[e] * MT;
                mts = a.mtile_off[e + 1] * MT - mt0;
                r0 = a.offsets[e];
                end = a.offsets[e + 1];
            } else {
                e = view_group(view, a.E, m);
                mt0 = at(view.mt0, e) * MT;
                mts = at(view.tiles, e) * MT;
                r0 = at(view.start, e);
                end = at(view.end, e);
            }
            const int64_t local = t - (int64_t)mt0 * ntn;
            n0 = (int)(local / mts) * BT;
            r0 += (int)(local % mts) * BT;
            rows = min(BT, end - r0);
            first = r0;
            K = a.K;
            if (rows <= 0) // the second half of a group's last M-tile
                continue;
        }
        const int cols = min(BT, a.N - n0);
        Stage<!TN, BT> A;
        Stage<KIND == F32_NT, BT> B;
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
        const int nk = (K + BK - 1) / BK;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            A.load(s, a.lda, s * BK, K);
            B.load(s, a.ldb, s * BK, K);
        }
        auto step = [&](int s, auto SLOT) {
            constexpr int slot = decltype(SLOT)::value; // of registers and of LDS
            A.store(slot, sA[slot]);
            B.store(slot, sB[slot]);
            __syncthreads();
            A.load(slot, a.lda, (s + 2) * BK, K);
            B.load(slot, a.ldb, (s + 2) * BK, K);
            const float *pa = sA[slot] + (wk + (lane >> 4)) * LD + (lane & 15) + wm;
            const float *pb = sB[slot] + (wk + (lane >> 4)) * LD + (lane & 15) + wn;
            constexpr int NK = KW / 4;
            float fa[NK][2], fb[NK][2];
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    fa[k][i] = pa[4 * k * LD + 16 * i];
                    fb[k][i] = pb[4 * k * LD + 16 * i];
                }
            // the columns as the instruction's rows: a lane then holds four
            // neighbouring columns of one row
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = Mfma<float>::mma(fb[k][j], fa[k][i], acc[i][j]);
            // the fragments of two k ahead of the products that take them
            constexpr int AHEAD = NK < 2 ? NK : 2;
            __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 0);
#pragma unroll
            for (int k = 0; k < NK - AHEAD; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 4 * AHEAD, 0);
        };
        // the buffer of step s is written again in step s + 2, after the barrier of s + 1
        for (int s = 0; s < nk; s += 2) {
            step(s, std::integral_constant<int, 0>{});
            if (s + 1 < nk)
                step(s + 1, std::integral_constant<int, 1>{});
        }
        float *C = TN ? a.C + (int64_t)e * a.M * a.N : a.C;
        auto out = [&](int i, int j, f32x4 v) {
            const int r = wm + 16 * i + (lane & 15), c = wn + 16 * j + (lane >> 4) * 4;
            if (r < rows && c < cols) // cols is a multiple of 8
                *reinterpret_cast<f32x4 *>(C + (int64_t)(r0 + r) * a.N + n0 + c) = v;
        };
        __syncthreads(); // every wave is past its reads: the buffers may be written
        if constexpr (BT == 64) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    out(i, j, acc[i][j]);
        } else {
            // wave w sums block w, in the order of the waves
            f32x4 *red = reinterpret_cast<f32x4 *>(wave < 2 ? sA[0] : sB[0]) + (wave & 1) * 256;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                red[b * 64 + lane] = acc[b >> 1][b & 1];
            __syncthreads();
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v += (reinterpret_cast<const f32x4 *>(w < 2 ? sA[0] : sB[0]) + (w & 1) * 256)[wave * 64 + lane];
            out(wave >> 1, wave & 1, v);
            __syncthreads();
        }
    }
}

} // namespace f32

// Tiles of 32 x 32 while there are fewer than two of 64 x 64 for each CU.
hipError_t launch_f32_grouped(int kind, const F32Grouped &a, int num_cus, hipStream_t s)
{
    auto tiles = [&](int bt) {
        const int64_t ntn = (a.N + bt - 1) / bt;
        return kind == F32_TN ? (int64_t)a.E * ((a.M + bt - 1) / bt) * ntn
                              : (int64_t)a.max_mtiles * (kF32Rows / bt) * ntn;
    };
    const bool small = tiles(64) < 2 * (int64_t)num_cus;
    const int64_t n = tiles(small ? 32 : 64);
    if (n <= 0)
        return hipSuccess;
    const dim3 grid((unsigned)(n < 65536 ? n : 65536));
    auto k = kind == F32_NN   ? small ? f32::f32_grouped_kernel<F32_NN, 32> : f32::f32_grouped_kernel<F32_NN, 64>
             : kind == F32_NT ? small ? f32::f32_grouped_kernel<F32_NT, 32> : f32::f32_grouped_kernel<F32_NT, 64>
             : small          ? f32::f32_grouped_kernel<F32_TN, 32>
                              : f32::f32_grouped_kernel<F32_TN, 64>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe
