// gemm_mx.hip — grouped GEMMs of the expert FFN on MXFP4 weights.
//
// GEMM1: act[p, :] = silu(g) * u, [g u] = x[token(p)] . W1[e], quantised to the
// activation format in the epilogue; GEMM2: o[p, :] = act[p] . W2[e], bf16.
// Both run on the scaled matrix instruction of 32 x 32 x 64 (mx.h) with the
// weights as the first operand (its rows are weight columns) and the token rows
// as the second: a lane then holds 16 weight columns of one token, so a block
// of 32 act columns is two lanes' registers and its scale needs one exchange.
#include "kernels.h"
#include "mx.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A lane's codes of one block of the token operand.
template <int BITS> struct MxFrag {
    u32x4 c;
    u32x2 t; // e2m3 only
};

// One k-step: weights e2m1, tokens e2m1 (BITS 4) or e2m3 (BITS 6); S picks the
// scale byte of both operands.
template <int BITS, int S>
__device__ inline f32x16 mx_mma(u32x4 w, int ws, const MxFrag<BITS> &a, int as, f32x16 c)
{
    const i32x8 wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    if constexpr (BITS == 4) {
        const i32x8 av = {(int)a.c[0], (int)a.c[1], (int)a.c[2], (int)a.c[3], 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 4, 4, S, ws, S, as);
    } else {
        const i32x8 av = {(int)a.c[0], (int)a.c[1], (int)a.c[2], (int)a.c[3],
                          (int)a.t[0], (int)a.t[1], 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, av, c, 4, 2, S, ws, S, as);
    }
}

// Register i of lane l of a 32 x 32 result is weight column
// 8 (i / 4) + 4 (l / 32) + i % 4 of token l % 32.  Exchanges with the lane's
// partner so that it holds the 16 consecutive columns 16 (l / 32) + [0, 16).
__device__ inline void gather_columns(float *v)
{
    float w[16];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the low half keeps column group p and gets its partner's; the
            // high half keeps group p + 2
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[4 * p + i]),
                                                            __float_as_uint(v[4 * (p + 2) + i]),
                                                            false, false);
            w[8 * p + i] = __uint_as_float(r[0]);
            w[8 * p + 4 + i] = __uint_as_float(r[1]);
        }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = w[i];
}

// Where GEMM1 writes a row of its output.
struct ActRow {
    uint8_t *codes, *tails, *scales;
};
template <int BITS> __device__ inline ActRow act_row(const MxGemmArgs &a, int64_t row)
{
    return {a.act_codes + row * (a.act_KS * 32),
            BITS == 6 ? a.act_tails + row * (a.act_KS * 16) : nullptr,
            a.act_scales + row * (a.act_KC * 8)};
}

// SwiGLU of one 32-column block of one token and its quantisation.  The 32
// values never leave fp32 before they are rounded to the block format.
template <int BITS>
__device__ inline void store_act(const f32x16 &g, const f32x16 &u, const ActRow &r, int block,
                                 bool store)
{
    const int h = (threadIdx.x >> 5) & 1;
    float v[16];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = silu_f(g[i]) * u[i];
        top = max(top, abs_bits(v[i]));
    }
    const auto other = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    top = max(other[0], other[1]);
    const int code = mx_scale_code(top);
    const float inv = mx_inverse(code);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] *= inv;
    gather_columns(v);
    if constexpr (BITS == 4) {
        const u32x2 out = {mx_pack8_fp4(v), mx_pack8_fp4(v + 8)};
        if (store)
            *reinterpret_cast<u32x2 *>(r.codes + block * 16 + h * 8) = out;
    } else {
        // 96 bits a lane: dwords 0-2 of the block's six from the low half
        const u32x6 c = mx_pack_fp6<16>(v);
        if (store && h == 0) {
            *reinterpret_cast<u32x2 *>(r.codes + block * 16) = u32x2{c[0], c[1]};
            *reinterpret_cast<uint32_t *>(r.codes + block * 16 + 8) = c[2];
        }
        if (store && h == 1) {
            *reinterpret_cast<uint32_t *>(r.codes + block * 16 + 12) = c[0];
            *reinterpret_cast<u32x2 *>(r.tails + block * 8) = u32x2{c[1], c[2]};
        }
    }
    if (store && h == 0)
        r.scales[mx_scale_at(block)] = (uint8_t)code;
}

// The block behind the last one where their number is odd (the second half of
// the last k-step).
template <int BITS> __device__ inline void store_empty(const ActRow &r, int block)
{
    const int h = (threadIdx.x >> 5) & 1;
    *reinterpret_cast<u32x2 *>(r.codes + block * 16 + h * 8) = u32x2{0u, 0u};
    if (h == 0) {
        if constexpr (BITS == 6)
            *reinterpret_cast<u32x2 *>(r.tails + block * 8) = u32x2{0u, 0u};
        r.scales[mx_scale_at(block)] = 0;
    }
}

// Weight streaming kernel.  A tile is 32 token rows of one expert times four
// column tiles (GEMM1: two gate and the same two up tiles); the four waves
// split the contraction, each streaming its part of the weights from memory
// straight into registers, and are summed through LDS at the end.
template <int BITS, bool G1>
__global__ __launch_bounds__(256, 2) void mx_stream_kernel(MxGemmArgs a)
{
    __shared__ f32x4 red[4][3][4][64]; // [tile][other wave][register / 4][lane]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5;
    constexpr int PER = G1 ? 2 : 4; // column tiles of a panel
    const int ncg = (a.NT + PER - 1) / PER;
    const int64_t total = (int64_t)a.mtile_off[a.E] * ncg;
    // an XCD's workgroups (blockIdx % 8) take a contiguous part of the tiles,
    // so an expert's token rows stay in one L2
    const int xcd = blockIdx.x & 7;
    const int64_t t1 = total * (xcd + 1) / 8;
    for (int64_t t = total * xcd / 8 + (blockIdx.x >> 3); t < t1; t += gridDim.x >> 3) {
        const int m = (int)(t / ncg), cg = (int)(t - (int64_t)m * ncg);
        const int e = a.mtile_expert[m];
        const int r0 = a.offsets[e] + (m - a.mtile_off[e]) * 32;
        const int nr = min(32, a.offsets[e + 1] - r0);
        const int row = r0 + min(lane & 31, nr - 1);
        const int64_t arow = G1 ? a.sorted_slot[row] / a.topk : row;
        const uint8_t *ac = a.acodes + arow * (a.KS * 32) + h * 16;
        const uint8_t *at = BITS == 6 ? a.atails + arow * (a.KS * 16) + h * 8 : nullptr;
        const uint8_t *as = a.ascales + arow * (a.KC * 8) + h * 4;
        const uint8_t *wc[4], *ws[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = min(cg * PER + (G1 ? j >> 1 : j), a.NT - 1);
            const int64_t tile = ((int64_t)e * (G1 ? 2 : 1) + (G1 ? j & 1 : 0)) * a.NT + c;
            wc[j] = a.wcodes + tile * a.KS * 1024 + lane * 16;
            ws[j] = a.wscales + tile * a.KC * 256 + lane * 4;
        }
        f32x16 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[j][i] = 0.f;
        const int c0 = a.KC * wave / 4, c1 = a.KC * (wave + 1) / 4;
        for (int kc = c0; kc < c1; ++kc) {
            int wsc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wsc[j] = *reinterpret_cast<const int *>(ws[j] + (int64_t)kc * 256);
            const int asc = *reinterpret_cast<const int *>(as + kc * 8);
            auto step = [&](auto S) {
                constexpr int s = decltype(S)::value;
                const int ks = kc * 4 + s;
                if (ks >= a.KS)
                    return;
                MxFrag<BITS> av;
                av.c = *reinterpret_cast<const u32x4 *>(ac + ks * 32);
                if constexpr (BITS == 6)
                    av.t = *reinterpret_cast<const u32x2 *>(at + ks * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(wc[j] + (int64_t)ks * 1024);
                    acc[j] = mx_mma<BITS, s>(w, wsc[j], av, asc, acc[j]);
                }
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        }
        // wave w sums tile w
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j != wave) {
                const int slot = wave < j ? wave : wave - 1;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    red[j][slot][q][lane] =
                        f32x4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
            }
        __syncthreads();
        f32x16 sum;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == wave)
                sum = acc[j];
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 v = red[wave][s][q][lane];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[4 * q + i] += v[i];
            }
        const bool live = (lane & 31) < nr;
        if constexpr (G1) {
            __syncthreads();
            if (wave & 1) { // the up tile goes to the wave of its gate tile
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    red[wave][0][q][lane] =
                        f32x4{sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]};
            }
            __syncthreads();
            if (!(wave & 1)) {
                f32x16 up;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 v = red[wave + 1][0][q][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        up[4 * q + i] = v[i];
                }
                const int c = cg * 2 + (wave >> 1);
                const ActRow r = act_row<BITS>(a, row);
                store_act<BITS>(sum, up, r, c, live && c < a.NT);
                if (c == a.NT - 1 && c + 1 < 2 * a.act_KS && live)
                    store_empty<BITS>(r, c + 1);
            }
        } else {
            const int c = cg * 4 + wave;
            bf16 *orow = static_cast<bf16 *>(a.o) + (int64_t)row * a.N;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = c * 32 + 8 * q + 4 * h;
                if (live && col < a.N) {
                    typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
                    const bf16x4 out = {(bf16)sum[4 * q], (bf16)sum[4 * q + 1],
                                        (bf16)sum[4 * q + 2], (bf16)sum[4 * q + 3]};
                    *reinterpret_cast<bf16x4 *>(orow + col) = out;
                }
            }
        }
        __syncthreads();
    }
}

hipError_t launch_mx_gemm(bool g1, int bits, const MxGemmArgs &a, int num_cus, hipStream_t s)
{
    const int per = g1 ? 2 : 4;
    const int64_t most = (int64_t)a.max_mtiles * ((a.NT + per - 1) / per);
    int64_t grid = (int64_t)num_cus * 16;
    if (most < grid)
        grid = most;
    grid = (grid + 7) / 8 * 8;
    auto k = g1 ? (bits == 4 ? mx_stream_kernel<4, true> : mx_stream_kernel<6, true>)
                : (bits == 4 ? mx_stream_kernel<4, false> : mx_stream_kernel<6, false>);
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe
