// gemm_rows.hip — grouped products of few rows a group, bf16 or fp32, where reading the
// weights once is the whole time:
//
//   y[m] = x[m] . W[e]      W [E, K, N], or [E, N, K] (NT)
//
// A tile is 16 TF token rows of one group times 16 P weight columns; its WV waves split
// the contraction, in steps of 32 or (bf16 NT) 64, each streaming its part of the weights from
// memory straight into registers with the next D - 1 steps in flight, across the end of a
// tile too, and are summed in the order of the waves through LDS at the end.  Every step
// issues all its loads, those past the end for zeros from nowhere, so that the waits
// count loads instead of emptying the queue.
//
// The weights are the first operand of the 16 x 16 x 32 instruction, of which a lane
// holds 8 k of one column.  Of [K, N] weights a lane loads P neighbouring columns of 8
// rows and turns that block in registers: column j of the block belongs to instruction
// j, so instruction j covers the columns P r + j of the tile, r < 16.  Of [N, K] weights
// a lane's load is 8 k of one column already, two of them one after the other, so that
// the four lanes of a column take 128 bytes together; the columns are dealt to the
// instructions alike, so that both end with P neighbouring columns of a token in a lane's
// registers.  In fp32 an instruction (16 x 16 x 4) takes one k of each lane, so nothing is
// turned: k 8 q + i of lane group q meet in instruction i, from one row of [K, N] weights
// each or from the two loads of a column of [N, K].
//
// Bound by the weights' bytes where every CU has tiles (8 rows over 8 of 32 groups of 7168 x
// 4096: 470 MB in 88 us, 5.4 TB/s; as [N, K] 108 us, for pieces of 128 bytes); with fewer
// tiles by the rate of a CU's scattered loads (1 row of 7168 x 4096, 128 workgroups:
// 59 MB in 30 us, as [N, K] 24; more steps in flight or fewer, wider tiles made it no
// shorter: 30 to 35 us); in small ones by the length of the chain (16 x 512 x 256 over 8
// groups: 5.9 us).  fp32: 8 rows over 8 of 32 groups of 2048 x 2816, 185 MB, 41 us; 31 as [N,
// K].
#include "common.h"
#include "group_view.h"
#include "kernels.h"
#include "tile_common.h"

namespace moe {
namespace rows {

constexpr uint32_t kOutside = 0xFFFFFFF0u; // a buffer offset past any matrix: loads zeros
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};
// [K, N] weights that are read about once (weights_once in kernels.h) are loaded non-temporally,
// past the token rows that L2 keeps: 8 rows of 7168 x 4096 over 8 groups 89 us against 98 without,
// 128 of 4096 x 1536 over 16 42 against 45, fp32 8 of 2048 x 2816 over 32 50 against 54; but with more M-tiles a
// group, and so more reads of them, 48 rows of 7168 x 4096 46 us against 35.5 without, 512 over 8
// groups of 7168 x 1024 93.5 against 75, 5000 of 4096 x 256 63 against 38.  Of [N, K] weights the two loads that
// share a line come apart by it (132 us against 109 without).
constexpr int kOnce = 2;

// One step of a wave: KL k of each lane, of the weights and of the token rows.
template <typename T, bool NT, int P, int TF> struct Step {
    static constexpr int KL = sizeof(T) == 2 && NT ? 16 : 8;
    static constexpr int NL = NT ? 2 * P : 8, DW = NT ? 4 : P * sizeof(T) / 4; // loads, dwords of each
    static constexpr int XL = KL * sizeof(T) / 16;                             // loads of a token row
    uint32_t w[NL][DW];
    u32x4 x[XL][TF];

    __device__ void sum(f32x4 (&acc)[TF][P]) const
    {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int h = 0; h < XL; ++h)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const bf16x8 c = column(h, j);
#pragma unroll
                    for (int f = 0; f < TF; ++f)
                        acc[f][j] = Mfma<bf16>::mma(c, __builtin_bit_cast(bf16x8, x[h][f]), acc[f][j]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j)
#pragma unroll
                    for (int f = 0; f < TF; ++f) {
                        const uint32_t c = NT ? w[2 * j + i / 4][i % DW] : w[i][j % DW];
                        const uint32_t r = x[i / 4][f][i % 4]; // not cast in the vector: that takes its first
                        acc[f][j] = Mfma<float>::mma(__builtin_bit_cast(float, c), __builtin_bit_cast(float, r),
                                                     acc[f][j]);
                    }
        }
    }
    // bf16: 8 k of column j
    __device__ bf16x8 column(int h, int j) const
    {
        u32x4 v;
        if constexpr (NT) {
            const auto &c = w[2 * j + h];
            v = u32x4{c[0], c[1], c[2], c[3]};
        } else {
            const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __builtin_amdgcn_perm(w[2 * i + 1][j >> 1], w[2 * i][j >> 1], sel);
        }
        return __builtin_bit_cast(bf16x8, v);
    }
};

// PO: cache policy
template <int DW, int PO>
__device__ inline void load_dwords(uint32_t (&d)[DW], __amdgpu_buffer_rsrc_t b, uint32_t at)
{
    if constexpr (DW == 4) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, PO);
        d[0] = v[0], d[1] = v[1], d[2] = v[2], d[3] = v[3];
    } else if constexpr (DW == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(b, at, 0, PO);
        d[0] = v[0], d[1] = v[1];
    } else {
        d[0] = __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, PO);
    }
}

template <typename T, bool NT, int P, int TF, int WV, int D, int POLICY>
__global__ __launch_bounds__(64 * WV, 8 / WV) void rows_kernel(RowsArgs a)
{
    using namespace tile;
    using S = Step<T, NT, P, TF>;
    constexpr int ROWS = 16 * TF, COLS = 16 * P, KL = S::KL, KSTEP = 4 * KL;
    constexpr int NH = KL / 8; // parts of 8 k, which are in or out of K
    constexpr uint32_t IT = sizeof(T);
    __shared__ f32x4 red[WV][TF][P][64];
    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int fr = lane & 15, q = lane >> 4;
    const int ncg = (a.N + COLS - 1) / COLS;
    const int steps = (a.K + KSTEP - 1) / KSTEP;
    GroupView view;
    if (!a.offsets) {
        view = group_view(a.src, ROWS);
        zero_ungrouped(view, a.src.M, a.C, (int64_t)a.N * IT);
    }
    const int64_t total = (int64_t)(a.offsets ? ldc(a.mtile_off, a.E) : view.total) * ncg;
    // an XCD's workgroups (blockIdx % 8) take a contiguous part of the tiles, so a group's
    // token rows stay in one L2
    const int xcd = blockIdx.x & 7;
    const int64_t t1 = total * (xcd + 1) / 8;
    int64_t t = total * xcd / 8 + (blockIdx.x >> 3);
    if (t >= t1)
        return;

    struct Place {
        int r0, nr, n0;
        __amdgpu_buffer_rsrc_t w;
        uint32_t at[NT ? P : 1]; // this lane's columns at k KL q
        const T *x[TF];          // this lane's token rows at k KL q
    };
    auto place = [&](Place &g) {
        const int m = uni((int)(t / ncg));
        int e, mt0, end;
        if (a.offsets) {
            e = ldc(a.mtile_expert, m);
            mt0 = ldc(a.mtile_off, e);
            g.r0 = ldc(a.offsets, e);
            end = ldc(a.offsets, e + 1);
        } else {
            e = view_group(view, a.E, m);
            mt0 = __builtin_amdgcn_readlane(view.mt0, e);
            g.r0 = __builtin_amdgcn_readlane(view.start, e);
            end = __builtin_amdgcn_readlane(view.end, e);
        }
        g.r0 += (m - mt0) * ROWS;
        g.nr = min(ROWS, end - g.r0);
        g.n0 = uni((int)(t - (int64_t)m * ncg)) * COLS;
        const uint64_t base = (uint64_t)(uintptr_t)(static_cast<const T *>(a.W) + (int64_t)uni(e) * a.K * a.N);
        g.w = __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)base, 0, (uint32_t)a.K * (uint32_t)a.N * IT,
                                                0x00020000);
#pragma unroll
        for (int j = 0; j < (NT ? P : 1); ++j) {
            const int n = g.n0 + fr * P + j; // N is a multiple of 8: P columns are in or out
            g.at[j] = n >= a.N ? kOutside
                      : NT     ? ((uint32_t)n * (uint32_t)a.K + KL * q) * IT
                               : ((uint32_t)(KL * q) * (uint32_t)a.N + (uint32_t)n) * IT;
        }
#pragma unroll
        for (int f = 0; f < TF; ++f)
            g.x[f] = static_cast<const T *>(a.A) + (int64_t)(g.r0 + min(f * 16 + fr, g.nr - 1)) * a.lda + KL * q;
    };
    // step p, zeros past K (a multiple of 8, so 8 k are in or out)
    auto load = [&](const Place &g, int p, S &s) {
        bool in[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h)
            in[h] = p * KSTEP + KL * q + 8 * h < a.K;
#pragma unroll
        for (int i = 0; i < S::NL; ++i) {
            const uint32_t at = g.at[NT ? i / 2 : 0];
            const uint32_t by = NT ? (uint32_t)p * (KSTEP * IT) + i % 2 * 16
                                   : ((uint32_t)p * 32u + i) * (uint32_t)a.N * IT;
            load_dwords<S::DW, POLICY>(
                s.w[i], g.w, in[i % NH] && at != kOutside ? at + by : kOutside);
        }
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int h = 0; h < S::XL; ++h)
                s.x[h][f] = *(const __attribute__((address_space(1))) u32x4 *)(uintptr_t)(
                    in[h % NH] ? (const void *)(g.x[f] + (p * KSTEP + h * (16 / (int)IT))) : (const void *)kZeros);
    };
    Place g;
    S s[D];
    auto first = [&] {
        place(g);
#pragma unroll
        for (int d = 0; d < D; ++d)
            load(g, wave + WV * d, s[d]);
    };
    first();
    while (true) {
        f32x4 acc[TF][P];
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int j = 0; j < P; ++j)
                acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int p = wave; p < steps; p += WV * D)
#pragma unroll
            for (int d = 0; d < D; ++d) {
                s[d].sum(acc);
                load(g, p + WV * (d + D), s[d]);
            }
        const int r0 = g.r0, nr = g.nr, n0 = g.n0;
        t += gridDim.x >> 3;
        if (t < t1)
            first();
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int j = 0; j < P; ++j)
                red[wave][f][j][lane] = acc[f][j];
        __syncthreads();
        // eight neighbouring columns of a token: of a lane's four results of every
        // instruction (columns P (4 q + i) + j) those of 8 / P of them
        constexpr int NI = 8 / P, PARTS = 4 / NI;
        for (int it = wave; it < TF * PARTS; it += WV) {
            const int f = it / PARTS, i0 = it % PARTS * NI;
            float o[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                o[c] = 0.f;
#pragma unroll
            for (int v = 0; v < WV; ++v)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    o[c] += reinterpret_cast<const float *>(&red[v][f][c % P][lane])[i0 + c / P];
            const int r = f * 16 + fr, n = n0 + P * (4 * q + i0);
            if (r < nr && n < a.N) {
                T *dst = static_cast<T *>(a.C) + (int64_t)(r0 + r) * a.N + n;
                if constexpr (sizeof(T) == 2) {
                    bf16x8 out;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        out[c] = (bf16)o[c];
                    *reinterpret_cast<bf16x8 *>(dst) = out;
                } else {
                    reinterpret_cast<f32x4 *>(dst)[0] = f32x4{o[0], o[1], o[2], o[3]};
                    reinterpret_cast<f32x4 *>(dst)[1] = f32x4{o[4], o[5], o[6], o[7]};
                }
            }
        }
        if (t >= t1)
            return;
        __syncthreads();
    }
}

template <typename T, bool NT, int P, int TF, int WV, int D>
static hipError_t launch(const RowsArgs &a, int num_cus, hipStream_t s)
{
    const int64_t most = (int64_t)a.max_mtiles * ((a.N + 16 * P - 1) / (16 * P));
    int64_t grid = (int64_t)num_cus * (8 / WV);
    if (most < grid)
        grid = most;
    grid = (grid + 7) / 8 * 8; // a whole number of workgroups for each XCD
    constexpr int POLICY = NT ? 0 : kOnce; // tiles of 16 rows: always once
    auto k = rows_kernel<T, NT, P, TF, WV, D, POLICY>;
    if constexpr (!NT && TF > 1)
        if (!a.once)
            k = rows_kernel<T, NT, P, TF, WV, D, 0>;
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(64 * WV), 0, s, a);
    return hipGetLastError();
}

// 128 columns of [K, N] weights in bf16 (256-byte pieces) while there are three tiles for
// four CUs, then 64, then 32: 64 rows of 4096 x 1536 over 16 groups, 204 tiles of 128, 46 us,
// by 64 columns 57; 1 row of 7168 x 4096 by 64 columns, 64 tiles, 33 us, by 32 30.  Four
// waves where a step is 8 KB, eight where it is less.
template <typename T, bool NT, int TF>
static hipError_t launch_width(const RowsArgs &a, int num_cus, hipStream_t s)
{
    auto enough = [&](int cols) { return a.max_mtiles * ((a.N + cols - 1) / cols) >= num_cus * 3 / 4; };
    constexpr bool F32 = sizeof(T) == 4;
    if constexpr (!NT && !F32)
        if (enough(128))
            return launch<T, NT, 8, TF, 4, 3>(a, num_cus, s);
    if (enough(64))
        return launch<T, NT, 4, TF, NT || F32 ? 4 : 8, 3>(a, num_cus, s);
    return launch<T, NT, 2, TF, 8, 4>(a, num_cus, s);
}

template <typename T>
static hipError_t launch_type(bool nt, int BM, const RowsArgs &a, int num_cus, hipStream_t s)
{
    if (BM == 16)
        return nt ? launch_width<T, true, 1>(a, num_cus, s) : launch_width<T, false, 1>(a, num_cus, s);
    return nt ? launch_width<T, true, 2>(a, num_cus, s) : launch_width<T, false, 2>(a, num_cus, s);
}

} // namespace rows

hipError_t launch_rows(int dtype, bool nt, int BM, const RowsArgs &a, int num_cus, hipStream_t s)
{
    if (a.max_mtiles <= 0)
        return hipSuccess;
    return dtype == 1 ? rows::launch_type<bf16>(nt, BM, a, num_cus, s)
                      : rows::launch_type<float>(nt, BM, a, num_cus, s);
}

} // namespace moe
