// gemm_i8.hip — grouped GEMMs on int8 codes with token and column scales.
//
//   h[p, n] = (sum_k codes[p, k] . code_e[k, n]) scale[p] scale_e[n]
//
// with the sum exact in 32 bits (Kd <= 131072) and one of three epilogues: the
// product itself in bf16 or fp32, or act = silu(gate) * up of the two panels in
// fp32, the rows gathered by the routing.  act stays in fp32 because it is
// quantised to 8 bits next, row by row, which needs the whole row's maximum: a
// rounding to bf16 first would move one code in ten by a step.
//
// All run on the 32 x 32 x 32 matrix instruction with the weights as the first
// operand (its rows are weight columns) and the token rows as the second: a lane
// then holds 16 weight columns of one token, in groups of four neighbours.
#include "group_view.h"
#include "i8.h"
#include "kernels.h"
#include "tile_common.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ inline i32x16 i8_mma(u32x4 w, u32x4 a, i32x16 c)
{
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, w),
                                                 __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
}

// `n` bytes from p as a buffer: loads take a scalar base, a scalar offset and
// one register of lane offset, and past the end they return zero.
__device__ inline __amdgpu_buffer_rsrc_t i8_bytes(const void *p, uint32_t n)
{
    const uint64_t b = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(n), 0x00020000);
}

// Byte of a column tile's k-step among an expert's codes: below 4 GiB (the host
// checks it), not below 2.
__device__ inline uint32_t i8_code_offset(int tile, int KS, int ks)
{
    return ((uint32_t)tile * (uint32_t)KS + (uint32_t)ks) * 1024u;
}

// Cache policy of weight loads where a group mostly has one M-tile (weights_once in
// kernels.h), so that a weight is read about once: non-temporal, past the token rows that L2
// keeps (one token through 8 of 32 experts of 7168 x 2048: 90 us without, 77 with; 128 tokens: 299
// and 273; 512 through 64 of 4096 x 1536, top 4: 264 and 247; but 128 rows a group in 64-row
// tiles, 4096 x 1536: 200 us without, 230 with).  The streaming kernel, weights out of memory,
// without and with: 32 rows of 7168 x 4096 15.3 and 14.5, 128 over 16 groups of 4096 x 1536 25.4 and 22.8,
// 160 over 8 of 2048 x 1408 10.2 and 9.2; more M-tiles a group: 33 rows of 7168 x 4096 13.5 and 15.7, 256
// over 8 groups of 7168 x 1024 24.8 and 27.4, 600 over 8 of 4096 x 1408 24.4 and 30.8, 1500 rows of 4096 x
// 1024 22.4 and 35.6.
constexpr int kOnce = 2;

// M-tiles: of the tables, or, without them (up to 64 groups), of the caller's offsets.
// SwiGLU always has the routing's tables.
struct I8Tile {
    int e, r0, end, mt0, mts; // group, its first row and end, its first M-tile and their number
};
template <bool G1> struct I8Groups {
    GroupView v;
    int total;
    __device__ I8Groups(const I8GemmArgs &a, int rows)
    {
        if (G1 || a.mtile_off) {
            total = tile::ldc(a.mtile_off, a.E);
            return;
        }
        if (!a.src.offsets) { // one group of all rows
            total = (int)((a.src.M + rows - 1) / rows);
            return;
        }
        v = group_view(a.src, rows);
        total = v.total;
        zero_ungrouped(v, a.src.M, a.out, (int64_t)a.N * a.out_bytes);
    }
    __device__ I8Tile of(const I8GemmArgs &a, int m) const
    {
        using namespace tile;
        if (G1 || a.mtile_off) {
            const int e = ldc(a.mtile_expert, m), mt0 = ldc(a.mtile_off, e);
            return {e, ldc(a.offsets, e), ldc(a.offsets, e + 1), mt0, ldc(a.mtile_off, e + 1) - mt0};
        }
        if (!a.src.offsets)
            return {0, 0, (int)a.src.M, 0, total};
        const int e = view_group(v, a.src.E, uni(m));
        auto at = [&](int x) { return __builtin_amdgcn_readlane(x, e); };
        return {e, at(v.start), at(v.end), at(v.mt0), at(v.tiles)};
    }
};

// sum * row * col stays in range wherever the whole product does.  A sum below 2^31 times a
// scale from 2^97 on could pass the largest number though the column's scale brings it back, so of a
// scale from 2^64 on 2^32 come last: what is multiplied until then lies between
// 2^(32 - 149), so nothing is lost below, and 2^127 times the column's scale.  A small scale needs
// nothing: an integer times it is a multiple of the scale's own last place.
struct I8RowScale {
    float by, last;
};
__device__ inline I8RowScale i8_row_scale(float s)
{
    const bool large = fabsf(s) >= 0x1p64f;
    return {large ? s * 0x1p-32f : s, large ? 0x1p32f : 1.f};
}
__device__ inline float i8_scaled(int sum, I8RowScale row, float col)
{
    return (float)sum * row.by * col * row.last;
}
// Four neighbouring columns of a token from their sums.
__device__ inline f32x4 i8_scaled(const i32x16 &acc, int q, I8RowScale row, f32x4 col)
{
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = i8_scaled(acc[4 * q + i], row, col[i]);
    return v;
}
__device__ inline f32x4 i8_swiglu(f32x4 g, f32x4 u)
{
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = silu_f(g[i]) * u[i];
    return v;
}

// First output column of a column tile of the product (which counts through the
// panels), and the end of its panel.
struct I8Columns {
    int first, end;
};
__device__ inline I8Columns i8_columns(const I8GemmArgs &a, int tile)
{
    const int panel = tile >= a.NT ? 1 : 0, pc = a.N / a.panels;
    return {panel * pc + (tile - panel * a.NT) * 32, (panel + 1) * pc};
}

// Weight streaming kernel.  A tile is 32 token rows of one group times CT column
// tiles (SwiGLU: half gate and the same up tiles); the WV waves split the
// contraction, each streaming its part of the weights from memory straight into
// registers with the next D - 1 pairs of k-steps in flight, across the end of a tile
// too, and are summed through LDS at the end.  Bound by the weights' bytes and, below 100 MB
// of them, by the launch and the first loads: with weights out of memory one row of 7168 x
// 4096 8.8 us (3.3 TB/s), of 4096 x 28672 24.0 (4.9), 32 rows of 1024 x 8192 4.9.
template <int CT> struct I8Part {
    u32x4 w[CT][2]; // [tile][k-step]
    u32x4 a[2];
};

template <int KIND, int CT, int WV, int D, int POLICY>
__global__ __launch_bounds__(64 * WV, 8 / WV > 1 ? 8 / WV : 1) void i8_stream_kernel(I8GemmArgs a)
{
    using namespace tile;
    constexpr bool G1 = KIND == I8_SWIGLU;
    __shared__ i32x4 red[WV][CT][4][64]; // [wave][tile][register / 4][lane]
    const int lane = threadIdx.x & 63;
    const int wave = uni(threadIdx.x >> 6);
    const int h = lane >> 5;
    constexpr int PER = G1 ? CT / 2 : CT; // column tiles of a panel
    const int ntt = G1 ? a.NT : a.NT * a.panels;
    const int ncg = (ntt + PER - 1) / PER;
    const I8Groups<G1> groups(a, 32);
    const int64_t total = (int64_t)groups.total * ncg;
    // an XCD's workgroups (blockIdx % 8) take a contiguous part of the tiles, so
    // a group's token rows stay in one L2
    const int xcd = blockIdx.x & 7;
    const int64_t t1 = total * (xcd + 1) / 8;
    // the wave's k-step pairs [p0, p1)
    const int KP = a.KS >> 1;
    const int p0 = KP * wave / WV, p1 = KP * (wave + 1) / WV;

    struct Place {
        int e, cg, nr, row;
        uint32_t ao;                    // this lane's token row
        float as;                       // and its scale
        __amdgpu_buffer_rsrc_t ac, wc;  // token rows, the group's weights
        int tile[CT];                   // column tiles, counted from there
    };
    const int64_t etiles = (int64_t)a.NT * a.panels; // of a group's weights
    auto column_tile = [&](int cg, int j) { // SwiGLU: gate tiles, then their up tiles
        return min(cg * PER + j % PER, ntt - 1) + (G1 ? j / PER * a.NT : 0);
    };
    auto place = [&](int64_t t, Place &q) {
        const int m = (int)(t / ncg);
        q.cg = uni((int)(t - (int64_t)m * ncg));
        const I8Tile g = groups.of(a, m);
        q.e = g.e;
        const int r0 = g.r0 + (m - g.mt0) * 32;
        q.nr = min(32, g.end - r0);
        const int r = min(lane & 31, q.nr - 1);
        q.row = r0 + r;
        const int64_t arow = G1 ? a.sorted_slot[q.row] / a.topk : q.row;
        q.as = a.ascales[arow];
        const int64_t first = G1 ? 0 : r0, n = G1 ? a.M : q.nr;
        q.ac = i8_bytes(a.acodes + first * (a.KS * 32), (uint32_t)(n * (a.KS * 32)));
        q.ao = (uint32_t)(arow - first) * (uint32_t)(a.KS * 32) + h * 16;
        q.wc = i8_bytes(a.wcodes + g.e * etiles * a.KS * 1024, (uint32_t)(etiles * a.KS * 1024));
#pragma unroll
        for (int j = 0; j < CT; ++j)
            q.tile[j] = column_tile(q.cg, j);
    };
    const uint32_t wl = lane * 16;
    auto load = [&](const Place &q, int p, I8Part<CT> &x) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            x.a[s] = __builtin_amdgcn_raw_buffer_load_b128(q.ac, q.ao + s * 32, p * 64, 0);
#pragma unroll
            for (int j = 0; j < CT; ++j)
                x.w[j][s] = __builtin_amdgcn_raw_buffer_load_b128(
                    q.wc, wl + s * 1024, i8_code_offset(q.tile[j], a.KS, p * 2), POLICY);
        }
    };
    int64_t t = total * xcd / 8 + (blockIdx.x >> 3);
    if (t >= t1)
        return;
    Place q;
    I8Part<CT> x[D];
    auto first = [&] {
        place(t, q);
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (p0 + d < p1)
                load(q, p0 + d, x[d]);
    };
    first();
    while (true) {
        i32x16 acc[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[j][i] = 0;
        for (int p = p0; p < p1; p += D)
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (p + d < p1) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int j = 0; j < CT; ++j)
                            acc[j] = i8_mma(x[d].w[j][s], x[d].a[s], acc[j]);
                    if (p + d + D < p1)
                        load(q, p + d + D, x[d]);
                }
        const int cg = q.cg, nr = q.nr, row = q.row, e = q.e;
        const I8RowScale as = i8_row_scale(q.as);
        t += gridDim.x >> 3;
        if (t < t1)
            first();
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                red[wave][j][r][lane] =
                    i32x4{acc[j][4 * r], acc[j][4 * r + 1], acc[j][4 * r + 2], acc[j][4 * r + 3]};
        __syncthreads();
        const bool live = (lane & 31) < nr;
        // four columns of a token: tile j, register group r
        auto sum = [&](int j, int r) {
            i32x4 v = red[0][j][r][lane];
#pragma unroll
            for (int w = 1; w < WV; ++w)
                v += red[w][j][r][lane];
            const f32x4 cs = *reinterpret_cast<const f32x4 *>(
                a.wscales + (e * etiles + column_tile(cg, j)) * 32 + 8 * r + 4 * h);
            f32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = i8_scaled(v[i], as, cs[i]);
            return o;
        };
        for (int it = wave; it < PER * 4; it += WV) {
            const int j = it >> 2, r = it & 3;
            const f32x4 o = G1 ? i8_swiglu(sum(j, r), sum(j + PER, r)) : sum(j, r);
            const I8Columns cols = G1 ? I8Columns{(cg * PER + j) * 32, a.N}
                                      : i8_columns(a, column_tile(cg, j));
            const int col = cols.first + 8 * r + 4 * h;
            if (!live || cg * PER + j >= ntt || col >= cols.end)
                continue;
            const int64_t at = (int64_t)row * a.N + col;
            if constexpr (KIND == I8_BF16)
                *reinterpret_cast<bf16x4 *>(static_cast<bf16 *>(a.out) + at) =
                    bf16x4{(bf16)o[0], (bf16)o[1], (bf16)o[2], (bf16)o[3]};
            else
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = o;
        }
        if (t >= t1)
            return;
        __syncthreads();
    }
}

// Tile kernel.  A tile is 32 TF token rows of one group times eight column tiles,
// two a wave: SwiGLU a gate tile and the up tile of the same columns (so the
// epilogue stays in the wave), else two neighbours.  The weights go from memory
// straight into registers, since the waves share none; the token rows, which
// all four waves read, are copied into a ring of LDS stages of two k-steps, 64
// bytes a row, swizzled so that the 32 rows of a fragment read spread over all banks.
//
// Long products are bound by power: 65536 x 7168 x 4096 over 32 groups 1775 us, 2.17 POP/s,
// matrix cores busy 65 % at 1.4 GHz; 8192^3 457 to 475 us, 2.3 to 2.4 (a library product
// 2.5).  Short contractions are bound by what a tile has beside its products, first
// loads and stores: 24576 x 1408 x 2048 over 64 groups 80 to 100 us, cores busy 31 % at 2.2 GHz;
// of GEMM1 of 4096 x 2048 x 1408, 64 experts, top 6, 199 us, the stores are 22 and cold
// weights 33, without both 159.
template <int KIND, int TF, int POLICY>
__global__ __launch_bounds__(256, 2) void i8_tile_kernel(I8GemmArgs a)
{
    using namespace tile;
    constexpr bool G1 = KIND == I8_SWIGLU;
    constexpr int ROWS = TF * 32, STAGE = ROWS * 64, RING = 4;
    constexpr int NC = TF / 2; // token copies of a wave and stage
    constexpr int NL = 4;      // weight loads of a wave and stage
    __shared__ __attribute__((aligned(1024))) unsigned char smem[RING * STAGE];
    const int wave = uni(threadIdx.x >> 6);
    constexpr int PER = G1 ? 4 : 8; // column tiles of a panel
    const int ntt = G1 ? a.NT : a.NT * a.panels;
    const int ncg = (ntt + PER - 1) / PER;
    const int KP = a.KS >> 1; // stages
    const I8Groups<G1> groups(a, ROWS);
    const int total = uni(groups.total) * ncg; // below 2^31 (checked at launch)
    const int64_t etiles = (int64_t)a.NT * a.panels;
    const int xcd = blockIdx.x & 7;
    const int t1 = (int)((int64_t)total * (xcd + 1) / 8), dt = gridDim.x >> 3;
    // group-major; inside a group groups of up to GM M-tiles, column groups outer
    // and M-tiles inner, so that tiles in flight share weights and rows (65536 x 7168
    // x 4096 over 32 groups: 1900 us with 4, 1803 with 8, 1770 with 16; 24576 x 1408 x
    // 2048 over 64 and 8192^3: the same within 1 %)
    constexpr int GM = 16;
    struct Place {
        int e, cg, r0, nr; // group, column group, first row, rows
    };
    auto place = [&](int t) {
        Place q;
        const I8Tile g = groups.of(a, uni((int)((unsigned)t / (unsigned)ncg)));
        q.e = uni(g.e);
        const unsigned local = t - g.mt0 * ncg;
        const int grp = uni(local / (unsigned)(GM * ncg));
        const unsigned gm = min(g.mts - grp * GM, GM);
        const unsigned rr = local - grp * GM * ncg;
        q.cg = uni(rr / gm);
        const int mt = grp * GM + (int)(rr - q.cg * gm);
        q.r0 = uni(g.r0 + mt * ROWS);
        q.nr = uni(min(ROWS, g.end - q.r0));
        return q;
    };
    int t = (int)((int64_t)total * xcd / 8) + (blockIdx.x >> 3);
    if (t >= t1)
        return;
    Place next = place(t);
    for (; t < t1; t += dt) {
        // what depends on the lane alone is formed anew for each tile: kept
        // across the tiles it would not fit beside the accumulators
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int h = lane >> 5, fr = lane & 31;
        const int e = next.e, cg = next.cg, r0 = next.r0, nr = next.nr;

        // a copy moves 1024 bytes, 16 rows.  Byte offsets of this lane's sources
        // from a scalar base (SwiGLU: all of x's codes, below 4 GiB; else the tile's
        // first row).
        const int64_t first = G1 ? 0 : r0;
        auto row_of = [&](int r) -> uint32_t {
            r = min(r, nr - 1);
            return G1 ? a.sorted_slot[r0 + r] / a.topk : r;
        };
        const uint8_t *const bc = a.acodes + first * (a.KS * 32);
        uint32_t src[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = (wave * NC + i) * 16 + (lane >> 2);
            src[i] = row_of(r) * (uint32_t)(a.KS * 32) + aswz<4>(r, lane & 3) * 16;
        }
        const auto wc = i8_bytes(a.wcodes + e * etiles * a.KS * 1024, (uint32_t)(etiles * a.KS * 1024));
        int tl[2]; // the wave's column tiles
#pragma unroll
        for (int j = 0; j < 2; ++j)
            tl[j] = uni(min(cg * PER + (G1 ? wave : 2 * wave + j), ntt - 1) + (G1 ? j * a.NT : 0));
        const uint32_t wl = lane * 16;
        // copies of stage p (past the end: of the last one, into a stage that is not read again)
        auto copy = [&](int p) {
            unsigned char *st = smem + (p & (RING - 1)) * STAGE;
            const int q = min(p, KP - 1);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                g2l16s(bc + q * 64, src[i], (lds_void *)(st + (wave * NC + i) * 1024));
        };
        struct W {
            u32x4 c[2][2];
        };
        auto load_w = [&](int p, W &w) {
            const int q = min(p, KP - 1) * 2;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    w.c[j][s] = __builtin_amdgcn_raw_buffer_load_b128(
                        wc, wl + s * 1024, i8_code_offset(tl[j], a.KS, q), POLICY);
        };
        i32x16 acc[2][TF];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[j][f][i] = 0;
        auto compute = [&](int p, const W &w) {
            const unsigned char *st = smem + (p & (RING - 1)) * STAGE;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int f = 0; f < TF; ++f) {
                    const int r = f * 32 + fr;
                    const u32x4 av =
                        *reinterpret_cast<const u32x4 *>(st + r * 64 + aswz<4>(r, 2 * s + h) * 16);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[j][f] = i8_mma(w.c[j][s], av, acc[j][f]);
                }
        };
        W w0, w1;
        copy(0);
        load_w(0, w0);
        copy(1);
        load_w(1, w1);
        next = place(min(t + dt, t1 - 1)); // under the first loads
        wait_vm<NC + 2 * NL>();
        lds_barrier();
        // Stage p: its copies and weights were issued two stages ago.  The
        // copies of p + 2 precede the weights' loads of p + 2, so waiting for
        // all but the youngest operations covers the copies of p + 1.
        constexpr int YOUNG = 2 * NL + NC;
        int p = 0;
        for (; p + 2 <= KP; p += 2) {
            compute(p, w0);
            copy(p + 2);
            load_w(p + 2, w0);
            wait_vm<YOUNG>();
            lds_barrier();
            compute(p + 1, w1);
            copy(p + 3);
            load_w(p + 3, w1);
            wait_vm<YOUNG>();
            lds_barrier();
        }
        if (p < KP)
            compute(p, w0);
        wait_vm<0>();
        lds_barrier();
        // the last barrier: every wave is past its reads, so the next tile may copy.
        // The 32 columns of a column tile are turned in LDS, 32 rows at a time, so
        // that a store instruction writes whole lines: of four row fragments the
        // turn lies in the ring's last two stages, which the next tile's copies
        // reach after a barrier; of two it takes the whole ring.
        unsigned char *const turn = smem + (TF == 4 ? 2 * STAGE : 0) + wave * 4096;
        f32x4 cs[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                cs[j][q] = *reinterpret_cast<const f32x4 *>(a.wscales + (e * etiles + tl[j]) * 32 +
                                                            8 * q + 4 * h);
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const I8RowScale rs = i8_row_scale(a.ascales[first + row_of(f * 32 + fr)]);
            if constexpr (KIND == I8_BF16) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = i8_scaled(acc[j][f], q, rs, cs[j][q]);
                        const bf16x4 o = {(bf16)v[0], (bf16)v[1], (bf16)v[2], (bf16)v[3]};
                        *reinterpret_cast<bf16x4 *>(turn + fr * 128 + aswz<8>(fr, j * 4 + q) * 16 +
                                                    h * 8) = o;
                    }
                asm volatile("" ::: "memory"); // a wave's LDS operations complete in order
                const int part = lane & 7, j = part >> 2; // 16 bytes: eight columns
                const I8Columns cols = i8_columns(a, tl[0] + j);
                const int col = cols.first + (part & 3) * 8;
                const bool in = cg * PER + 2 * wave + j < ntt && col < cols.end;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rl = i * 8 + (lane >> 3), r = f * 32 + rl;
                    const u32x4 v =
                        *reinterpret_cast<const u32x4 *>(turn + rl * 128 + aswz<8>(rl, part) * 16);
                    if (r < nr && in) {
                        u32x4 *dst = reinterpret_cast<u32x4 *>(static_cast<bf16 *>(a.out) +
                                                               (int64_t)(r0 + r) * a.N + col);
                        if (a.stream_out)
                            __builtin_nontemporal_store(v, dst);
                        else
                            *dst = v;
                    }
                }
                asm volatile("" ::: "memory");
            } else {
#pragma unroll
                for (int j = 0; j < (G1 ? 1 : 2); ++j) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 v = i8_scaled(acc[j][f], q, rs, cs[j][q]);
                        if constexpr (G1)
                            v = i8_swiglu(v, i8_scaled(acc[1][f], q, rs, cs[1][q]));
                        *reinterpret_cast<f32x4 *>(turn + fr * 128 + aswz<8>(fr, 2 * q + h) * 16) = v;
                    }
                    asm volatile("" ::: "memory");
                    const int part = lane & 7; // 16 bytes: four columns
                    const I8Columns cols = G1 ? I8Columns{tl[0] * 32, a.N} : i8_columns(a, tl[j]);
                    const int col = cols.first + part * 4;
                    const bool in = cg * PER + (G1 ? wave : 2 * wave + j) < ntt && col < cols.end;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rl = i * 8 + (lane >> 3), r = f * 32 + rl;
                        const u32x4 v =
                            *reinterpret_cast<const u32x4 *>(turn + rl * 128 + aswz<8>(rl, part) * 16);
                        if (r < nr && in) {
                            u32x4 *dst = reinterpret_cast<u32x4 *>(static_cast<float *>(a.out) +
                                                                   (int64_t)(r0 + r) * a.N + col);
                            if (a.stream_out)
                                __builtin_nontemporal_store(v, dst);
                            else
                                *dst = v;
                        }
                    }
                    asm volatile("" ::: "memory");
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F); // LDS only: writes of rows past nr had no reader
        if (TF == 2)
            lds_barrier();
    }
}

template <int KIND>
static void i8_launch(const I8GemmArgs &a, int num_cus, hipStream_t s)
{
    constexpr bool G1 = KIND == I8_SWIGLU;
    const int ntt = G1 ? a.NT : a.NT * a.panels;
    auto run = [&](auto *kernel, int per, int threads, int groups_a_cu) {
        const int64_t most = (int64_t)a.max_mtiles * ((ntt + per - 1) / per);
        int64_t grid = (int64_t)num_cus * groups_a_cu;
        if (most < grid)
            grid = most;
        grid = (grid + 7) / 8 * 8; // a whole number of workgroups for each XCD
        hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3((unsigned)threads), 0, s, a);
    };
    if (a.BM == 32) {
        // tiles of two column tiles by four waves, if there is one for each CU; else a
        // single one (SwiGLU: a pair) by eight
        const bool two = (int64_t)a.max_mtiles * (G1 ? ntt : (ntt + 1) / 2) >= num_cus;
        if (two && a.once)
            run(i8_stream_kernel<KIND, 2, 4, 4, kOnce>, G1 ? 1 : 2, 256, 2);
        else if (two)
            run(i8_stream_kernel<KIND, 2, 4, 4, 0>, G1 ? 1 : 2, 256, 2);
        else if (a.once)
            run(i8_stream_kernel<KIND, G1 ? 2 : 1, 8, 4, kOnce>, 1, 512, 2);
        else
            run(i8_stream_kernel<KIND, G1 ? 2 : 1, 8, 4, 0>, 1, 512, 2);
    } else if (a.BM == 64) {
        if (a.once)
            run(i8_tile_kernel<KIND, 2, kOnce>, G1 ? 4 : 8, 256, 2);
        else
            run(i8_tile_kernel<KIND, 2, 0>, G1 ? 4 : 8, 256, 2);
    } else {
        run(i8_tile_kernel<KIND, 4, 0>, G1 ? 4 : 8, 256, 2);
    }
}

hipError_t launch_i8_gemm(int kind, const I8GemmArgs &a, int num_cus, hipStream_t s)
{
    const int64_t columns = (int64_t)a.NT * a.panels;
    if (a.max_mtiles * columns >= ((int64_t)1 << 31))
        return hipErrorInvalidValue;
    if (a.max_mtiles == 0)
        return hipSuccess;
    if (kind == I8_SWIGLU)
        i8_launch<I8_SWIGLU>(a, num_cus, s);
    else if (kind == I8_BF16)
        i8_launch<I8_BF16>(a, num_cus, s);
    else
        i8_launch<I8_F32>(a, num_cus, s);
    return hipGetLastError();
}

} // namespace moe
