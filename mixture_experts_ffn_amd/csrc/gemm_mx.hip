// gemm_mx.hip — grouped GEMMs of the expert FFN on MXFP4 weights.
//
// GEMM1: act[p, :] = silu(g) * u, [g u] = x[token(p)] . W1[e], quantised to the
// activation format in the epilogue; GEMM2: o[p, :] = act[p] . W2[e], rounded to
// bf16 as in the bf16 layer: half the bytes that GEMM2 writes and the combine
// reads (0.36 of 1.84 ms for the skewed workload), for at most 2^-8 of each term.
// Both run on the scaled matrix instruction of 32 x 32 x 64 (mx.h) with the
// weights as the first operand (its rows are weight columns) and the token rows
// as the second: a lane then holds 16 weight columns of one token, so a block
// of 32 act columns is two lanes' registers and its scale needs one exchange.
#include "kernels.h"
#include "mx.h"
#include "tile_common.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));

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
            a.act_scales + row * a.act_srow};
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

// The up to three blocks from `block` to the end of the row's last k-step pair.
template <int BITS> __device__ inline void store_empty(const ActRow &r, int block, int end)
{
    const int h = (threadIdx.x >> 5) & 1;
    for (; block < end; ++block) {
        *reinterpret_cast<u32x2 *>(r.codes + block * 16 + h * 8) = u32x2{0u, 0u};
        if (h == 0) {
            if constexpr (BITS == 6)
                *reinterpret_cast<u32x2 *>(r.tails + block * 8) = u32x2{0u, 0u};
            r.scales[mx_scale_at(block)] = 0;
        }
    }
}

// `n` bytes from p as a buffer: loads take a scalar base, a scalar offset and
// one register of lane offset, and past the end they return zero.
__device__ inline __amdgpu_buffer_rsrc_t bytes_at(const void *p, uint32_t n)
{
    const uint64_t b = (uint64_t)(uintptr_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(uintptr_t)((uint64_t)hi << 32 | lo), 0,
                                             __builtin_amdgcn_readfirstlane(n), 0x00020000);
}

// Byte of a column tile's k-step among an expert's codes: below 4 GiB (the host
// checks it), not below 2.
__device__ inline uint32_t code_offset(int tile, int KS, int ks)
{
    return ((uint32_t)tile * (uint32_t)KS + (uint32_t)ks) * 1024u;
}

// The token operand of a tile of rows r0 .. r0 + nr - 1: GEMM1 gathers rows of
// x (all of them within 4 GiB of codes, which the host checks), GEMM2 reads
// consecutive rows of act.
struct TokenRows {
    __amdgpu_buffer_rsrc_t codes, tails, scales;
};
template <int BITS, bool G1>
__device__ inline TokenRows token_rows(const MxGemmArgs &a, int64_t r0, int64_t nr)
{
    const int64_t first = G1 ? 0 : r0, n = G1 ? a.T : nr;
    TokenRows t;
    t.codes = bytes_at(a.acodes + first * (a.KS * 32), (uint32_t)(n * (a.KS * 32)));
    t.tails = t.codes;
    if constexpr (BITS == 6)
        t.tails = bytes_at(a.atails + first * (a.KS * 16), (uint32_t)(n * (a.KS * 16)));
    t.scales = bytes_at(a.ascales + first * a.srow, (uint32_t)(n * a.srow));
    return t;
}

// Weight streaming kernel.  A tile is 32 token rows of one expert times four
// column tiles (GEMM1: two gate and the same two up tiles); the four waves
// split the contraction, each streaming its part of the weights from memory
// straight into registers, and are summed through LDS at the end.  What a wave
// needs is in flight two k-steps (8 KB of weights) ahead, across the end of a
// tile too: the next tile's first steps are requested before this tile's sums
// are joined.  One token through 8 of 32 experts of 7168 x 2048: 21.5 + 12.2 us
// for 187 MB of weights, the rate of a large copy and a little more.
template <int BITS> struct StreamPair {
    u32x4 w[4][2]; // [tile][k-step]
    MxFrag<BITS> a[2];
};
struct StreamScales {
    int w[4], a;
};

template <int BITS, bool G1>
__global__ __launch_bounds__(256, 2) void mx_stream_kernel(MxGemmArgs a)
{
    using namespace tile;
    __shared__ f32x4 red[4][3][4][64]; // [tile][other wave][register / 4][lane]
    const int lane = threadIdx.x & 63;
    const int wave = uni(threadIdx.x >> 6);
    const int h = lane >> 5;
    constexpr int PER = G1 ? 2 : 4; // column tiles of a panel
    const int ncg = (a.NT + PER - 1) / PER;
    const int64_t total = (int64_t)ldc(a.mtile_off, a.E) * ncg;
    // an XCD's workgroups (blockIdx % 8) take a contiguous part of the tiles,
    // so an expert's token rows stay in one L2
    const int xcd = blockIdx.x & 7;
    const int64_t t1 = total * (xcd + 1) / 8;
    // the wave's k-step pairs [p0, p1): whole chunks, the last one may be half
    const int p0 = a.KC * wave / 4 * 2, p1 = min(a.KC * (wave + 1) / 4 * 2, a.KS >> 1);

    struct Place {
        int cg, nr, row;
        uint32_t ao, so;                       // this lane's token row: codes, scales
        __amdgpu_buffer_rsrc_t ac, at, as;     // token rows
        __amdgpu_buffer_rsrc_t wc, ws;         // the expert's weights
        int tile[4];                           // column tiles, counted from there
    };
    auto place = [&](int64_t t, Place &q) {
        const int m = (int)(t / ncg);
        q.cg = uni((int)(t - (int64_t)m * ncg));
        const int e = ldc(a.mtile_expert, m);
        const int r0 = ldc(a.offsets, e) + (m - ldc(a.mtile_off, e)) * 32;
        q.nr = min(32, ldc(a.offsets, e + 1) - r0);
        const int r = min(lane & 31, q.nr - 1);
        q.row = r0 + r;
        const TokenRows tr = token_rows<BITS, G1>(a, r0, q.nr);
        q.ac = tr.codes;
        q.at = tr.tails;
        q.as = tr.scales;
        const uint32_t arow = G1 ? a.sorted_slot[q.row] / a.topk : r;
        q.ao = arow * (uint32_t)(a.KS * 32) + h * 16;
        q.so = arow * (uint32_t)a.srow + h * 4;
        const int64_t tiles = (int64_t)a.NT * (G1 ? 2 : 1); // of an expert
        q.wc = bytes_at(a.wcodes + e * tiles * a.KS * 1024, (uint32_t)(tiles * a.KS * 1024));
        q.ws = bytes_at(a.wscales + e * tiles * a.KC * 256, (uint32_t)(tiles * a.KC * 256));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q.tile[j] = min(q.cg * PER + (G1 ? j >> 1 : j), a.NT - 1) + (G1 ? (j & 1) * a.NT : 0);
    };
    const uint32_t wl = lane * 16, sl = lane * 4;
    auto load = [&](const Place &q, int p, StreamPair<BITS> &x) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            x.a[s].c = __builtin_amdgcn_raw_buffer_load_b128(q.ac, q.ao + s * 32, p * 64, 0);
            if constexpr (BITS == 6)
                x.a[s].t = __builtin_amdgcn_raw_buffer_load_b64(q.at, (q.ao >> 1) + s * 16, p * 32, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x.w[j][s] = __builtin_amdgcn_raw_buffer_load_b128(
                    q.wc, wl + s * 1024, code_offset(q.tile[j], a.KS, p * 2), 0);
        }
    };
    auto load_scales = [&](const Place &q, int kc, StreamScales &x) {
        x.a = __builtin_amdgcn_raw_buffer_load_b32(q.as, q.so, kc * 8, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x.w[j] = __builtin_amdgcn_raw_buffer_load_b32(q.ws, sl, (q.tile[j] * a.KC + kc) * 256, 0);
    };
    f32x16 acc[4];
    auto compute = [&](const StreamPair<BITS> &x, const StreamScales &sc, auto ODD) {
        constexpr int s = 2 * decltype(ODD)::value;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = mx_mma<BITS, s>(x.w[j][0], sc.w[j], x.a[0], sc.a, acc[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[j] = mx_mma<BITS, s + 1>(x.w[j][1], sc.w[j], x.a[1], sc.a, acc[j]);
    };

    int64_t t = total * xcd / 8 + (blockIdx.x >> 3);
    if (t >= t1)
        return;
    Place q;
    StreamPair<BITS> x, y;
    StreamScales sc, next;
    auto first = [&] {
        place(t, q);
        if (p0 < p1) {
            load_scales(q, p0 >> 1, next);
            load(q, p0, x);
        }
    };
    first();
    while (true) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                acc[j][i] = 0.f;
        for (int p = p0; p < p1; p += 2) {
            sc = next;
            if (p + 1 < p1)
                load(q, p + 1, y);
            compute(x, sc, IC<0>{});
            if (p + 1 < p1) {
                if (p + 2 < p1) {
                    load_scales(q, (p >> 1) + 1, next);
                    load(q, p + 2, x);
                }
                compute(y, sc, IC<1>{});
            }
        }
        const int cg = q.cg, nr = q.nr, row = q.row;
        t += gridDim.x >> 3;
        if (t < t1)
            first();
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
                if (c == a.NT - 1 && live)
                    store_empty<BITS>(r, c + 1, 2 * a.act_KS);
            }
        } else {
            const int c = cg * 4 + wave;
            bf16 *orow = static_cast<bf16 *>(a.o) + (int64_t)row * a.N;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = c * 32 + 8 * q + 4 * h;
                if (live && col < a.N) {
                    const bf16x4 out = {(bf16)sum[4 * q], (bf16)sum[4 * q + 1],
                                        (bf16)sum[4 * q + 2], (bf16)sum[4 * q + 3]};
                    *reinterpret_cast<bf16x4 *>(orow + col) = out;
                }
            }
        }
        if (t >= t1)
            return;
        __syncthreads();
    }
}

// Tile kernel.  A tile is 32 TF token rows of one expert times eight column
// tiles, two a wave: GEMM1 a gate tile and the up tile of the same columns (so
// the epilogue stays in the wave), GEMM2 two neighbours.  The weights go from
// memory straight into registers, since the waves share none; the token rows,
// which all four waves read, are copied into a ring of LDS stages of two
// k-steps, 64 bytes of codes a row, swizzled like the bf16 kernels' rows.
// GEMM1 of 65536 x 7168 x 4096: 1.03 ms, 3.7 PFLOP/s, where the instruction
// alone, on random codes in registers, reaches 6.3: the matrix cores are busy
// half of the time, at 1.8 GHz, to which the power limit takes the clock (codes
// of zero: 0.89 ms).  GEMM2 writes 0.94 GB of o besides: 0.66 ms.
//
// Workgroups of a CU: three with 64 rows and MXFP4, else two; held to the 168
// registers of three, the MXFP6 kernels spill (128 x 7168 x 2048, 32 experts, top
// 8: 108 + 56 us against 97 + 51).
constexpr int tile_groups(int bits, int rows) { return rows == 64 && bits == 4 ? 3 : 2; }

template <int BITS, bool G1, int TF>
__global__ __launch_bounds__(256, tile_groups(BITS, 32 * TF)) void mx_tile_kernel(MxGemmArgs a)
{
    using namespace tile;
    constexpr int ROWS = TF * 32;
    constexpr int CODES = ROWS * 64, TAILS = BITS == 6 ? ROWS * 32 : 0, SCALES = ROWS * 16;
    constexpr int STAGE = CODES + TAILS, RING = 4;
    constexpr int NC = TF / 2;                       // code copies of a wave and stage
    constexpr int NTL = BITS == 6 ? (TF + 3) / 4 : 0; // tail copies
    constexpr int NL = 4;                            // weight loads of a wave and stage
    __shared__ __attribute__((aligned(1024))) unsigned char smem[RING * STAGE + 2 * SCALES];
    unsigned char *const sscale = smem + RING * STAGE;
    const int wave = uni(threadIdx.x >> 6);
    constexpr int PER = G1 ? 4 : 8; // column tiles of a panel
    const int ncg = (a.NT + PER - 1) / PER;
    const int KP = a.KS >> 1; // stages
    const int total = uni(ldc(a.mtile_off, a.E)) * ncg; // below 2^31 (checked at launch)
    const int xcd = blockIdx.x & 7;
    const int t1 = (int)((int64_t)total * (xcd + 1) / 8), dt = gridDim.x >> 3;
    // expert-major; inside an expert groups of up to GM M-tiles, column groups
    // outer and M-tiles inner, so that tiles in flight share weights and rows.
    // Whole calls, GEMM2 with 4 against 8, three series in turn: 8192 x 7168 x 2048,
    // 32 experts, top 8: 1875-1886 us and 1888-1903 (Zipf 1869-1879, 1880-1887); x 4096 x
    // 1536, 16, top 4: 448 and 456; 16384 x 2048 x 1408, 8, top 8: 811 and 813, 64, top 6:
    // 666 and 669; but 16384 x 4096 x 2048, 8, top 2: 585 and 576
    constexpr int GM = G1 ? 8 : 4;
    struct Place {
        int e, cg, r0, nr; // expert, column group, first row, rows
    };
    auto place = [&](int t) {
        Place q;
        q.e = ldc(a.mtile_expert, uni((int)((unsigned)t / (unsigned)ncg)));
        const int mt0 = ldc(a.mtile_off, q.e), mts = ldc(a.mtile_off, q.e + 1) - mt0;
        const unsigned local = t - mt0 * ncg;
        const int grp = uni(local / (unsigned)(GM * ncg));
        const unsigned gm = min(mts - grp * GM, GM);
        const unsigned rr = local - grp * GM * ncg;
        q.cg = uni(rr / gm);
        const int mt = grp * GM + (int)(rr - q.cg * gm);
        q.r0 = ldc(a.offsets, q.e) + mt * ROWS;
        q.nr = min(ROWS, ldc(a.offsets, q.e + 1) - q.r0);
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

        // a copy moves 1024 bytes: 16 rows of codes, 32 of tails, 64 of scales.
        // Byte offsets of this lane's sources from a scalar base (GEMM1: the
        // whole of x's codes, below 4 GiB; GEMM2: the tile's first row).
        const int64_t first = G1 ? 0 : r0;
        auto row_of = [&](int r) -> uint32_t {
            r = min(r, nr - 1);
            return G1 ? a.sorted_slot[r0 + r] / a.topk : r;
        };
        const uint8_t *const bc = a.acodes + first * (a.KS * 32);
        const uint8_t *const bt = BITS == 6 ? a.atails + first * (a.KS * 16) : nullptr;
        const uint8_t *const bs = a.ascales + first * a.srow;
        uint32_t src_c[NC], src_t[NTL + 1], src_s;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int r = (wave * NC + i) * 16 + (lane >> 2);
            src_c[i] = row_of(r) * (uint32_t)(a.KS * 32) + aswz<4>(r, lane & 3) * 16;
        }
#pragma unroll
        for (int i = 0; i < NTL; ++i) {
            const int r = ((wave * NTL + i) * 32 + (lane >> 1)) & (ROWS - 1);
            src_t[i] = row_of(r) * (uint32_t)(a.KS * 16) + (lane & 1) * 16;
        }
        src_s = row_of((wave * 64 + lane) & (ROWS - 1)) * (uint32_t)a.srow;
        const int64_t tiles = (int64_t)a.NT * (G1 ? 2 : 1); // of an expert
        const auto wc = bytes_at(a.wcodes + e * tiles * a.KS * 1024, (uint32_t)(tiles * a.KS * 1024));
        const auto ws = bytes_at(a.wscales + e * tiles * a.KC * 256, (uint32_t)(tiles * a.KC * 256));
        int tl[2]; // the wave's column tiles
#pragma unroll
        for (int j = 0; j < 2; ++j)
            tl[j] = uni(min(cg * PER + (G1 ? wave : 2 * wave + j), a.NT - 1) + (G1 ? j * a.NT : 0));
        const uint32_t wl = lane * 16, sl = lane * 4;
        // copies of stage p (past the end: of the last one, into a stage that is not read again)
        auto copy = [&](int p) {
            unsigned char *st = smem + (p & (RING - 1)) * STAGE;
            const int q = min(p, KP - 1);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                g2l16s(bc + q * 64, src_c[i], (lds_void *)(st + (wave * NC + i) * 1024));
#pragma unroll
            for (int i = 0; i < NTL; ++i)
                if (TF >= 4 || wave < 2)
                    g2l16s(bt + q * 32, src_t[i],
                           (lds_void *)(st + CODES + (wave * NTL + i) * 1024));
        };
        // scales of the four stages 4g .. 4g + 3, 16 bytes of a row (past its end: the
        // last ones again, into the half that is not read any more)
        auto copy_scales = [&](int g) {
            const int q = min(g, (a.KC - 1) >> 1);
            if (wave < ROWS / 64)
                g2l16s(bs + q * 16, src_s, (lds_void *)(sscale + (g & 1) * SCALES + wave * 1024));
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
                        wc, wl + s * 1024, code_offset(tl[j], a.KS, q), 0);
        };
        struct S {
            int w[2];
        };
        auto load_s = [&](int kc, S &s) {
            const int q = min(kc, a.KC - 1);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                s.w[j] = __builtin_amdgcn_raw_buffer_load_b32(ws, sl, (tl[j] * a.KC + q) * 256, 0);
        };
        f32x16 acc[2][TF];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[j][f][i] = 0.f;
        // the two k-steps of stage p; ODD: the second half of the scale dwords
        auto compute = [&](int p, const W &w, const S &sw, auto ODD) {
            const unsigned char *st = smem + (p & (RING - 1)) * STAGE;
            const unsigned char *sc = sscale + ((p >> 2) & 1) * SCALES + ((p >> 1) & 1) * 8 + h * 4;
            int as[TF];
#pragma unroll
            for (int f = 0; f < TF; ++f)
                as[f] = *reinterpret_cast<const int *>(sc + (f * 32 + fr) * 16);
            auto step = [&](auto H) {
                constexpr int s = decltype(H)::value;
                constexpr int sel = 2 * decltype(ODD)::value + s;
#pragma unroll
                for (int f = 0; f < TF; ++f) {
                    const int r = f * 32 + fr;
                    MxFrag<BITS> av;
                    av.c = *reinterpret_cast<const u32x4 *>(st + r * 64 + aswz<4>(r, 2 * s + h) * 16);
                    if constexpr (BITS == 6)
                        av.t = *reinterpret_cast<const u32x2 *>(st + CODES + r * 32 + s * 16 + h * 8);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[j][f] = mx_mma<BITS, sel>(w.c[j][s], sw.w[j], av, as[f], acc[j][f]);
                }
            };
            step(IC<0>{});
            step(IC<1>{});
        };
        W w0, w1;
        S s0, s1;
        copy_scales(0);
        copy(0);
        load_w(0, w0);
        load_s(0, s0);
        copy(1);
        load_w(1, w1);
        next = place(min(t + dt, t1 - 1)); // under the first loads
        wait_vm<NC + NTL + NL>();
        lds_barrier();
        // Stage p: its copies and weights were issued two stages ago.  The
        // copies of p + 2 precede the weights' loads of p + 2, so waiting for
        // all but the youngest operations covers the copies of p + 1.
        constexpr int YOUNG = 2 * NL + NC + (TF >= 4 ? NTL : 0);
        int p = 0;
        for (; p + 2 <= KP; p += 2) {
            if ((p & 3) == 0)
                copy_scales((p >> 2) + 1);
            copy(p + 2);
            compute(p, w0, s0, IC<0>{});
            load_w(p + 2, w0);
            load_s((p >> 1) + 1, s1);
            wait_vm<YOUNG>();
            lds_barrier();
            copy(p + 3);
            compute(p + 1, w1, s0, IC<1>{});
            load_w(p + 3, w1);
            s0 = s1;
            wait_vm<YOUNG>();
            lds_barrier();
        }
        if (p < KP)
            compute(p, w0, s0, IC<0>{});
        wait_vm<0>();
        lds_barrier();
        // the last barrier: every wave is past its reads, so the next tile may copy
        if constexpr (G1) {
            const int c = cg * 4 + wave;
#pragma unroll
            for (int f = 0; f < TF; ++f) {
                const int r = f * 32 + fr;
                const bool live = r < nr && c < a.NT;
                const ActRow ar = act_row<BITS>(a, r0 + min(r, nr - 1));
                store_act<BITS>(acc[0][f], acc[1][f], ar, c, live);
                if (c == a.NT - 1 && live)
                    store_empty<BITS>(ar, c + 1, 2 * a.act_KS);
            }
        } else {
            // The 64 columns of a wave are turned in LDS, 32 rows at a time, so
            // that a store instruction writes eight rows of 128 bytes; straight
            // from the registers it would touch 32 rows in pieces of 16 bytes
            // (65536 x 2048 x 7168, MXFP4: 810 us, this way 697, and 650 with the
            // stores that pass the cache).  Of four row fragments the turn lies
            // in the ring's last two stages, which the next tile's copies reach
            // after a barrier; of two it takes the whole ring.
            unsigned char *const turn = smem + (TF == 4 ? 2 * STAGE : 0) + wave * 4096;
            const int part = lane & 7, col = (cg * 8 + 2 * wave) * 32 + part * 8;
#pragma unroll
            for (int f = 0; f < TF; ++f) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        bf16x4 o;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = (bf16)acc[j][f][4 * q + i];
                        *reinterpret_cast<bf16x4 *>(turn + fr * 128 +
                                                    aswz<8>(fr, j * 4 + q) * 16 + h * 8) = o;
                    }
                asm volatile("" ::: "memory"); // a wave's LDS operations complete in order
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rl = i * 8 + (lane >> 3), r = f * 32 + rl;
                    const u32x4 v =
                        *reinterpret_cast<const u32x4 *>(turn + rl * 128 + aswz<8>(rl, part) * 16);
                    if (r < nr && col < a.N) { // N is a multiple of 8
                        u32x4 *dst = reinterpret_cast<u32x4 *>(static_cast<bf16 *>(a.o) +
                                                               (int64_t)(r0 + r) * a.N + col);
                        if (a.stream_o)
                            __builtin_nontemporal_store(v, dst);
                        else
                            *dst = v;
                    }
                }
                asm volatile("" ::: "memory");
            }
            __builtin_amdgcn_s_waitcnt(0xC07F); // LDS only: writes of rows past nr had no reader
            if (TF == 2)
                lds_barrier();
        }
    }
}

template <int BITS, bool G1> static auto tile_kernel(int BM)
{
    return BM == 64 ? mx_tile_kernel<BITS, G1, 2> : mx_tile_kernel<BITS, G1, 4>;
}

hipError_t launch_mx_gemm(bool g1, int bits, const MxGemmArgs &a, int num_cus, hipStream_t s)
{
    const bool stream = a.BM == 32;
    const int per = stream ? (g1 ? 2 : 4) : (g1 ? 4 : 8);
    const int64_t most = (int64_t)a.max_mtiles * ((a.NT + per - 1) / per);
    if (most >= ((int64_t)1 << 31))
        return hipErrorInvalidValue;
    int64_t grid = (int64_t)num_cus * tile_groups(bits, a.BM);
    if (most < grid)
        grid = most;
    grid = (grid + 7) / 8 * 8; // a whole number of workgroups for each XCD
    auto k = stream ? (g1 ? (bits == 4 ? mx_stream_kernel<4, true> : mx_stream_kernel<6, true>)
                          : (bits == 4 ? mx_stream_kernel<4, false> : mx_stream_kernel<6, false>))
             : g1   ? (bits == 4 ? tile_kernel<4, true>(a.BM) : tile_kernel<6, true>(a.BM))
                    : (bits == 4 ? tile_kernel<4, false>(a.BM) : tile_kernel<6, false>(a.BM));
    hipLaunchKernelGGL(k, dim3((unsigned)grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe
