// group.hip — set-up of the grouped products: from a caller's offsets to what
// the GEMM kernels walk.
//
// One block forms, of offsets that may hold anything, o'[e] = max over e' <= e of
// offsets[e'] held to [0, M]: ascending and inside the rows, so that no later
// kernel indexes outside them, and equal to valid offsets.  From these it builds the
// M-tile tables (prefix of ceil(rows / BM), owner of every tile) and the groups'
// order by their rows, for the weight gradient.  The other blocks zero the output
// rows that belong to no group, which no GEMM tile covers.  A launch of 4 us: the
// scans' barriers and one dependent load each way.
#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kSetupThreads = 1024;

__device__ inline int32_t held_offset(const GroupSetup &g, int e)
{
    const int64_t v = g.off64 ? static_cast<const int64_t *>(g.offsets)[e]
                              : (int64_t)static_cast<const int32_t *>(g.offsets)[e];
    return (int32_t)(v < 0 ? 0 : v > g.M ? g.M : v);
}

// Inclusive scan over the block by `op` (identity 0: the values are not negative).
template <typename Op> __device__ inline int32_t block_scan(int32_t v, int32_t *s_w, Op op)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(v, d, 64);
        if (lane >= d)
            v = op(v, o);
    }
    if (lane == 63)
        s_w[wave] = v;
    __syncthreads();
    int32_t before = 0;
    for (int w = 0; w < wave; ++w)
        before = op(before, s_w[w]);
    __syncthreads(); // s_w may be used again
    return op(v, before);
}

__global__ __launch_bounds__(kSetupThreads) void group_setup_kernel(GroupSetup g)
{
    __shared__ int32_t s_off[1025], s_moff[1025], s_w[16];
    const int t = threadIdx.x, E = g.E;
    const int32_t raw = t <= E ? held_offset(g, t) : 0;
    const int32_t o = block_scan(raw, s_w, [](int32_t a, int32_t b) { return max(a, b); });
    if (t <= E)
        s_off[t] = o;
    if (t == kSetupThreads - 1 && E == kSetupThreads)
        s_off[E] = max(o, held_offset(g, E));
    __syncthreads();
    if (blockIdx.x > 0) {
        // rows [0, o'[0]) and [o'[E], M), 16 bytes a thread
        const int64_t head = (int64_t)s_off[0] * g.out_row / 16;
        const int64_t tail = (int64_t)s_off[E] * g.out_row / 16;
        const int64_t end = g.M * g.out_row / 16;
        u32x4 *out = static_cast<u32x4 *>(g.out);
        const int64_t step = (int64_t)(gridDim.x - 1) * kSetupThreads;
        for (int64_t i = (int64_t)(blockIdx.x - 1) * kSetupThreads + t; i < head + end - tail; i += step)
            out[i < head ? i : i - head + tail] = u32x4{0u, 0u, 0u, 0u};
        return;
    }
    if (t <= E)
        g.out_offsets[t] = s_off[t];
    if (t == 0)
        g.out_offsets[E] = s_off[E];
    if (t < 16)
        g.tickets[t] = 0;
    auto sum = [](int32_t a, int32_t b) { return a + b; };
    auto tiles_of = [&](int BM) { return t < E ? (s_off[t + 1] - s_off[t] + BM - 1) / BM : 0; };
    // M-tiles of BM rows into a table, or, if not `used`, none
    auto table = [&](int BM, int32_t *off, int32_t *owner, bool used) {
        const int32_t upto = block_scan(used ? tiles_of(BM) : 0, s_w, sum);
        if (t < E) {
            s_moff[t + 1] = upto;
            off[t + 1] = upto;
        }
        if (t == 0) {
            s_moff[0] = 0;
            off[0] = 0;
        }
        __syncthreads();
        for (int m = t; m < s_moff[E]; m += kSetupThreads) {
            int lo = 0, hi = E; // the group e with moff[e] <= m < moff[e + 1]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_moff[mid] <= m)
                    lo = mid;
                else
                    hi = mid;
            }
            owner[m] = lo;
        }
    };
    if (!g.alt.mtile_off) {
        table(g.BM, g.mtile_off, g.mtile_expert, true);
    } else {
        __shared__ int32_t s_tiles[2];
        const int32_t a = block_scan(tiles_of(256), s_w, sum), b = block_scan(tiles_of(128), s_w, sum);
        if (t == kSetupThreads - 1) {
            s_tiles[0] = a;
            s_tiles[1] = b;
        }
        __syncthreads();
        const float rows = (float)(s_off[E] - s_off[0]);
        const bool tall = tall_tiles(g.alt.model, rows, (float)s_tiles[0], (float)s_tiles[1]);
        table(256, g.mtile_off, g.mtile_expert, tall);
        __syncthreads(); // s_moff is read
        table(128, g.alt.mtile_off, g.alt.mtile_expert, !tall);
    }
    if (g.order && t < E) { // descending by rows, equals by number
        const int32_t rows = s_off[t + 1] - s_off[t];
        int rank = 0;
        for (int e = 0; e < E; ++e) {
            const int32_t other = s_off[e + 1] - s_off[e];
            rank += other > rows || (other == rows && e < t);
        }
        g.order[rank] = t;
    }
}

hipError_t launch_group_setup(const GroupSetup &g, hipStream_t s)
{
    int64_t zero_blocks = 0;
    if (g.out) { // where there are such rows at all, they are mostly few
        zero_blocks = (g.M * g.out_row + (256 << 10) - 1) / (256 << 10);
        zero_blocks = zero_blocks < 1 ? 1 : zero_blocks > 512 ? 512 : zero_blocks;
    }
    hipLaunchKernelGGL(group_setup_kernel, dim3((unsigned)(1 + zero_blocks)), dim3(kSetupThreads), 0,
                       s, g);
    return hipGetLastError();
}

} // namespace moe
