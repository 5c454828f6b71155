// group_view.h — row groups straight from a caller's offsets, for up to 64 groups: lane
// e of every wave holds group e, so that kernels that are shorter than a set-up launch
// (group.hip, 4 us with its gap) need none.  The same rule as there: each offset held to
// [0, M], then their running maximum.  Internal.
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kViewGroups = 64;

struct GroupView {
    int start, end;  // this lane's group's rows
    int mt0, tiles;  // its first M-tile and their number
    int total;       // M-tiles of all groups (uniform)
    int first, last; // the rows that belong to groups (uniform)
};

__device__ inline GroupView group_view(const GroupSource &g, int BM)
{
    const int lane = threadIdx.x & 63;
    auto held = [&](int e) -> int {
        const int64_t v = g.off64 ? static_cast<const int64_t *>(g.offsets)[e]
                                  : (int64_t)static_cast<const int32_t *>(g.offsets)[e];
        return (int)(v < 0 ? 0 : v > g.M ? g.M : v);
    };
    GroupView v;
    v.start = lane <= g.E ? held(lane) : 0;
    v.end = lane == 63 && g.E == 64 ? held(64) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v.start, d, 64);
        if (lane >= d)
            v.start = max(v.start, o);
    }
    // the next lane's start, and for lane 63 the 65th offset
    const int after = __shfl_down(v.start, 1, 64);
    v.end = lane == 63 ? max(v.start, v.end) : after;
    v.tiles = lane < g.E ? (v.end - v.start + BM - 1) / BM : 0;
    int upto = v.tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(upto, d, 64);
        if (lane >= d)
            upto += o;
    }
    v.mt0 = upto - v.tiles;
    v.total = __builtin_amdgcn_readlane(upto, 63);
    v.first = __builtin_amdgcn_readlane(v.start, 0);
    v.last = __builtin_amdgcn_readlane(v.end, g.E - 1);
    return v;
}

// The group of M-tile m (0 <= m < total).
__device__ inline int view_group(const GroupView &v, int E, int m)
{
    const int lane = threadIdx.x & 63;
    return 63 - __builtin_clzll(__ballot(lane < E && v.mt0 <= m));
}

// Zeros in the output rows [0, v.first) and [v.last, M) of `row` bytes each (a multiple of
// 16), by all threads of the grid.
__device__ inline void zero_ungrouped(const GroupView &v, int64_t M, void *out, int64_t row)
{
    const int64_t head = v.first * row / 16, tail = v.last * row / 16, end = M * row / 16;
    u32x4 *o = static_cast<u32x4 *>(out);
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < head + end - tail; i += step)
        o[i < head ? i : i - head + tail] = u32x4{0u, 0u, 0u, 0u};
}

} // namespace moe
