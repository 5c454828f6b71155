// xcd_split.h — how the weight-gradient tiles of uneven row groups are shared out
// over the eight XCDs.  Internal.
#pragma once

#include "kernels.h"

namespace moe {

// Cost-balanced XCD bounds of the weight-gradient launches.  A tile of
// expert e contracts over its count[e] rows; its cost is modelled as
// count[e] + TILE_EPS rows (TILE_EPS for the epilogue and tile switch), so
// with F tiles per expert the cost before tile e F + j is
// F (off[e] + e TILE_EPS) + j (count[e] + TILE_EPS).  XCD x starts at the
// first tile whose cost prefix reaches x/8 of the total; that start is then
// moved to a whole number of rounds of the XCD's workgroups (a multiple of
// wgx tiles from the previous bound, when there are two rounds or more), so
// that tiles of equal cost split evenly over the workgroups.
//
// s_off: the E + 1 offsets in LDS; s_raw: scratch in LDS.  For a whole block of
// at least 16 threads.
__device__ inline void xcd_split(const int32_t *s_off, int E, const XcdSplits &splits,
                                 int32_t (&s_raw)[2][8])
{
    constexpr int TILE_EPS = 64;
    if (splits.n > 0) {
        const int k = threadIdx.x >> 3, x = threadIdx.x & 7;
        if (k < splits.n && x > 0) {
            const int64_t F = k == 0 ? splits.F[0] : splits.F[1];
            auto prefix = [&](int ex) { return F * ((int64_t)s_off[ex] + (int64_t)ex * TILE_EPS); };
            const int64_t target = prefix(E) * x / 8;
            int lo = 0, hi = E; // largest ex in [0, E] with prefix(ex) <= target
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix(mid) <= target)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            int64_t L = (int64_t)E * F;
            if (lo < E) {
                const int64_t w = (int64_t)(s_off[lo + 1] - s_off[lo]) + TILE_EPS;
                const int64_t j = (target - prefix(lo) + w - 1) / w;
                L = lo * F + (j < F ? j : F);
            }
            s_raw[k][x] = (int32_t)L;
        }
        __syncthreads();
        if (threadIdx.x < splits.n) {
            const int kk = threadIdx.x;
            const int F = kk == 0 ? splits.F[0] : splits.F[1];
            const int wgx = kk == 0 ? splits.wgx[0] : splits.wgx[1];
            const int32_t total = E * F;
            int32_t b = 0;
            splits.bounds[9 * kk] = 0;
            for (int xx = 1; xx < 8; ++xx) {
                int32_t n = max(s_raw[kk][xx], b) - b;
                if (n >= 2 * wgx)
                    n = (n + wgx / 2) / wgx * wgx;
                b = min(b + n, total);
                splits.bounds[9 * kk + xx] = b;
            }
            splits.bounds[9 * kk + 8] = total;
        }
    }
}

} // namespace moe
