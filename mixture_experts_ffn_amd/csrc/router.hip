// router.hip — router logits to expert ids and gates, and the gradient.
//
// For a token's logits l [E], with score s_j = softmax(l)_j or sigmoid(l_j):
//   key_j = s_j + bias_j (no bias: l_j, which orders the experts like s_j does)
//   groups: only the experts of the topk_groups best groups stay open, a
//           group's value being its largest key or the sum of its two largest
//   ids    = the K open experts of largest key, ties to the lower id
//   w_k    = scale * s_k, or scale * s_k / sum of the selected s
// An expert whose logit (or bias) is -inf is closed; slots left without an
// open expert get id -1 and gate 0.  A NaN key is below every number.
//
// Gradients (u_k = s_k / sum of the selected s, g_k = scale * d w_k):
//   softmax, renormalised  dl_k = u_k (g_k - sum_i g_i u_i)
//   softmax                dl_j = s_j ([j selected] g_j - sum_i g_i s_i)
//   sigmoid, renormalised  dl_k = u_k (1 - s_k) (g_k - sum_i g_i u_i)
//   sigmoid                dl_k = g_k s_k (1 - s_k)
// and zero elsewhere; the selection has no gradient.
#include <float.h>

#include "kernels.h"
#include "common.h"

namespace moe {

// ---- reductions over a wave's 64 lanes, the result in every lane -----------------
// Exchanges with lane ^ 1, ^ 2 (quad permutes), then mirrors of 8 and 16 lanes
// (whose halves already hold one value each), then swaps of rows and halves.
template <int CTRL> __device__ inline uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// reduces over groups of N consecutive lanes (N a power of two)
template <int N, typename F> __device__ inline uint32_t lanes_reduce(uint32_t v, F f)
{
    if constexpr (N >= 2)
        v = f(v, dpp<0xB1>(v)); // quad_perm 1, 0, 3, 2
    if constexpr (N >= 4)
        v = f(v, dpp<0x4E>(v)); // quad_perm 2, 3, 0, 1
    if constexpr (N >= 8)
        v = f(v, dpp<0x141>(v)); // row_half_mirror
    if constexpr (N >= 16)
        v = f(v, dpp<0x140>(v)); // row_mirror
    if constexpr (N >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    if constexpr (N >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f(r[0], r[1]);
    }
    return v;
}
__device__ inline uint32_t wave_max_u(uint32_t v)
{
    return lanes_reduce<64>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ inline float wave_max(float v)
{
    return __uint_as_float(lanes_reduce<64>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ inline float wave_min(float v) { return -wave_max(-v); }
__device__ inline float wave_sum(float v)
{
    return __uint_as_float(lanes_reduce<64>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
__device__ inline double wave_max_d(double v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v = fmax(v, __shfl_xor(v, m));
    return v;
}
__device__ inline double wave_sum_d(double v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}
__device__ inline float lane_value(float v, int lane)
{
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// sum of n <= 16 values in a tree, so that an element passes log2 n roundings
template <int N> __device__ inline float tree_sum(const float *v)
{
    if constexpr (N == 1)
        return v[0];
    else
        return tree_sum<N / 2>(v) + tree_sum<N / 2>(v + N / 2);
}

__device__ inline float load_logit(const RouterArgs &a, int64_t t, int j)
{
    const int64_t at = t * a.stride + j;
    return a.bf16 ? (float)static_cast<const bf16 *>(a.logits)[at]
                  : static_cast<const float *>(a.logits)[at];
}

// This lane's R consecutive logits of token t, experts lane R + [0, R); -inf
// past the last.  `vec`: rows start at multiples of 16 bytes.
template <int R>
__device__ inline void load_row(const RouterArgs &a, int64_t t, int lane, float *l)
{
    const int j0 = lane * R;
    const int64_t at = t * a.stride + j0;
    if (a.vec && j0 + R <= a.E) {
        if (a.bf16) {
            typedef bf16 V __attribute__((ext_vector_type(R)));
            const V v = *reinterpret_cast<const V *>(static_cast<const bf16 *>(a.logits) + at);
#pragma unroll
            for (int i = 0; i < R; ++i)
                l[i] = (float)v[i];
        } else {
            typedef float V __attribute__((ext_vector_type(R)));
            const V v = *reinterpret_cast<const V *>(static_cast<const float *>(a.logits) + at);
#pragma unroll
            for (int i = 0; i < R; ++i)
                l[i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            l[i] = j0 + i < a.E ? load_logit(a, t, j0 + i) : -INFINITY;
    }
}

// Order-preserving integer of a key: closed 0, NaN 1, numbers above; -0 = +0.
__device__ inline uint32_t order_of(float key, bool closed)
{
    const uint32_t b = __float_as_uint(key + 0.0f);
    const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return closed ? 0u : isnan(key) ? 1u : u;
}
__device__ inline float key_of(uint32_t u)
{
    return u == 1u ? NAN : __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// What the selection leaves in lane k < K: slot k's expert (or -1) and logit.
struct Slot {
    int id;
    float l;
};

// Selection in 64 bits: one wave, expert j on lane j % 64.  For the rows whose
// keys or group values lie too close together for the fp32 selection.
template <int EPL>
__device__ inline Slot select_exact(const RouterArgs &a, int64_t t, int lane, double *keys)
{
    const int E = a.E;
    float l[EPL];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 64 * i;
        l[i] = j < E ? load_logit(a, t, j) : -INFINITY;
        top = fmaxf(top, l[i]);
    }
    top = wave_max(top);
    const bool grouped = a.topk_groups < a.groups;
    const bool need_score = a.bias || (grouped && a.group_top == 2);
    double total = 0.0; // softmax denominator
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (l[i] > -INFINITY)
                total += exp((double)l[i] - (double)top);
        total = wave_sum_d(total);
    }
    double key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 64 * i;
        double k = l[i];
        if (need_score && j < E && l[i] > -INFINITY) {
            k = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)top) / total;
            if (a.bias)
                k += (double)a.bias[j];
        }
        if (isnan(k))
            k = -DBL_MAX;
        key[i] = l[i] == -INFINITY ? -INFINITY : k;
    }
    if (grouped) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 64 * i < E)
                keys[lane + 64 * i] = key[i];
        __builtin_amdgcn_wave_barrier();
        const int n = E / a.groups;
        double value = -INFINITY;
        if (lane < a.groups) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int i = 0; i < n; ++i) {
                const double k = keys[lane * n + i];
                b1 = fmax(b1, fmin(b0, k));
                b0 = fmax(b0, k);
            }
            value = a.group_top == 2 ? b0 + b1 : b0;
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double v = __shfl(value, g);
            rank += v > value || (v == value && g < lane);
        }
        const uint64_t kept = __ballot(lane < a.groups && rank < a.topk_groups);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int j = lane + 64 * i;
            if (j < E && !(kept >> (j / n) & 1))
                key[i] = -INFINITY;
        }
        // without a bias the experts of the kept groups are ordered by logit
        if (!a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] > -INFINITY)
                    key[i] = isnan(l[i]) ? -DBL_MAX : (double)l[i];
        }
    }
    // K times the largest key; lane k keeps slot k
    Slot mine = {-1, -INFINITY};
    for (int k = 0; k < a.K; ++k) {
        double b = -INFINITY;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > b) {
                b = key[i];
                at = i;
            }
        const double best = wave_max_d(b);
        if (!(best > -INFINITY))
            break;
        // lowest id among the holders
        int id = b == best ? lane + 64 * at : 1 << 30;
#pragma unroll
        for (int m = 32; m; m >>= 1)
            id = min(id, __shfl_xor(id, m));
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 64 * i == id) {
                key[i] = -INFINITY;
                v = l[i];
            }
        v = __shfl(v, id & 63);
        if (lane == k)
            mine = {id, v};
    }
    return mine;
}

// Selection in 32 bits, one wave a row, R experts a lane.  Logits order the
// experts exactly.  Keys that are a sum (score and bias, two scores of a
// group) are rounded, and where two that were compared lie closer than the
// rounding may move them the row is left to select_exact (returns false; with
// scores spread over (0, 1) about one row in a thousand).  The bound, with
// u = 2^-24 and every compared value at most `size`:
//   sigmoid: exponential 2u, sum u, reciprocal 2u of a value <= 1: 5u
//   softmax: exponent |x| u (times p <= e^-|x|: 0.4u), exponential 2u, the
//            denominator 10u (tree of 16 a lane and six levels) + 2u + u times
//            the mean |x| <= ln E < 7, reciprocal 2u, product u: below 25u
//   key:     u size on top
// and twice that between two keys; `margin` (1 + size) covers 10u = 2^-20.7
// and 50u = 2^-18.4 with more than a factor of two to spare.  Sums of two keys
// have twice the error.
template <int R>
__device__ inline bool select_fast(const RouterArgs &a, const float *l, float top, float total,
                                   int lane, float *keys, Slot *out)
{
    const int E = a.E, K = a.K;
    const bool grouped = a.topk_groups < a.groups;
    const bool sums = a.bias != nullptr;
    const bool pair = grouped && a.group_top == 2;
    bool ok = true;
    float score[R];
    if (sums || pair) {
        const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
        for (int i = 0; i < R; ++i)
            score[i] = a.sigmoid ? __builtin_amdgcn_rcpf(1.f + expf(-l[i])) : expf(l[i] - top) * inv;
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            score[i] = l[i];
    }
    uint32_t key[R];
    if (sums) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int j = lane * R + i;
            const float b = j < E ? a.bias[j] : -INFINITY;
            score[i] += b;
            key[i] = order_of(score[i], l[i] == -INFINITY || b == -INFINITY);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            key[i] = order_of(l[i], l[i] == -INFINITY);
    }
    float margin = 0.f;
    if (sums || grouped) {
        float size = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (key[i] != 0u) {
                size = fmaxf(size, fabsf(score[i]));
                nan |= isnan(score[i]);
            }
        margin = (a.sigmoid ? 0x1p-19f : 0x1p-17f) * (1.f + wave_max(size));
        ok = __ballot(nan) == 0;
    }
    if (grouped) {
        // a group's value: a power of two of lanes scan its experts in LDS
        const int n = E / a.groups;
        const int lg = a.group_lanes, g = lane / lg;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (lane * R + i < E)
                keys[lane * R + i] = key[i] == 0u  ? -INFINITY
                                     : isnan(score[i]) ? -FLT_MAX
                                                       : score[i];
        __builtin_amdgcn_wave_barrier();
        float b0 = -INFINITY, b1 = -INFINITY;
        if (g < a.groups)
            for (int i = lane & (lg - 1); i < n; i += lg) {
                const float k = keys[g * n + i];
                b1 = fmaxf(b1, fminf(b0, k));
                b0 = fmaxf(b0, k);
            }
        auto join = [&](float o0, float o1) {
            b1 = fmaxf(fmaxf(b1, o1), fminf(b0, o0));
            b0 = fmaxf(b0, o0);
        };
        auto from = [](uint32_t v) { return __uint_as_float(v); };
        const auto bits = [](float v) { return __float_as_uint(v); };
        if (lg >= 2)
            join(from(dpp<0xB1>(bits(b0))), from(dpp<0xB1>(bits(b1))));
        if (lg >= 4)
            join(from(dpp<0x4E>(bits(b0))), from(dpp<0x4E>(bits(b1))));
        if (lg >= 8)
            join(from(dpp<0x141>(bits(b0))), from(dpp<0x141>(bits(b1))));
        if (lg >= 16)
            join(from(dpp<0x140>(bits(b0))), from(dpp<0x140>(bits(b1))));
        if (lg >= 32)
            join(__shfl_xor(b0, 16), __shfl_xor(b1, 16));
        const float value = g >= a.groups ? -INFINITY : pair ? b0 + b1 : b0;
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float v = lane_value(value, o * lg);
            rank += v > value || (v == value && o < g);
        }
        const bool keep = g < a.groups && rank < a.topk_groups;
        const uint64_t kept = __ballot(keep);
        if (sums || pair) {
            const float lo = wave_min(keep ? value : INFINITY);
            const float hi = wave_max(keep ? -INFINITY : value);
            ok = ok && (!(lo - hi <= 2.f * margin) || hi == -INFINITY);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t j = lane * R + i;
            const int og = a.group_m ? (int)__umulhi(j, a.group_m) : (int)j; // expert / n
            if (j >= (uint32_t)E || !(kept >> (og * lg) & 1))
                key[i] = 0u;
        }
    }
    Slot mine = {-1, -INFINITY};
    float last = INFINITY;
    const int rounds = sums ? K + 1 : K; // with sums, also the first one left out
    for (int k = 0; k < rounds; ++k) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            m = max(m, key[i]);
        const uint32_t best = __builtin_amdgcn_readfirstlane(wave_max_u(m));
        if (best == 0u)
            break;
        if (sums) {
            const float v = key_of(best);
            ok = ok && !(last - v <= margin);
            last = v;
            if (k == K)
                break;
        }
        // the lowest lane that holds it, and there the lowest expert
        const int from = __builtin_ctzll(__ballot(m == best));
        int at = 0;
        float v = l[0];
#pragma unroll
        for (int i = R - 1; i >= 0; --i)
            if (key[i] == best) {
                at = i;
                v = l[i];
            }
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (lane == from && at == i)
                key[i] = 0u;
        const int id = from * R + (R == 1 ? 0 : __builtin_amdgcn_readlane(at, from));
        const float vl = lane_value(v, from);
        if (lane == k)
            mine = {id, vl};
    }
    *out = mine;
    return ok;
}

// One wave per token.
template <int R>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ double s_key[]; // [4 waves][E], with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int K = a.K;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T)
        return;
    double *keys = s_key + (int64_t)wave * a.E;
    float l[R];
    load_row<R>(a, t, lane, l);
    float top = 0.f, total = 1.f;
    bool bad = false; // softmax of a row with NaN or +inf
    if (!a.sigmoid) {
        top = l[0];
        bool odd = !(l[0] < INFINITY);
#pragma unroll
        for (int i = 1; i < R; ++i) {
            top = fmaxf(top, l[i]);
            odd |= !(l[i] < INFINITY);
        }
        top = wave_max(top);
        bad = __ballot(odd) != 0;
        if (a.need_total) {
            float e[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                e[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - top);
            total = wave_sum(tree_sum<R>(e));
        }
    }
    Slot mine;
    if (!select_fast<R>(a, l, top, total, lane, reinterpret_cast<float *>(keys), &mine)) {
        __builtin_amdgcn_wave_barrier();
        mine = select_exact<R>(a, t, lane, keys);
    }
    const bool live = mine.id >= 0;
    float w;
    if (a.sigmoid) {
        if (a.renorm) {
            // s = e^min(l,0) / (1 + e^-|l|); e^-M cancels, so that a row of
            // very negative logits keeps its ratios
            const float neg = live ? fminf(mine.l, 0.f) : -INFINITY;
            const float M = wave_max(neg);
            const float s = live ? expf(neg - M) / (1.f + expf(-fabsf(mine.l))) : 0.f;
            w = s / wave_sum(s);
        } else {
            w = 1.f / (1.f + expf(-mine.l));
        }
    } else if (a.renorm) {
        const float M = wave_max(mine.l);
        const float s = live ? expf(mine.l - M) : 0.f;
        w = s / wave_sum(s);
    } else {
        w = expf(mine.l - top) / total;
    }
    if (bad)
        w = NAN;
    if (lane < K) {
        a.weights[t * K + lane] = live ? a.scale * w : 0.f;
        if (a.ids64)
            static_cast<int64_t *>(a.ids)[t * K + lane] = mine.id;
        else
            static_cast<int32_t *>(a.ids)[t * K + lane] = mine.id;
    }
}

// One wave per token.  Lane k < K owns slot k; then every lane writes its R
// experts' gradients, zeros included.
template <int R>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = a.E, K = a.K;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T)
        return;
    int id = -1;
    float g = 0.f;
    if (lane < K) {
        const int64_t v = a.ids64 ? static_cast<const int64_t *>(a.ids)[t * K + lane]
                                  : static_cast<const int32_t *>(a.ids)[t * K + lane];
        if (v >= 0 && v < E) {
            id = (int)v;
            g = a.scale * a.d_weights[t * K + lane];
        }
    }
    const bool dense = !a.sigmoid && !a.renorm;
    float l[R];
    float top = -INFINITY, total = 1.f;
    if (dense) {
        load_row<R>(a, t, lane, l);
#pragma unroll
        for (int i = 0; i < R; ++i)
            top = fmaxf(top, l[i]);
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < R; ++i)
            l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - top);
        total = wave_sum(tree_sum<R>(l));
    }
    const float lk = id >= 0 ? load_logit(a, t, id) : -INFINITY;
    if (lk == -INFINITY) {
        id = -1;
        g = 0.f;
    }
    // d: this slot's own part of the gradient; dot: what every score loses
    float d = 0.f, dot = 0.f;
    if (dense) {
        const float p = id >= 0 ? expf(lk - top) / total : 0.f;
        dot = wave_sum(g * p);
        d = g;
    } else if (a.renorm) {
        const float neg = id < 0 ? -INFINITY : a.sigmoid ? fminf(lk, 0.f) : lk;
        const float M = wave_max(neg);
        float s = id >= 0 ? expf(neg - M) : 0.f;
        if (a.sigmoid && id >= 0)
            s /= 1.f + expf(-fabsf(lk));
        const float sum = wave_sum(s);
        const float u = id >= 0 ? s / sum : 0.f;
        d = u * (g - wave_sum(g * u));
        if (a.sigmoid && id >= 0)
            d *= 1.f / (1.f + expf(lk));
    } else if (id >= 0) {
        const float e = expf(-fabsf(lk));
        d = g * e / ((1.f + e) * (1.f + e));
    }
    float own[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        own[i] = 0.f;
    for (int k = 0; k < K; ++k) {
        const int j = __builtin_amdgcn_readlane(id, k);
        const float v = lane_value(d, k);
#pragma unroll
        for (int i = 0; i < R; ++i)
            own[i] += lane * R + i == j ? v : 0.f;
    }
    if (dense) {
        const float inv = 1.f / total;
#pragma unroll
        for (int i = 0; i < R; ++i)
            own[i] = l[i] == 0.f ? 0.f : l[i] * inv * (own[i] - dot);
    }
    const int64_t at = t * E + lane * R;
    if (a.vec_out && lane * R + R <= E) {
        if (a.bf16) {
            typedef bf16 V __attribute__((ext_vector_type(R)));
            V v;
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = (bf16)own[i];
            *reinterpret_cast<V *>(static_cast<bf16 *>(a.d_logits) + at) = v;
        } else {
            typedef float V __attribute__((ext_vector_type(R)));
            V v;
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = own[i];
            *reinterpret_cast<V *>(static_cast<float *>(a.d_logits) + at) = v;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (lane * R + i >= E)
            continue;
        if (a.bf16)
            static_cast<bf16 *>(a.d_logits)[at + i] = (bf16)own[i];
        else
            static_cast<float *>(a.d_logits)[at + i] = own[i];
    }
}

// The kernels' own fields.  Vectors of R elements (up to 64 bytes) are taken
// where every row starts at a multiple of 16 bytes, of the vector's size if
// that is less.
static RouterArgs prepared(const RouterArgs &in)
{
    RouterArgs a = in;
    const int64_t es = a.bf16 ? 2 : 4;
    auto aligned = [&](const void *p, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * es)) % 16 == 0;
    };
    a.vec = aligned(a.logits, a.stride);
    a.vec_out = a.d_logits && aligned(a.d_logits, a.E);
    a.need_total = !a.sigmoid && (!a.renorm || a.bias || (a.topk_groups < a.groups && a.group_top == 2));
    int lanes = 64;
    while (lanes * a.groups > 64)
        lanes /= 2;
    a.group_lanes = lanes;
    // expert / n by multiplication: exact for expert < 1024, n <= 1024 (n = 1
    // needs 2^32, which does not fit; groups of one expert use the identity)
    const int n = a.E / a.groups;
    a.group_m = n == 1 ? 0u : (uint32_t)(((uint64_t)1 << 32) / (uint64_t)n + 1);
    return a;
}

hipError_t launch_router_fwd(const RouterArgs &in, hipStream_t s)
{
    const RouterArgs a = prepared(in);
    const dim3 grid((unsigned)((a.T + 3) / 4));
    const size_t lds = a.topk_groups < a.groups ? sizeof(double) * 4 * (size_t)a.E : 0;
    auto k = a.E <= 64    ? router_fwd_kernel<1>
             : a.E <= 128 ? router_fwd_kernel<2>
             : a.E <= 256 ? router_fwd_kernel<4>
             : a.E <= 512 ? router_fwd_kernel<8>
                          : router_fwd_kernel<16>;
    hipLaunchKernelGGL(k, grid, dim3(256), lds, s, a);
    return hipGetLastError();
}

hipError_t launch_router_bwd(const RouterArgs &in, hipStream_t s)
{
    const RouterArgs a = prepared(in);
    const dim3 grid((unsigned)((a.T + 3) / 4));
    auto k = a.E <= 64    ? router_bwd_kernel<1>
             : a.E <= 128 ? router_bwd_kernel<2>
             : a.E <= 256 ? router_bwd_kernel<4>
             : a.E <= 512 ? router_bwd_kernel<8>
                          : router_bwd_kernel<16>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace moe
