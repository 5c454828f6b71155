// router.hip — router logits to expert ids and gates, and the gradient.
//
// For a token's logits l [E], with score s_j = softmax(l)_j or sigmoid(l_j):
//   key_j = s_j + bias_j (no bias: l_j, which orders the experts like s_j does)
//   groups: only the experts of the topk_groups best groups stay open, a
//           group's value being its largest key or the sum of its two largest
//   ids    = the K open experts of largest key, ties to the lower id
//   w_k    = scale * s_k, or scale * s_k / sum of the selected s
// An expert whose logit (or bias) is -inf is closed; slots left without an
// open expert get id -1 and gate 0.  A NaN key is below every number, a sum of
// two keys with a NaN below every sum without; a group with fewer open experts
// than its value adds up has the lowest value.
//
// Gradients (u_k = s_k / sum of the selected s, g_k = scale * d w_k):
//   softmax, renormalised  dl_k = u_k (g_k - sum_i g_i u_i)
//   softmax                dl_j = s_j ([j selected] g_j - sum_i g_i s_i)
//   sigmoid, renormalised  dl_k = u_k (1 - s_k) (g_k - sum_i g_i u_i)
//   sigmoid                dl_k = g_k s_k (1 - s_k)
// and zero elsewhere; the selection has no gradient.
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
struct Bits64 {
    uint32_t lo, hi;
    Bits64() = default;
    __device__ Bits64(uint32_t l, uint32_t h) : lo(l), hi(h) {}
    __device__ explicit Bits64(double v)
    {
        const uint64_t b = (uint64_t)__double_as_longlong(v);
        lo = (uint32_t)b;
        hi = (uint32_t)(b >> 32);
    }
    __device__ double value() const
    {
        return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
    }
};
// The maximum instruction itself, for operands that are no NaNs (fmax would
// first quieten both).
__device__ inline double max_d(double x, double y)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(x), "v"(y));
    return r;
}
// The two wait states between an instruction that writes a register and a DPP
// move or lane swap that reads it: the compiler adds them behind its own
// instructions, not behind an asm block.
__device__ inline double settled(double v)
{
    asm("s_nop 1" : "+v"(v));
    return v;
}
template <int CTRL> __device__ inline double dpp_d(double v)
{
    const Bits64 b(v);
    return Bits64(dpp<CTRL>(b.lo), dpp<CTRL>(b.hi)).value();
}
__device__ inline double row_max_d(double v) // over 16 lanes
{
    v = settled(v);
    v = settled(max_d(v, dpp_d<0xB1>(v)));
    v = settled(max_d(v, dpp_d<0x4E>(v)));
    v = settled(max_d(v, dpp_d<0x141>(v)));
    return settled(max_d(v, dpp_d<0x140>(v)));
}
__device__ inline double wave_max_d(double v)
{
    v = row_max_d(v);
    Bits64 b(v);
    auto l = __builtin_amdgcn_permlane16_swap(b.lo, b.lo, false, false);
    auto h = __builtin_amdgcn_permlane16_swap(b.hi, b.hi, false, false);
    b = Bits64(settled(max_d(Bits64(l[0], h[0]).value(), Bits64(l[1], h[1]).value())));
    l = __builtin_amdgcn_permlane32_swap(b.lo, b.lo, false, false);
    h = __builtin_amdgcn_permlane32_swap(b.hi, b.hi, false, false);
    return max_d(Bits64(l[0], h[0]).value(), Bits64(l[1], h[1]).value());
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

// The same of the bias; -inf past the last.
template <int R> __device__ inline void load_bias(const RouterArgs &a, int lane, float *b)
{
    const int j0 = lane * R;
    if (a.vec_bias && j0 + R <= a.E) {
        typedef float V __attribute__((ext_vector_type(R)));
        const V v = *reinterpret_cast<const V *>(a.bias + j0);
#pragma unroll
        for (int i = 0; i < R; ++i)
            b[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            b[i] = j0 + i < a.E ? a.bias[j0 + i] : -INFINITY;
    }
}

// What a launch compares: logits, logits within groups of the largest logits,
// or scores (with a bias, or in groups by the sum of two), by score function.
enum { BY_LOGIT = 0, BY_LOGIT_GROUPED = 1, BY_SOFTMAX = 2, BY_SIGMOID = 3 };

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

// A NaN key in 64 bits: below every fp32 number, and so is the sum of two of
// them, which stays above a closed expert's -inf.
constexpr double kNanKey = -1e300;

// What the selection leaves in lane k < K: slot k's expert (or -1) and logit.
struct Slot {
    int id;
    float l;
};

// Selection in 64 bits, one wave a row, R experts a lane: for the rows whose
// keys or group values lie too close together for the fp32 selection.
template <int R>
__device__ inline Slot select_exact(const RouterArgs &a, int64_t t, int lane, double *keys)
{
    const int E = a.E;
    float l[R];
    load_row<R>(a, t, lane, l);
    float top = l[0];
#pragma unroll
    for (int i = 1; i < R; ++i)
        top = fmaxf(top, l[i]);
    top = wave_max(top);
    const bool grouped = a.topk_groups < a.groups;
    const bool pair = grouped && a.group_top == 2;
    double key[R];
    if (a.bias || pair) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
        } else {
            double total = 0.0;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                key[i] = l[i] == -INFINITY ? 0.0 : exp((double)l[i] - (double)top);
                total += key[i];
            }
            total = wave_sum_d(total);
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i] /= total;
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            key[i] = (double)l[i];
    }
    bool closed[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        closed[i] = l[i] == -INFINITY;
    if (a.bias) {
        float b[R];
        load_bias<R>(a, lane, b);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            key[i] += (double)b[i];
            closed[i] |= b[i] == -INFINITY;
        }
    }
    // closed before NaN: a NaN score and a bias of -inf add up to NaN
#pragma unroll
    for (int i = 0; i < R; ++i)
        key[i] = closed[i] ? -INFINITY : isnan(key[i]) ? kNanKey : key[i];
    if (grouped) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (lane * R + i < E)
                keys[lane * R + i] = key[i];
        __builtin_amdgcn_wave_barrier();
        const int n = E / a.groups, lg = a.group_lanes, g = lane / lg;
        double b0 = -INFINITY, b1 = -INFINITY;
        if (g < a.groups)
            for (int i = lane & (lg - 1); i < n; i += lg) {
                const double k = keys[g * n + i];
                b1 = fmax(b1, fmin(b0, k));
                b0 = fmax(b0, k);
            }
        for (int m = 1; m < lg; m *= 2) {
            const double o0 = __shfl_xor(b0, m), o1 = __shfl_xor(b1, m);
            b1 = fmax(fmax(b1, o1), fmin(b0, o0));
            b0 = fmax(b0, o0);
        }
        // +inf beside a closed expert would add up to NaN
        const double value = g >= a.groups          ? -INFINITY
                             : pair && b1 > -INFINITY ? b0 + b1
                             : pair                   ? -INFINITY
                                                      : b0;
        const Bits64 vb(value);
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const double v = Bits64(__builtin_amdgcn_readlane(vb.lo, o * lg),
                                    __builtin_amdgcn_readlane(vb.hi, o * lg))
                                 .value();
            rank += v > value || (v == value && o < g);
        }
        const uint64_t kept = __ballot(g < a.groups && rank < a.topk_groups);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t j = lane * R + i;
            const uint32_t og = a.group_m ? __umulhi(j, a.group_m) : j; // expert / n
            const bool in = j < (uint32_t)E && (kept >> (og * lg & 63) & 1);
            // without a bias, by logit within the groups
            const double k = a.bias ? key[i] : isnan(l[i]) ? kNanKey : (double)l[i];
            key[i] = in && key[i] > -INFINITY ? k : -INFINITY;
        }
    }
    // K times the largest key; lane k keeps slot k
    Slot mine = {-1, -INFINITY};
    for (int k = 0; k < a.K; ++k) {
        double m = key[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            m = max_d(m, key[i]);
        const double best = wave_max_d(m);
        if (__ballot(best > -INFINITY) == 0)
            break;
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
                key[i] = -INFINITY;
        const int id = from * R + __builtin_amdgcn_readlane(at, from);
        const float vl = lane_value(v, from);
        if (lane == k)
            mine = {id, vl};
    }
    return mine;
}

// Selection in 32 bits, one wave a row, R experts a lane.  Logits order the
// experts exactly.  Keys that are a sum (score and bias, two scores of a
// group) are rounded, and where two that were compared lie closer than the
// rounding may move them the row is left to select_exact (returns false; with
// scores spread over (0, 1) about one row in a thousand).  The bound, with
// u = 2^-24:
//   sigmoid: exponential 2u, sum u, reciprocal 2u of a value <= 1: 5u
//   softmax: exponent |x| u (times p <= e^-|x|: 0.4u), exponential 2u, the
//            denominator 10u (tree of 16 a lane and six levels) + 2u + u times
//            the mean |x| <= ln E < 7, reciprocal 2u, product u: below 25u
//   key:     u |key| on top
// so two keys of at most `size` may move 10u or 50u and 2u size against each
// other; key_margin has 16u or 56u and 3u size, for its own rounding too.  Only
// neighbours in the order are compared: towards a lower key the distance grows
// faster than its margin.  `size` is that of the two keys alone, so an expert
// that a bias of -1e9 switches off costs nothing.
template <int KIND>
constexpr float kMargin = KIND == BY_SIGMOID ? 0x1p-20f : 7 * 0x1p-21f;
template <int KIND> __device__ inline float key_margin(float x, float y)
{
    return kMargin<KIND> + 3 * 0x1p-24f * fmaxf(fabsf(x), fabsf(y));
}
// How far a group's value may be off: a key, or half the sum of two, b0 >= b1,
// rounded (2u of the larger), and the rounding of value -+ error where it is
// compared (u more).  Every kept group has to stay above every other one.
template <int KIND> __device__ inline float group_error(bool pair, float b0, float b1, float value)
{
    const float size = pair ? fmaxf(b0, -b1) : fabsf(b0);
    return value == -INFINITY ? 0.f : 0.5f * kMargin<KIND> + 0x1p-22f * size;
}

// A group's value by the sum of two is compared by its half: the sum of two
// biases of a type's lowest value would be that of a closed group, -inf.
__device__ inline float half_sum(float x, float y) { return 0.5f * x + 0.5f * y; }

template <int R, int KIND>
__device__ inline bool select_fast(const RouterArgs &a, const float *l, float top, float total,
                                   int lane, float *keys, Slot *out)
{
    const int E = a.E, K = a.K;
    const bool grouped = KIND != BY_LOGIT && a.topk_groups < a.groups;
    const bool sums = KIND >= BY_SOFTMAX && a.bias != nullptr;
    const bool pair = KIND >= BY_SOFTMAX && grouped && a.group_top == 2;
    bool ok = true;
    float score[R];
    if constexpr (KIND == BY_SIGMOID) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            score[i] = __builtin_amdgcn_rcpf(1.f + __expf(-l[i]));
    } else if constexpr (KIND == BY_SOFTMAX) {
        const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
        for (int i = 0; i < R; ++i)
            score[i] = expf(l[i] - top) * inv;
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            score[i] = l[i];
    }
    uint32_t key[R];
    if (sums) {
        float b[R];
        load_bias<R>(a, lane, b);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            score[i] += b[i];
            key[i] = order_of(score[i], l[i] == -INFINITY || b[i] == -INFINITY);
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            key[i] = order_of(l[i], l[i] == -INFINITY);
    }
    if (KIND != BY_LOGIT) {
        bool odd = false; // scores that are no finite numbers are left to select_exact
#pragma unroll
        for (int i = 0; i < R; ++i)
            odd |= key[i] != 0u && !(fabsf(score[i]) < INFINITY);
        ok = __ballot(odd) == 0;
    }
    if (grouped) {
        // a group's value: a power of two of lanes scan its experts in LDS
        const int n = E / a.groups;
        const int lg = a.group_lanes, g = lane / lg;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (lane * R + i < E)
                keys[lane * R + i] = key[i] == 0u ? -INFINITY : score[i];
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
        const float value = g >= a.groups ? -INFINITY : pair ? half_sum(b0, b1) : b0;
        int rank = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float v = lane_value(value, o * lg);
            rank += v > value || (v == value && o < g);
        }
        const bool keep = g < a.groups && rank < a.topk_groups;
        const uint64_t kept = __ballot(keep);
        if (sums || pair) {
            const float err = group_error<KIND>(pair, b0, b1, value);
            const float lo = wave_min(keep ? value - err : INFINITY);
            const float hi = wave_max(keep ? -INFINITY : value + err);
            ok = ok && (lo > hi || hi == -INFINITY);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint32_t j = lane * R + i;
            const int og = a.group_m ? (int)__umulhi(j, a.group_m) : (int)j; // expert / n
            key[i] = j < (uint32_t)E && (kept >> (og * lg & 63) & 1) ? key[i] : 0u;
        }
    }
    Slot mine = {-1, -INFINITY};
    float last = 0.f;
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
            ok = ok && (k == 0 || last - v > key_margin<KIND>(last, v));
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

// Gate and id of slot k, kept by lane k of N lanes, to memory.
template <int N>
__device__ inline void store_slots(const RouterArgs &a, int64_t t, int k, const Slot &mine, float top,
                                   float total, bool bad, bool write)
{
    const auto fmax2 = [](uint32_t x, uint32_t y) {
        return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
    };
    const auto fadd2 = [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    };
    const auto largest = [&](float v) {
        return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), fmax2));
    };
    const auto sum = [&](float v) {
        return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), fadd2));
    };
    const bool live = mine.id >= 0;
    float w;
    if (a.sigmoid) {
        if (a.renorm) {
            // s = e^min(l,0) / (1 + e^-|l|); e^-M cancels, so that a row of
            // very negative logits keeps its ratios
            const float neg = live ? fminf(mine.l, 0.f) : -INFINITY;
            const float M = largest(neg);
            const float s = live ? expf(neg - M) / (1.f + expf(-fabsf(mine.l))) : 0.f;
            w = s / sum(s);
        } else {
            w = 1.f / (1.f + expf(-mine.l));
        }
    } else if (a.renorm) {
        const float M = largest(mine.l);
        const float s = live ? expf(mine.l - M) : 0.f;
        w = s / sum(s);
    } else {
        w = expf(mine.l - top) / total;
    }
    if (bad)
        w = NAN;
    if (write && k < a.K) {
        a.weights[t * a.K + k] = live ? a.scale * w : 0.f;
        if (a.ids64)
            static_cast<int64_t *>(a.ids)[t * a.K + k] = mine.id;
        else
            static_cast<int32_t *>(a.ids)[t * a.K + k] = mine.id;
    }
}

// ---- sixteen lanes a row ------------------------------------------------------------
//
// Four rows share a wave, and with them what a round of the selection costs
// whatever the row's length: with 64 lanes a row, 32768 rows of 256 experts in
// 8 groups take 50 us, here 23 (their bytes need 7).  A key is a double: an fp32 key, exactly, with
// the expert's number in the 29 bits below it, so that one maximum finds the
// largest key, breaks ties towards the lower id and names the expert.
constexpr uint32_t kClosedHi = 0xD2B00000u; // -2^300: closed or taken
constexpr uint32_t kNanHi = 0xCC700000u;    // -2^200: a NaN, below every number
constexpr uint32_t kInfHi = 0x4C700000u;    //  2^200: +inf

// of a finite value
__device__ inline Bits64 number_key(float v, bool closed, int j)
{
    Bits64 k((double)v);
    k.lo |= (int32_t)k.hi < 0 ? (uint32_t)j : 1023u - (uint32_t)j;
    k.hi = closed ? kClosedHi : k.hi;
    return k;
}
// of any
__device__ inline Bits64 any_key(float v, bool closed, int j)
{
    Bits64 k((double)(v + 0.0f));
    if (!(fabsf(v) < INFINITY)) {
        k.hi = v == INFINITY ? kInfHi : kNanHi;
        k.lo = 0u;
    }
    k.lo |= (int32_t)k.hi < 0 ? (uint32_t)j : 1023u - (uint32_t)j;
    k.hi = closed ? kClosedHi : k.hi;
    return k;
}
template <int R> __device__ inline double largest_of(const Bits64 *k)
{
    if constexpr (R == 1)
        return k[0].value();
    else
        return max_d(largest_of<R / 2>(k), largest_of<R / 2>(k + R / 2));
}
__device__ inline float row_max(float v)
{
    return __uint_as_float(lanes_reduce<16>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
__device__ inline bool row_any(bool v, int lane)
{
    return (__ballot(v) >> (lane & 48) & 0xffffu) != 0;
}

// How many of the row's other groups (of 2^shift lanes each) come before this
// lane's: those of a larger value, or of an equal one and a lower number.
template <int O> __device__ inline int rank_step(float value, int sub, int shift)
{
    int r = 0;
    if ((O & ((1 << shift) - 1)) == 0) {
        const float v = __uint_as_float(dpp<0x120 + O>(__float_as_uint(value))); // row_ror: O
        // the lane the value came from, O below, or wrapped around above
        r = v > value || (v == value && sub >= O);
    }
    if constexpr (O < 15)
        r += rank_step<O + 1>(value, sub, shift);
    return r;
}

template <int R, int KIND>
__global__ __launch_bounds__(256) void router_rows_kernel(RouterArgs a)
{
    extern __shared__ double s_key[]; // [4 waves][E], with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
    if (t0 >= a.T)
        return;
    const bool here = t0 + (lane >> 4) < a.T;
    const int64_t t = here ? t0 + (lane >> 4) : a.T - 1;
    float l[R];
    load_row<R>(a, t, sub, l);
    float top = 0.f, total = 1.f;
    bool bad = false;
    if (!a.sigmoid) {
        top = l[0];
        bool odd = !(l[0] < INFINITY);
#pragma unroll
        for (int i = 1; i < R; ++i) {
            top = fmaxf(top, l[i]);
            odd |= !(l[i] < INFINITY);
        }
        top = row_max(top);
        bad = row_any(odd, lane);
        if (a.need_total) {
            float e[R];
#pragma unroll
            for (int i = 0; i < R; ++i)
                e[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - top);
            total = __uint_as_float(lanes_reduce<16>(
                __float_as_uint(tree_sum<R>(e)), [](uint32_t x, uint32_t y) {
                    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
                }));
        }
    }
    // keys, and whether fp32 orders them (select_fast)
    const bool grouped = KIND != BY_LOGIT && a.topk_groups < a.groups;
    const bool sums = KIND >= BY_SOFTMAX && a.bias != nullptr;
    const bool pair = KIND >= BY_SOFTMAX && grouped && a.group_top == 2;
    bool ok = true;
    Bits64 key[R];
    if constexpr (KIND == BY_LOGIT) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            key[i] = any_key(l[i], l[i] == -INFINITY, sub * R + i);
    } else {
        float v[R];
        if constexpr (KIND == BY_SIGMOID) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = __builtin_amdgcn_rcpf(1.f + __expf(-l[i]));
        } else if constexpr (KIND == BY_SOFTMAX) {
            const float inv = __builtin_amdgcn_rcpf(total);
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = expf(l[i] - top) * inv;
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                v[i] = l[i];
        }
        bool closed[R];
        if (sums) {
            float b[R];
            load_bias<R>(a, sub, b);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                closed[i] = fminf(l[i], b[i]) == -INFINITY;
                v[i] += b[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                closed[i] = l[i] == -INFINITY;
        }
        // scores that are no finite numbers are left to the exact selection
        bool odd = false;
#pragma unroll
        for (int i = 0; i < R; ++i)
            odd |= !(closed[i] || fabsf(v[i]) < INFINITY);
        if constexpr (KIND == BY_LOGIT_GROUPED) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i] = any_key(l[i], closed[i], sub * R + i);
        } else if (sums) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i] = number_key(v[i], closed[i], sub * R + i);
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i] = any_key(l[i], closed[i], sub * R + i);
        }
        ok = !row_any(odd, lane);
        float b0 = -INFINITY, b1 = -INFINITY;
        if (grouped) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float x = closed[i] ? -INFINITY : v[i];
                b1 = __builtin_amdgcn_fmed3f(b0, b1, x); // b0 >= b1
                b0 = fmaxf(b0, x);
            }
        }
        if (grouped) {
            // a group is 2^shift whole lanes (the launch checks it)
            const int shift = a.group_shift;
            auto join = [&](uint32_t o0, uint32_t o1) {
                const float f0 = __uint_as_float(o0), f1 = __uint_as_float(o1);
                b1 = fmaxf(fmaxf(b1, f1), fminf(b0, f0));
                b0 = fmaxf(b0, f0);
            };
            if (shift >= 1)
                join(dpp<0xB1>(__float_as_uint(b0)), dpp<0xB1>(__float_as_uint(b1)));
            if (shift >= 2)
                join(dpp<0x4E>(__float_as_uint(b0)), dpp<0x4E>(__float_as_uint(b1)));
            if (shift >= 3)
                join(dpp<0x141>(__float_as_uint(b0)), dpp<0x141>(__float_as_uint(b1)));
            const float value = pair ? half_sum(b0, b1) : b0;
            const bool keep = rank_step<1>(value, sub, shift) < a.topk_groups;
            if (sums || pair) {
                const float err = group_error<KIND>(pair, b0, b1, value);
                const float lo = -row_max(keep ? err - value : -INFINITY);
                const float hi = row_max(keep ? -INFINITY : value + err);
                ok = ok && (lo > hi || hi == -INFINITY);
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
                key[i].hi = keep ? key[i].hi : kClosedHi;
        }
    }
    // lane k keeps slot k's key
    Bits64 kept(0u, kClosedHi), m;
    for (int k = 0; k < a.K; ++k) {
        m = Bits64(row_max_d(largest_of<R>(key)));
        kept.lo = sub == k ? m.lo : kept.lo;
        kept.hi = sub == k ? m.hi : kept.hi;
#pragma unroll
        for (int i = 0; i < R; ++i)
            key[i].hi = key[i].lo == m.lo ? kClosedHi : key[i].hi; // one expert's (256 at most)
    }
    if (sums) {
        // each slot against the next, the last against the first one left out
        m = Bits64(row_max_d(largest_of<R>(key)));
        Bits64 below(dpp<0x12F>(kept.lo), dpp<0x12F>(kept.hi)); // lane + 1's
        if (sub == a.K - 1)
            below = m;
        const auto number = [](const Bits64 &k) {
            return (float)Bits64(k.lo & 0xE0000000u, k.hi).value();
        };
        const float x = number(kept), y = number(below);
        const bool near = !(x - y > key_margin<KIND>(x, y));
        ok = ok && !row_any(sub < a.K && below.hi != kClosedHi && near, lane);
    }
    const int n = (int)(kept.lo & 1023u);
    const int my_id = kept.hi == kClosedHi ? -1 : (int32_t)kept.hi < 0 ? n : 1023 - n;
    Slot mine = {my_id, my_id >= 0 ? load_logit(a, t, my_id) : -INFINITY};
    const uint64_t again = KIND == BY_LOGIT ? 0 : __ballot(!ok && here);
    if (again) {
        double *keys = s_key + (int64_t)wave * a.E;
        for (int r = 0; r < 4; ++r) {
            if (!(again >> (16 * r) & 1))
                continue;
            __builtin_amdgcn_wave_barrier();
            const Slot x = select_exact<(R + 3) / 4>(a, t0 + r, lane, keys);
            const int id = __shfl(x.id, sub);
            const float xl = __shfl(x.l, sub);
            if (lane >> 4 == r)
                mine = {id, xl};
        }
    }
    store_slots<16>(a, t, sub, mine, top, total, bad, here);
}

// One wave per token.
template <int R, int KIND>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ double s_key[]; // [4 waves][E], with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    if (!select_fast<R, KIND>(a, l, top, total, lane, reinterpret_cast<float *>(keys), &mine)) {
        __builtin_amdgcn_wave_barrier();
        mine = select_exact<R>(a, t, lane, keys);
    }
    store_slots<64>(a, t, lane, mine, top, total, bad, true);
}

// ---- gradient -------------------------------------------------------------------------

// Slot k of a row, in lane k of the row's N lanes: its expert (-1: none), and
// its own part of that expert's gradient; `dot` is what softmax's every score
// loses (and then `d` still has to be scaled by the score).
struct SlotGrad {
    int id;
    float d, dot;
};
template <int N>
__device__ inline SlotGrad slot_grad(const RouterArgs &a, int64_t t, int k, float top, float total)
{
    const auto largest = [](float v) {
        return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
            return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
        }));
    };
    const auto sum = [](float v) {
        return __uint_as_float(lanes_reduce<N>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
            return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
        }));
    };
    SlotGrad s = {-1, 0.f, 0.f};
    float g = 0.f, lk = -INFINITY;
    if (k < a.K) {
        const int64_t v = a.ids64 ? static_cast<const int64_t *>(a.ids)[t * a.K + k]
                                  : static_cast<const int32_t *>(a.ids)[t * a.K + k];
        if (v >= 0 && v < a.E) {
            lk = load_logit(a, t, (int)v);
            if (lk != -INFINITY) {
                s.id = (int)v;
                g = a.scale * a.d_weights[t * a.K + k];
            }
        }
    }
    const bool live = s.id >= 0;
    if (!a.sigmoid && !a.renorm) {
        const float p = live ? expf(lk - top) / total : 0.f;
        s.dot = sum(g * p);
        s.d = g;
    } else if (a.renorm) {
        const float neg = !live ? -INFINITY : a.sigmoid ? fminf(lk, 0.f) : lk;
        const float M = largest(neg);
        float e = live ? expf(neg - M) : 0.f;
        if (a.sigmoid && live)
            e /= 1.f + expf(-fabsf(lk));
        const float all = sum(e);
        const float u = live ? e / all : 0.f;
        s.d = u * (g - sum(g * u));
        if (a.sigmoid && live)
            s.d *= 1.f / (1.f + expf(lk));
    } else if (live) {
        const float e = expf(-fabsf(lk));
        s.d = g * e / ((1.f + e) * (1.f + e));
    }
    return s;
}

// The softmax denominator's parts of a lane's logits, in place of them; a closed
// expert's is -0, which the sum does not see.
template <int R> __device__ inline void exponentials(float *l, float top)
{
#pragma unroll
    for (int i = 0; i < R; ++i)
        l[i] = l[i] == -INFINITY ? -0.f : expf(l[i] - top);
}
// A row of closed experts only, a padded token's, takes the short way below too.
__device__ inline float inverse_total(float total) { return total == 0.f ? 0.f : 1.f / total; }

// Softmax's gradients g[0, N) from the experts' own parts g and those.  Where the
// row's values are finite a closed expert's comes out as zero by itself.  Else
// every open expert takes the formula, one that underflowed to +0 as well, so
// that a NaN of the row reaches it; closed ones, and rows without a slot, have
// no gradient.  (With the selection in every row: 32768 x 256 f32 14.7 us, so 14.4.)
template <int N>
__device__ inline void dense_grads(const float *part, float inv, float dot, bool any, float *g)
{
    if (fabsf(inv * dot) < INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            g[i] = part[i] * inv * (g[i] - dot);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool closed = __float_as_uint(part[i]) == 0x80000000u;
            g[i] = closed || !any ? 0.f : part[i] * inv * (g[i] - dot);
        }
    }
}

// N consecutive gradients of token t, from expert j0 on (zeros included).
template <int N>
__device__ inline void store_grads(const RouterArgs &a, int64_t t, int j0, const float *v)
{
    const int64_t at = t * a.E + j0;
    if (a.vec_out && j0 + N <= a.E) {
        if (a.bf16) {
            typedef bf16 V __attribute__((ext_vector_type(N)));
            V o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = (bf16)v[i];
            *reinterpret_cast<V *>(static_cast<bf16 *>(a.d_logits) + at) = o;
        } else {
            typedef float V __attribute__((ext_vector_type(N)));
            V o;
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = v[i];
            *reinterpret_cast<V *>(static_cast<float *>(a.d_logits) + at) = o;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (j0 + i >= a.E)
            continue;
        if (a.bf16)
            static_cast<bf16 *>(a.d_logits)[at + i] = (bf16)v[i];
        else
            static_cast<float *>(a.d_logits)[at + i] = v[i];
    }
}

// One wave per token.
template <int R>
__global__ __launch_bounds__(256) void router_bwd_kernel(RouterArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T)
        return;
    const bool dense = !a.sigmoid && !a.renorm;
    float l[R];
    float top = 0.f, total = 1.f;
    if (dense) {
        load_row<R>(a, t, lane, l);
        top = l[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            top = fmaxf(top, l[i]);
        top = wave_max(top);
        exponentials<R>(l, top);
        total = wave_sum(tree_sum<R>(l));
    }
    const SlotGrad s = slot_grad<64>(a, t, lane, top, total);
    float own[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        own[i] = 0.f;
    for (int k = 0; k < a.K; ++k) {
        const int j = __builtin_amdgcn_readlane(s.id, k);
        const float v = lane_value(s.d, k);
#pragma unroll
        for (int i = 0; i < R; ++i)
            own[i] += lane * R + i == j ? v : 0.f;
    }
    if (dense) {
        dense_grads<R>(l, inverse_total(total), s.dot, __ballot(s.id >= 0) != 0, own);
    }
    store_grads<R>(a, t, lane * R, own);
}

// Sum over the row's slots of the same expert as this lane's, in the order of
// the slots, and whether an earlier slot has that expert.
template <int O>
__device__ inline void join_slots(int K, int id, float d, int sub, float *sum, bool *later)
{
    if (O < K) {
        const int oid = (int)dpp<0x150 + O>((uint32_t)id); // row_newbcast: lane O of the 16
        const float od = __uint_as_float(dpp<0x150 + O>(__float_as_uint(d)));
        *sum += oid == id ? od : 0.f;
        *later |= oid == id && O < sub;
    }
    if constexpr (O < 15)
        join_slots<O + 1>(K, id, d, sub, sum, later);
}

// Sixteen lanes a row, up to 256 experts and 16 slots: the slots' parts reach
// their experts' lanes through LDS, and the gradients leave through it, so
// that a store covers consecutive experts (a lane's own are R apart).  With 64
// lanes a row, 32768 rows of 256 experts take 18 us and of 64 experts 12, here
// 9 and 5.
template <int R>
__global__ __launch_bounds__(256) void router_bwd_rows_kernel(RouterArgs a)
{
    __shared__ __attribute__((aligned(16))) float s_own[16][16 * R + (R > 4 ? R : 0)];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
    if (t0 >= a.T)
        return;
    const bool here = t0 + (lane >> 4) < a.T;
    const int64_t t = here ? t0 + (lane >> 4) : a.T - 1;
    const bool dense = !a.sigmoid && !a.renorm;
    float l[R];
    float top = 0.f, total = 1.f;
    if (dense) {
        load_row<R>(a, t, sub, l);
        top = l[0];
#pragma unroll
        for (int i = 1; i < R; ++i)
            top = fmaxf(top, l[i]);
        top = row_max(top);
        exponentials<R>(l, top);
        total = __uint_as_float(lanes_reduce<16>(
            __float_as_uint(tree_sum<R>(l)), [](uint32_t x, uint32_t y) {
                return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
            }));
    }
    const SlotGrad s = slot_grad<16>(a, t, sub, top, total);
    float d = 0.f;
    bool later = false;
    join_slots<0>(a.K, s.id, s.d, sub, &d, &later);
    constexpr int V = R < 4 ? R : 4, LINE = 16 * V + (R > V ? 4 : 0);
    typedef float Vec __attribute__((ext_vector_type(V)));
    // expert j at line (j % R) / V, place j / R
    float *const row = s_own[wave * 4 + (lane >> 4)];
#pragma unroll
    for (int i = 0; i < R / V; ++i)
        *reinterpret_cast<Vec *>(row + i * LINE + sub * V) = Vec{};
    __builtin_amdgcn_wave_barrier(); // one wave's LDS accesses are in order
    if (s.id >= 0 && !later) {
        const int i = s.id % R;
        row[i / V * LINE + s.id / R * V + i % V] = d;
    }
    __builtin_amdgcn_wave_barrier();
    if (dense) {
        const float inv = inverse_total(total);
        const bool any = row_any(s.id >= 0, lane);
#pragma unroll
        for (int i = 0; i < R / V; ++i) {
            Vec v = *reinterpret_cast<const Vec *>(row + i * LINE + sub * V);
            float g[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                g[j] = v[j];
            dense_grads<V>(l + i * V, inv, s.dot, any, g);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = g[j];
            *reinterpret_cast<Vec *>(row + i * LINE + sub * V) = v;
        }
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int n = 0; n < R / V; ++n) {
        const int c = n * 16 + sub; // experts c V + [0, V)
        const Vec v = *reinterpret_cast<const Vec *>(row + c % (R / V) * LINE + c / (R / V) * V);
        float out[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
            out[j] = v[j];
        if (here)
            store_grads<V>(a, t, c * V, out);
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
    a.vec_bias = a.bias && aligned(a.bias, 0);
    a.vec_out = a.d_logits && aligned(a.d_logits, a.E);
    a.need_total = !a.sigmoid && (!a.renorm || a.bias || (a.topk_groups < a.groups && a.group_top == 2));
    int lanes = 64;
    while (lanes * a.groups > 64)
        lanes /= 2;
    a.group_lanes = lanes;
    a.group_shift = 0;
    while (a.groups << (a.group_shift + 1) <= 16)
        ++a.group_shift;
    // expert / n by multiplication: exact for expert < 1024, n <= 1024 (n = 1
    // needs 2^32, which does not fit; groups of one expert use the identity)
    const int n = a.E / a.groups;
    a.group_m = n == 1 ? 0u : (uint32_t)(((uint64_t)1 << 32) / (uint64_t)n + 1);
    return a;
}

template <int KIND> static hipError_t launch_fwd(const RouterArgs &a, hipStream_t s)
{
    const size_t lds = a.topk_groups < a.groups ? sizeof(double) * 4 * (size_t)a.E : 0;
    // Sixteen lanes a row up to 256 experts and 16 slots; groups must be whole
    // lanes there, a power of two of them.
    const int R = a.E <= 16 ? 1 : a.E <= 32 ? 2 : a.E <= 64 ? 4 : a.E <= 128 ? 8 : 16;
    const bool whole = a.E == 16 * R && (a.groups & (a.groups - 1)) == 0 && a.groups <= 16;
    if (a.E <= 256 && a.K <= 16 && (whole || a.topk_groups == a.groups)) {
        auto rows = R == 1   ? router_rows_kernel<1, KIND>
                    : R == 2 ? router_rows_kernel<2, KIND>
                    : R == 4 ? router_rows_kernel<4, KIND>
                    : R == 8 ? router_rows_kernel<8, KIND>
                             : router_rows_kernel<16, KIND>;
        hipLaunchKernelGGL(rows, dim3((unsigned)((a.T + 15) / 16)), dim3(256), lds, s, a);
        return hipGetLastError();
    }
    auto k = a.E <= 64    ? router_fwd_kernel<1, KIND>
             : a.E <= 128 ? router_fwd_kernel<2, KIND>
             : a.E <= 256 ? router_fwd_kernel<4, KIND>
             : a.E <= 512 ? router_fwd_kernel<8, KIND>
                          : router_fwd_kernel<16, KIND>;
    hipLaunchKernelGGL(k, dim3((unsigned)((a.T + 3) / 4)), dim3(256), lds, s, a);
    return hipGetLastError();
}

static hipError_t launch_bwd(const RouterArgs &a, hipStream_t s)
{
    if (a.E <= 256 && a.K <= 16) {
        auto rows = a.E <= 16    ? router_bwd_rows_kernel<1>
                    : a.E <= 32  ? router_bwd_rows_kernel<2>
                    : a.E <= 64  ? router_bwd_rows_kernel<4>
                    : a.E <= 128 ? router_bwd_rows_kernel<8>
                                 : router_bwd_rows_kernel<16>;
        hipLaunchKernelGGL(rows, dim3((unsigned)((a.T + 15) / 16)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    auto k = a.E <= 64    ? router_bwd_kernel<1>
             : a.E <= 128 ? router_bwd_kernel<2>
             : a.E <= 256 ? router_bwd_kernel<4>
             : a.E <= 512 ? router_bwd_kernel<8>
                          : router_bwd_kernel<16>;
    hipLaunchKernelGGL(k, dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

// A launch has fewer than 2^32 threads, up to 64 a row: longer batches take
// several, of 2^25 rows.
template <typename F> static hipError_t in_parts(const RouterArgs &in, F launch)
{
    constexpr int64_t ROWS = (int64_t)1 << 25;
    const RouterArgs a = prepared(in);
    const int64_t es = a.bf16 ? 2 : 4, is = a.ids64 ? 8 : 4;
    for (int64_t t0 = 0; t0 < a.T; t0 += ROWS) {
        RouterArgs p = a;
        p.T = a.T - t0 < ROWS ? a.T - t0 : ROWS;
        p.logits = static_cast<const char *>(a.logits) + t0 * a.stride * es;
        p.ids = static_cast<char *>(a.ids) + t0 * a.K * is;
        if (a.d_logits) {
            p.d_weights = a.d_weights + t0 * a.K;
            p.d_logits = static_cast<char *>(a.d_logits) + t0 * a.E * es;
        } else {
            p.weights = a.weights + t0 * a.K;
        }
        const hipError_t err = launch(p);
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

hipError_t launch_router_fwd(const RouterArgs &in, hipStream_t s)
{
    return in_parts(in, [&](const RouterArgs &a) {
        const bool grouped = a.topk_groups < a.groups;
        if (a.bias || (grouped && a.group_top == 2))
            return a.sigmoid ? launch_fwd<BY_SIGMOID>(a, s) : launch_fwd<BY_SOFTMAX>(a, s);
        return grouped ? launch_fwd<BY_LOGIT_GROUPED>(a, s) : launch_fwd<BY_LOGIT>(a, s);
    });
}

hipError_t launch_router_bwd(const RouterArgs &in, hipStream_t s)
{
    return in_parts(in, [&](const RouterArgs &a) { return launch_bwd(a, s); });
}

} // namespace moe
