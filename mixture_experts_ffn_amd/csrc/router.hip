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

__device__ inline double wave_max_d(double v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v = fmax(v, __shfl_xor(v, m));
    return v;
}
__device__ inline float wave_max(float v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v = fmaxf(v, __shfl_xor(v, m));
    return v;
}
template <typename V> __device__ inline V wave_sum(V v)
{
#pragma unroll
    for (int m = 32; m; m >>= 1)
        v += __shfl_xor(v, m);
    return v;
}

__device__ inline float load_logit(const RouterArgs &a, int64_t t, int j)
{
    const int64_t at = t * a.stride + j;
    return a.bf16 ? (float)static_cast<const bf16 *>(a.logits)[at]
                  : static_cast<const float *>(a.logits)[at];
}

// One wave per token, expert j on lane j % 64.  Scores that are compared with
// each other are formed in 64 bits: sums of a score and a bias, or of two
// scores, of different experts lie within fp32's rounding of each other often
// enough to change ids.
template <int EPL>
__global__ __launch_bounds__(256) void router_fwd_kernel(RouterArgs a)
{
    extern __shared__ double s_key[]; // [4 waves][E]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = a.E, K = a.K;
    double *keys = s_key + (int64_t)wave * E;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= a.T)
        return;
    float l[EPL];
    float top = -INFINITY;
    bool bad = false; // NaN or +inf: the softmax of the row is NaN
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 64 * i;
        l[i] = j < E ? load_logit(a, t, j) : -INFINITY;
        top = fmaxf(top, l[i]);
        bad |= !(l[i] < INFINITY);
    }
    top = wave_max(top);
    bad = __ballot(bad) != 0;
    const bool grouped = a.topk_groups < a.groups;
    const bool need_score = a.bias || (grouped && a.group_top == 2);
    double total = 0.0; // softmax denominator
    if (!a.sigmoid && (need_score || !a.renorm)) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (l[i] > -INFINITY)
                total += exp((double)l[i] - (double)top);
        total = wave_sum(total);
    }
    auto score = [&](float v) {
        return a.sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top) / total;
    };
    double key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 64 * i;
        double k = l[i];
        if (need_score && j < E && l[i] > -INFINITY) {
            k = score(l[i]);
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
        if (need_score && !a.bias) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] > -INFINITY)
                    key[i] = isnan(l[i]) ? -DBL_MAX : (double)l[i];
        }
    }
    // K times the largest key; lane k keeps slot k
    int my_id = -1;
    float my_l = -INFINITY;
    for (int k = 0; k < K; ++k) {
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
        // lowest id among the holders: lowest register index, then lowest lane
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
        if (lane == k) {
            my_id = id;
            my_l = v;
        }
    }
    const bool live = my_id >= 0;
    float w;
    if (a.sigmoid) {
        if (a.renorm) {
            // s = e^min(l,0) / (1 + e^-|l|); e^-M cancels, so that a row of
            // very negative logits keeps its ratios
            const float neg = live ? fminf(my_l, 0.f) : -INFINITY;
            const float M = wave_max(neg);
            const float s = live ? expf(neg - M) / (1.f + expf(-fabsf(my_l))) : 0.f;
            w = s / wave_sum(s);
        } else {
            w = 1.f / (1.f + expf(-my_l));
        }
    } else if (a.renorm) {
        const float M = wave_max(my_l);
        const float s = live ? expf(my_l - M) : 0.f;
        w = s / wave_sum(s);
    } else {
        w = (float)(exp((double)my_l - (double)top) / total);
    }
    if (!a.sigmoid && bad)
        w = NAN;
    if (lane < K) {
        a.weights[t * K + lane] = live ? a.scale * w : 0.f;
        if (a.ids64)
            static_cast<int64_t *>(a.ids)[t * K + lane] = my_id;
        else
            static_cast<int32_t *>(a.ids)[t * K + lane] = my_id;
    }
}

// One wave per token.  Lane k < K owns slot k; then every lane writes its
// experts' gradients, zeros included.
template <int EPL>
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
    const float lk = id >= 0 ? load_logit(a, t, id) : -INFINITY;
    if (lk == -INFINITY) {
        id = -1;
        g = 0.f;
    }
    float l[EPL];
    float top = -INFINITY, total = 1.f;
    const bool dense = !a.sigmoid && !a.renorm;
    if (dense) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int j = lane + 64 * i;
            l[i] = j < E ? load_logit(a, t, j) : -INFINITY;
            top = fmaxf(top, l[i]);
        }
        top = wave_max(top);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            l[i] = l[i] == -INFINITY ? 0.f : expf(l[i] - top);
            z += l[i];
        }
        total = wave_sum(z);
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
    float own[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        own[i] = 0.f;
    for (int k = 0; k < K; ++k) {
        const int j = __shfl(id, k);
        const float v = __shfl(d, k);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (lane + 64 * i == j)
                own[i] += v;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 64 * i;
        if (j >= E)
            continue;
        float v = own[i];
        if (dense)
            v = l[i] > 0.f || isnan(l[i]) ? l[i] / total * (v - dot) : 0.f;
        if (a.bf16)
            static_cast<bf16 *>(a.d_logits)[t * E + j] = (bf16)v;
        else
            static_cast<float *>(a.d_logits)[t * E + j] = v;
    }
}

hipError_t launch_router_fwd(const RouterArgs &a, hipStream_t s)
{
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

hipError_t launch_router_bwd(const RouterArgs &a, hipStream_t s)
{
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
