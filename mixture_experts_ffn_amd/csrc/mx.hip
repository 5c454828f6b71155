// mx.hip — MXFP4 quantisation of expert weights and its inverse, and the
// per-call quantisation of the token rows (formats and layouts: mx.h).
//
// All three are single passes bound by HBM: a weight of n values moves 2n (or
// 4n) + 17n/32 bytes in either direction, a token row 2H + 17H/32 (MXFP4) or
// 2H + 25H/32 (MXFP6).
#include "kernels.h"
#include "mx.h"

namespace moe {

// Weights.  A block of 32 runs down a column, so a lane owns the blocks of two
// neighbouring columns in one k-block: its 32 loads take 128 bytes a row (256
// in fp32) across 32 lanes, the maxima need no other lane, and its codes are 32
// consecutive bytes of a k-step in the packed layout.  A wave has 64 columns
// (two column tiles) of the two k-blocks of a k-step.  [64, 2048, 2816] bf16
// takes 203 us one way and 160 back, where a large copy of as many bytes takes
// 193; one column a lane, 64 bytes a row, took 498 for the two.
template <typename T> struct __attribute__((aligned(2 * sizeof(T)))) Pair {
    T v[2];
};

// Place of a lane: its columns (col, col + 1) of a panel, its k-step.  Column
// pairs of tiles run fastest in blockIdx.x, which alone carries large numbers.
struct WeightPlace {
    int64_t ep;  // expert * panels + panel
    int col, ks; // ks >= KS: nothing to do
};
__device__ inline WeightPlace weight_place(int NT)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t ntp = (uint32_t)(NT + 1) / 2;
    const uint32_t kq = blockIdx.x / ntp, tp = blockIdx.x - kq * ntp;
    return {(int64_t)blockIdx.y, (int)tp * 64 + (lane & 31) * 2, (int)kq * 4 + wave};
}

template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_weight_kernel(
    const T *__restrict__ w, u32x4 *__restrict__ codes, uint8_t *__restrict__ scales, int Kd, int N,
    int panels, int NT, int KS, int KC)
{
    const WeightPlace q = weight_place(NT);
    const int half = (threadIdx.x & 63) >> 5;
    const int tile = q.col >> 5;
    if (q.ks >= KS || tile >= NT)
        return;
    const int e = (int)(q.ep / panels), panel = (int)(q.ep % panels);
    const int pc = N / panels; // a multiple of 8: both columns are in or out
    const T *base = w + (int64_t)e * Kd * N + (int64_t)panel * pc + q.col;
    const int k0 = q.ks * 64 + half * 32;
    float v[2][32];
    if (q.col < pc && k0 + 32 <= Kd) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const Pair<T> x = *reinterpret_cast<const Pair<T> *>(base + (int64_t)(k0 + i) * N);
            v[0][i] = to_f32<T>(x.v[0]);
            v[1][i] = to_f32<T>(x.v[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                v[c][i] = q.col < pc && k0 + i < Kd ? to_f32<T>(base[(int64_t)(k0 + i) * N + c]) : 0.f;
    }
    const int64_t t = q.ep * NT + tile;
    const int place = half * 32 + (q.col & 31); // lane of the packed layout
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            top = max(top, abs_bits(v[c][i]));
        const int code = mx_scale_code(top);
        const float inv = mx_inverse(code);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[c][i] *= inv;
        u32x4 out;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = mx_pack8_fp4(v[c] + 8 * i);
        codes[(t * KS + q.ks) * 64 + place + c] = out;
        scales[((t * KC + (q.ks >> 2)) * 64 + place + c) * 4 + (q.ks & 3)] = (uint8_t)code;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void mx_dequantize_weight_kernel(
    const u32x4 *__restrict__ codes, const uint8_t *__restrict__ scales, T *__restrict__ w, int Kd,
    int N, int panels, int NT, int KS, int KC)
{
    const WeightPlace q = weight_place(NT);
    const int half = (threadIdx.x & 63) >> 5;
    const int tile = q.col >> 5;
    const int pc = N / panels;
    if (q.ks >= KS || q.col >= pc)
        return;
    const int e = (int)(q.ep / panels), panel = (int)(q.ep % panels);
    T *base = w + (int64_t)e * Kd * N + (int64_t)panel * pc + q.col;
    const int k0 = q.ks * 64 + half * 32;
    const int64_t t = q.ep * NT + tile;
    const int place = half * 32 + (q.col & 31);
    u32x4 code[2];
    float x[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        code[c] = codes[(t * KS + q.ks) * 64 + place + c];
        x[c] = mx_scale_value(scales[((t * KC + (q.ks >> 2)) * 64 + place + c) * 4 + (q.ks & 3)]);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        Pair<T> o;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            o.v[c] = from_f32<T>(mx_fp4_value(code[c][i / 8] >> (4 * (i % 8)) & 15) * x[c]);
        if (k0 + i < Kd)
            *reinterpret_cast<Pair<T> *>(base + (int64_t)(k0 + i) * N) = o;
    }
}

// Token rows by a launch of their own (they mostly ride in the routing launch).
template <int BITS>
__global__ __launch_bounds__(256) void mx_quantize_rows_kernel(MxRows r)
{
    const int64_t n = r.T * (2 * r.KS);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256)
        mx_quantize_block<BITS>(r, i);
}

template <typename T>
static hipError_t weight_t(bool quantize, const void *src, void *codes, void *scales, void *dst,
                           int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const MxDims d(Kd, N / panels);
    // E * panels <= 2048; Kd * N < 2^31 keeps grid.x within 2^22
    const dim3 grid((unsigned)((d.NT + 1) / 2) * (unsigned)((d.KS + 3) / 4), (unsigned)(E * panels));
    if (quantize)
        hipLaunchKernelGGL(mx_quantize_weight_kernel<T>, grid, dim3(256), 0, s,
                           static_cast<const T *>(src), static_cast<u32x4 *>(codes),
                           static_cast<uint8_t *>(scales), (int)Kd, (int)N, panels, d.NT, d.KS, d.KC);
    else
        hipLaunchKernelGGL(mx_dequantize_weight_kernel<T>, grid, dim3(256), 0, s,
                           static_cast<const u32x4 *>(codes), static_cast<const uint8_t *>(scales),
                           static_cast<T *>(dst), (int)Kd, (int)N, panels, d.NT, d.KS, d.KC);
    return hipGetLastError();
}

hipError_t launch_mx_quantize_weight(int dtype, const void *w, void *codes, void *scales, int64_t E,
                                     int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    return dtype == 1 ? weight_t<bf16>(true, w, codes, scales, nullptr, E, Kd, N, panels, s)
                      : weight_t<float>(true, w, codes, scales, nullptr, E, Kd, N, panels, s);
}

hipError_t launch_mx_dequantize_weight(int dtype, const void *codes, const void *scales, void *w,
                                       int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    void *c = const_cast<void *>(codes), *x = const_cast<void *>(scales);
    return dtype == 1 ? weight_t<bf16>(false, nullptr, c, x, w, E, Kd, N, panels, s)
                      : weight_t<float>(false, nullptr, c, x, w, E, Kd, N, panels, s);
}

hipError_t launch_mx_quantize_rows(const MxRows &r, hipStream_t s)
{
    const int64_t blocks = (r.T * r.KS * 2 + 255) / 256;
    const dim3 grid((unsigned)(blocks < 8192 ? blocks : 8192));
    auto k = r.bits == 4 ? mx_quantize_rows_kernel<4> : mx_quantize_rows_kernel<6>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, r);
    return hipGetLastError();
}

} // namespace moe
