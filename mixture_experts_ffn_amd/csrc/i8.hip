// i8.hip — int8 quantisation of weights by column and of token rows, and the
// packed weights' inverse (layouts: i8.h).
//
// A vector's codes need its largest magnitude first: each kernel reads its vectors
// twice, the second time from cache.  Bound by HBM: a weight of n values moves 2n
// (or 4n) + n bytes, a row of Kd 2 Kd (or 4 Kd) + Kd.
#include "i8.h"
#include "kernels.h"

namespace moe {

template <typename T> struct __attribute__((aligned(2 * sizeof(T)))) I8Pair {
    T v[2];
};

// Weights.  A workgroup of eight waves owns 64 columns of a panel; a lane two
// neighbouring columns and 16 of the 32 rows of a k-step, so that a load takes 128
// bytes a row (256 in fp32) and the codes are the lane's own 16 bytes of the
// packed layout.  The waves share out the k-steps.
constexpr int kI8WeightWaves = 8;

template <typename T>
__global__ __launch_bounds__(64 * kI8WeightWaves) void i8_quantize_weight_kernel(
    const T *__restrict__ w, u32x4 *__restrict__ codes, float *__restrict__ scales, int Kd, int N,
    int panels, int NT, int KS)
{
    __shared__ uint32_t s_top[kI8WeightWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int col = blockIdx.x * 64 + (lane & 31) * 2; // of the panel
    const int e = blockIdx.y / panels, panel = blockIdx.y % panels;
    const int pc = N / panels; // a multiple of 8: both columns are in or out
    const bool in = col < pc;
    const T *base = w + (int64_t)e * Kd * N + (int64_t)panel * pc + (in ? col : 0);
    uint32_t top[2] = {0u, 0u};
    for (int ks = wave; ks < KS; ks += kI8WeightWaves) {
        const int k0 = ks * 32 + half * 16;
        if (in) {
            I8Pair<T> x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) // past the end: the last row again
                x[i] = *reinterpret_cast<const I8Pair<T> *>(base + (int64_t)min(k0 + i, Kd - 1) * N);
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    top[c] = max(top[c], i8_abs_bits(to_f32<T>(x[i].v[c])));
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        top[c] = max(top[c], (uint32_t)__shfl_xor((int)top[c], 32, 64));
        if (half == 0)
            s_top[wave][(lane & 31) * 2 + c] = top[c];
    }
    __syncthreads();
    I8Scale s[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < kI8WeightWaves; ++v)
            m = max(m, s_top[v][(lane & 31) * 2 + c]);
        s[c] = i8_scale(m);
    }
    const int tile = col >> 5;
    if (tile >= NT)
        return;
    const int64_t t = (int64_t)blockIdx.y * NT + tile;
    const int place = half * 32 + (col & 31); // lane of the packed layout
    if (wave == 0 && half == 0) {
        scales[t * 32 + (col & 31)] = in ? s[0].scale : 0.f;
        scales[t * 32 + (col & 31) + 1] = in ? s[1].scale : 0.f;
    }
    for (int ks = wave; ks < KS; ks += kI8WeightWaves) {
        const int k0 = ks * 32 + half * 16;
        I8Pair<T> x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = *reinterpret_cast<const I8Pair<T> *>(base + (int64_t)min(k0 + i, Kd - 1) * N);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 out;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                int v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = in && k0 + 4 * q + i < Kd ? i8_code(to_f32<T>(x[4 * q + i].v[c]), s[c]) : 0;
                out[q] = i8_pack4(v[0], v[1], v[2], v[3]);
            }
            codes[(t * KS + ks) * 64 + place + c] = out;
        }
    }
}

// Weights in int8 already: the same places, one pass.
__global__ __launch_bounds__(64 * kI8WeightWaves) void i8_pack_weight_kernel(
    const int8_t *__restrict__ w, const float *__restrict__ w_scales, u32x4 *__restrict__ codes,
    float *__restrict__ scales, int Kd, int N, int panels, int NT, int KS)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int col = blockIdx.x * 64 + (lane & 31) * 2;
    const int e = blockIdx.y / panels, panel = blockIdx.y % panels;
    const int pc = N / panels;
    const bool in = col < pc;
    const int tile = col >> 5;
    if (tile >= NT)
        return;
    const int8_t *base = w + (int64_t)e * Kd * N + (int64_t)panel * pc + (in ? col : 0);
    const int64_t t = (int64_t)blockIdx.y * NT + tile;
    const int place = half * 32 + (col & 31);
    if (wave == 0 && half == 0) {
        const float *ws = w_scales + (int64_t)e * N + (int64_t)panel * pc + (in ? col : 0);
        scales[t * 32 + (col & 31)] = in ? ws[0] : 0.f;
        scales[t * 32 + (col & 31) + 1] = in ? ws[1] : 0.f;
    }
    for (int ks = wave; ks < KS; ks += kI8WeightWaves) {
        const int k0 = ks * 32 + half * 16;
        uint16_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = in && k0 + i < Kd
                       ? *reinterpret_cast<const uint16_t *>(base + (int64_t)(k0 + i) * N)
                       : (uint16_t)0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 out;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                out[q] = i8_pack4(x[4 * q] >> 8 * c, x[4 * q + 1] >> 8 * c, x[4 * q + 2] >> 8 * c,
                                  x[4 * q + 3] >> 8 * c);
            codes[(t * KS + ks) * 64 + place + c] = out;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(64 * kI8WeightWaves) void i8_dequantize_weight_kernel(
    const u32x4 *__restrict__ codes, const float *__restrict__ scales, T *__restrict__ w, int Kd,
    int N, int panels, int NT, int KS)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int col = blockIdx.x * 64 + (lane & 31) * 2;
    const int e = blockIdx.y / panels, panel = blockIdx.y % panels;
    const int pc = N / panels;
    if (col >= pc)
        return;
    T *base = w + (int64_t)e * Kd * N + (int64_t)panel * pc + col;
    const int64_t t = (int64_t)blockIdx.y * NT + (col >> 5);
    const int place = half * 32 + (col & 31);
    const float x[2] = {scales[t * 32 + (col & 31)], scales[t * 32 + (col & 31) + 1]};
    for (int ks = blockIdx.z * kI8WeightWaves + wave; ks < KS; ks += gridDim.z * kI8WeightWaves) {
        const int k0 = ks * 32 + half * 16;
        const u32x4 c0 = codes[(t * KS + ks) * 64 + place], c1 = codes[(t * KS + ks) * 64 + place + 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            I8Pair<T> o;
            o.v[0] = from_f32<T>((float)(int8_t)(c0[i / 4] >> (8 * (i % 4))) * x[0]);
            o.v[1] = from_f32<T>((float)(int8_t)(c1[i / 4] >> (8 * (i % 4))) * x[1]);
            if (k0 + i < Kd)
                *reinterpret_cast<I8Pair<T> *>(base + (int64_t)(k0 + i) * N) = o;
        }
    }
}

// Token rows.  W waves a row: one for rows that it covers in few steps or where there
// are many rows, else the whole workgroup, whose waves then exchange their maxima.
template <typename T> struct I8Eight {
    u32x4 v[sizeof(T) / 2]; // eight values
};
template <typename T, int W>
__global__ __launch_bounds__(256) void i8_quantize_rows_kernel(const T *__restrict__ x, int64_t stride,
                                                               uint8_t *__restrict__ codes,
                                                               float *__restrict__ scales, int64_t M,
                                                               int Kd, int row_bytes)
{
    __shared__ uint32_t s_top[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int me = W == 4 ? threadIdx.x : lane;
    for (int64_t m = W == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave; m < M;
         m += (int64_t)gridDim.x * (4 / W)) {
        const T *row = x + m * stride;
        uint32_t top = 0;
        for (int k = me * 8; k < Kd; k += 64 * W * 8) { // Kd is a multiple of 8
            const I8Eight<T> e = *reinterpret_cast<const I8Eight<T> *>(row + k);
            const T *v = reinterpret_cast<const T *>(&e);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, i8_abs_bits(to_f32<T>(v[i])));
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
        if constexpr (W == 4) {
            __syncthreads(); // the last row's maxima are read
            if (lane == 0)
                s_top[wave] = top;
            __syncthreads();
            top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
        }
        const I8Scale s = i8_scale(top);
        if (me == 0)
            scales[m] = s.scale;
        uint8_t *out = codes + m * row_bytes;
        for (int k = me * 8; k < row_bytes; k += 64 * W * 8) {
            u32x2 c = {0u, 0u};
            if (k < Kd) {
                const I8Eight<T> e = *reinterpret_cast<const I8Eight<T> *>(row + k);
                const T *v = reinterpret_cast<const T *>(&e);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    c[h] = i8_pack4(i8_code(to_f32<T>(v[4 * h]), s), i8_code(to_f32<T>(v[4 * h + 1]), s),
                                    i8_code(to_f32<T>(v[4 * h + 2]), s),
                                    i8_code(to_f32<T>(v[4 * h + 3]), s));
            }
            *reinterpret_cast<u32x2 *>(out + k) = c;
        }
    }
}

static dim3 weight_grid(const I8Dims &d, int64_t E, int panels)
{
    // E * panels <= 2048; Kd >= 8 and Kd * N < 2^31 keep x within 2^22
    return dim3((unsigned)((d.NT + 1) / 2), (unsigned)(E * panels));
}

hipError_t launch_i8_quantize_weight(int dtype, const void *w, void *codes, float *scales, int64_t E,
                                     int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    const dim3 grid = weight_grid(d, E, panels), block(64 * kI8WeightWaves);
    u32x4 *c = static_cast<u32x4 *>(codes);
    if (dtype == 1)
        hipLaunchKernelGGL(i8_quantize_weight_kernel<bf16>, grid, block, 0, s,
                           static_cast<const bf16 *>(w), c, scales, (int)Kd, (int)N, panels, d.NT, d.KS);
    else
        hipLaunchKernelGGL(i8_quantize_weight_kernel<float>, grid, block, 0, s,
                           static_cast<const float *>(w), c, scales, (int)Kd, (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

hipError_t launch_i8_pack_weight(const void *w, const float *w_scales, void *codes, float *scales,
                                 int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    hipLaunchKernelGGL(i8_pack_weight_kernel, weight_grid(d, E, panels), dim3(64 * kI8WeightWaves), 0,
                       s, static_cast<const int8_t *>(w), w_scales, static_cast<u32x4 *>(codes), scales,
                       (int)Kd, (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

hipError_t launch_i8_dequantize_weight(int dtype, const void *codes, const float *scales, void *w,
                                       int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    dim3 grid = weight_grid(d, E, panels);
    grid.z = (unsigned)((d.KS + 4 * kI8WeightWaves - 1) / (4 * kI8WeightWaves));
    const dim3 block(64 * kI8WeightWaves);
    const u32x4 *c = static_cast<const u32x4 *>(codes);
    if (dtype == 1)
        hipLaunchKernelGGL(i8_dequantize_weight_kernel<bf16>, grid, block, 0, s, c, scales,
                           static_cast<bf16 *>(w), (int)Kd, (int)N, panels, d.NT, d.KS);
    else
        hipLaunchKernelGGL(i8_dequantize_weight_kernel<float>, grid, block, 0, s, c, scales,
                           static_cast<float *>(w), (int)Kd, (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

template <typename T>
static hipError_t rows_t(const void *x, int64_t stride, void *codes, float *scales, int64_t M,
                         int64_t Kd, hipStream_t s)
{
    const I8Dims d(Kd, 8);
    const bool whole = Kd > 1024;
    const int64_t blocks = whole ? M : (M + 3) / 4;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    auto k = whole ? i8_quantize_rows_kernel<T, 4> : i8_quantize_rows_kernel<T, 1>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, s, static_cast<const T *>(x), stride,
                       static_cast<uint8_t *>(codes), scales, M, (int)Kd, (int)d.row());
    return hipGetLastError();
}

hipError_t launch_i8_quantize_rows(int dtype, const void *x, int64_t stride, void *codes,
                                   float *scales, int64_t M, int64_t Kd, hipStream_t s)
{
    if (M <= 0)
        return hipSuccess;
    return dtype == 1 ? rows_t<bf16>(x, stride, codes, scales, M, Kd, s)
                      : rows_t<float>(x, stride, codes, scales, M, Kd, s);
}

} // namespace moe
