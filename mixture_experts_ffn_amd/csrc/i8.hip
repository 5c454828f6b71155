// i8.hip — int8 quantisation of weights by column and of token rows, and the
// packed weights' inverse (layouts: i8.h).
//
// A vector's codes need its largest magnitude first: a workgroup or a wave holds its
// vectors in registers between the two, where they fit.  Bound by HBM: a weight of n
// values moves 2n (or 4n) + n bytes, a row of Kd 2 Kd (or 4 Kd) + Kd.
#include "i8.h"
#include "kernels.h"

namespace moe {

// Place of a lane among a weight's values: a workgroup owns 64 columns of a panel, its
// waves share out the pairs of k-steps (64 rows), and a lane has four neighbouring
// columns of 16 rows, which are 16 codes of each column's lane in the packed layout.
// A load takes 128 bytes of a row in bf16, 256 in fp32, of four rows at once.
struct I8Place {
    int e, panel, col, tile; // col: the first of four, of the panel
    bool in;                 // a panel's columns are a multiple of 8: four are in or out
    int rows;                // 16 * the lane's quarter of the 64 rows
    int lane;                // of the packed layout, of the first column
};
__device__ inline I8Place i8_place(int N, int panels)
{
    const int l = threadIdx.x & 63;
    I8Place q;
    q.e = blockIdx.y / panels;
    q.panel = blockIdx.y - q.e * panels;
    q.col = blockIdx.x * 64 + (l & 15) * 4;
    q.tile = q.col >> 5;
    q.in = q.col < N / panels;
    q.rows = l >> 4 << 4;
    q.lane = (q.rows & 16) * 2 + (q.col & 31);
    return q;
}
// u32x4 of the packed codes for the lane's first column in pair p
__device__ inline int64_t i8_packed_at(const I8Place &q, int NT, int KS, int p)
{
    return (((int64_t)blockIdx.y * NT + q.tile) * KS + 2 * p + (q.rows >> 5)) * 64 + q.lane;
}

template <typename T> struct __attribute__((aligned(4 * sizeof(T)))) I8Four {
    T v[4];
};
// The largest magnitudes of a lane's four columns.
template <typename T> struct I8Tops;
template <> struct I8Tops<float> {
    I8Top<float> t[4];
    __device__ void add(const I8Four<float> &x)
    {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            t[c].add(x.v[c]);
    }
    __device__ uint32_t bits(int c) const { return t[c].bits(); }
};
template <> struct I8Tops<bf16> {
    I8Top2 t[2];
    __device__ void add(const I8Four<bf16> &x)
    {
        const u32x2 d = __builtin_bit_cast(u32x2, x);
        t[0].add(d[0]);
        t[1].add(d[1]);
    }
    __device__ uint32_t bits(int c) const { return t[c >> 1].bits(c & 1); }
};
template <typename T> struct I8Step { // a lane's 16 rows of four columns
    I8Four<T> x[16];
};
template <typename T>
__device__ inline void i8_load_step(const T *base, int k0, int Kd, int N, I8Step<T> &d)
{
    const T *p = base + (int64_t)k0 * N;
    if (k0 + 16 <= Kd) {
#pragma unroll
        for (int i = 0; i < 16; ++i, p += N)
            d.x[i] = *reinterpret_cast<const I8Four<T> *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i, p += N) {
            d.x[i] = I8Four<T>{};
            if (k0 + i < Kd)
                d.x[i] = *reinterpret_cast<const I8Four<T> *>(p);
        }
    }
}

// Weights.  HELD pairs of k-steps a wave stay in registers between the maximum and
// the codes (Kd up to 2048 in bf16, 1024 in fp32, which fill half the CU's
// registers); 0: longer columns, read twice.  [64, 2048, 2816] bf16, 1.1 GB of
// traffic: 281 us held by eight waves of four pairs, 294 by sixteen of two, 333 read
// twice (a large copy of as many bytes: 224); [16, 1024, 4096] fp32 83; read twice
// [32, 7168, 4096] bf16 1110.
template <typename T, int WAVES, int HELD>
__global__ __launch_bounds__(64 * WAVES) void i8_quantize_weight_kernel(
    const T *__restrict__ w, u32x4 *__restrict__ codes, float *__restrict__ scales, int Kd, int N,
    int panels, int NT, int KS)
{
    __shared__ uint32_t s_top[WAVES][64];
    const int wave = threadIdx.x >> 6, c0 = (threadIdx.x & 15) * 4, KP = KS >> 1;
    const I8Place q = i8_place(N, panels);
    // columns past the panel's end read its first ones
    const T *base = w + (int64_t)q.e * Kd * N + (int64_t)q.panel * (N / panels) + (q.in ? q.col : 0);
    I8Tops<T> tops;
    I8Step<T> held[HELD ? HELD : 1];
    auto maximum = [&](const I8Step<T> &d) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            tops.add(d.x[i]);
    };
    if constexpr (HELD > 0) {
#pragma unroll
        for (int s = 0; s < HELD; ++s) // past the end: zeros
            i8_load_step(base, (s * WAVES + wave) * 64 + q.rows, Kd, N, held[s]);
#pragma unroll
        for (int s = 0; s < HELD; ++s)
            maximum(held[s]);
    } else {
        for (int p = wave; p < KP; p += WAVES) {
            i8_load_step(base, p * 64 + q.rows, Kd, N, held[0]);
            maximum(held[0]);
        }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t top = tops.bits(c);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        if (q.rows == 0)
            s_top[wave][c0 + c] = top;
    }
    __syncthreads();
    if (q.tile >= NT)
        return;
    I8Scale s[4];
    float *const ts = scales + ((int64_t)blockIdx.y * NT + q.tile) * 32 + (q.col & 31);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < WAVES; ++v)
            m = max(m, s_top[v][c0 + c]);
        s[c] = i8_scale<T>(m);
        if (wave == 0 && q.rows == 0)
            ts[c] = q.in ? s[c].scale : 0.f;
    }
    auto store = [&](int p, const I8Step<T> &d) {
        u32x4 *const out = codes + i8_packed_at(q, NT, KS, p);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = to_f32<T>(d.x[i].v[c]);
            u32x4 o;
            i8_codes<T, 16>(v, s[c], reinterpret_cast<uint32_t *>(&o));
            out[c] = q.in ? o : u32x4{0u, 0u, 0u, 0u};
        }
    };
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (i * WAVES + wave < KP)
                store(i * WAVES + wave, held[i]);
    } else {
        for (int p = wave; p < KP; p += WAVES) {
            i8_load_step(base, p * 64 + q.rows, Kd, N, held[0]);
            store(p, held[0]);
        }
    }
}

// Weights in int8 already: the same places, one pass.
constexpr int kI8Waves = 8;
__global__ __launch_bounds__(64 * kI8Waves) void i8_pack_weight_kernel(
    const int8_t *__restrict__ w, const float *__restrict__ w_scales, u32x4 *__restrict__ codes,
    float *__restrict__ scales, int Kd, int N, int panels, int NT, int KS)
{
    const int wave = threadIdx.x >> 6;
    const I8Place q = i8_place(N, panels);
    if (q.tile >= NT)
        return;
    const int64_t at = (int64_t)q.panel * (N / panels) + (q.in ? q.col : 0);
    const int8_t *base = w + (int64_t)q.e * Kd * N + at;
    if (wave == 0 && blockIdx.z == 0 && q.rows == 0) {
        const float *ws = w_scales + (int64_t)q.e * N + at;
        float *const ts = scales + ((int64_t)blockIdx.y * NT + q.tile) * 32 + (q.col & 31);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            ts[c] = q.in ? ws[c] : 0.f;
    }
    for (int p = blockIdx.z * kI8Waves + wave; p < KS >> 1; p += gridDim.z * kI8Waves) {
        const int k0 = p * 64 + q.rows;
        uint32_t x[16]; // four columns of a row
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = q.in && k0 + i < Kd
                       ? *reinterpret_cast<const uint32_t *>(base + (int64_t)(k0 + i) * N)
                       : 0u;
        u32x4 *const out = codes + i8_packed_at(q, NT, KS, p);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u32x4 o;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                o[r] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    o[r] |= (x[4 * r + b] >> (8 * c) & 255u) << (8 * b);
            }
            out[c] = o;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(64 * kI8Waves) void i8_dequantize_weight_kernel(
    const u32x4 *__restrict__ codes, const float *__restrict__ scales, T *__restrict__ w, int Kd,
    int N, int panels, int NT, int KS)
{
    const int wave = threadIdx.x >> 6;
    const I8Place q = i8_place(N, panels);
    if (!q.in)
        return;
    T *base = w + (int64_t)q.e * Kd * N + (int64_t)q.panel * (N / panels) + q.col;
    const f32x4 x = *reinterpret_cast<const f32x4 *>(
        scales + ((int64_t)blockIdx.y * NT + q.tile) * 32 + (q.col & 31));
    for (int p = blockIdx.z * kI8Waves + wave; p < KS >> 1; p += gridDim.z * kI8Waves) {
        const int k0 = p * 64 + q.rows;
        const u32x4 *const in = codes + i8_packed_at(q, NT, KS, p);
        u32x4 code[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            code[c] = in[c];
        T *row = base + (int64_t)k0 * N;
#pragma unroll
        for (int i = 0; i < 16; ++i, row += N) {
            I8Four<T> o;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                o.v[c] = from_f32<T>((float)(int8_t)(code[c][i / 4] >> (8 * (i % 4))) * x[c]);
            if (k0 + i < Kd)
                *reinterpret_cast<I8Four<T> *>(row) = o;
        }
    }
}

template <typename T, int W, int HELD>
__global__ __launch_bounds__(256) void i8_quantize_rows_kernel(const T *__restrict__ x, int64_t stride,
                                                               uint8_t *__restrict__ codes,
                                                               float *__restrict__ scales, int64_t M,
                                                               int Kd, int row_bytes)
{
    i8_quantize_rows<T, W, HELD, 4>(x, stride, codes, scales, M, Kd, row_bytes, blockIdx.x, gridDim.x);
}

static dim3 weight_grid(const I8Dims &d, int64_t E, int panels)
{
    // E * panels <= 2048; Kd >= 8 and Kd * N < 2^31 keep x within 2^22
    return dim3((unsigned)((d.NT + 1) / 2), (unsigned)(E * panels));
}

template <typename T, int WAVES, int HELD>
static hipError_t quantize_weight_t(const void *w, void *codes, float *scales, int64_t E, int64_t Kd,
                                    int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    hipLaunchKernelGGL((i8_quantize_weight_kernel<T, WAVES, HELD>), weight_grid(d, E, panels),
                       dim3(64 * WAVES), 0, s, static_cast<const T *>(w), static_cast<u32x4 *>(codes),
                       scales, (int)Kd, (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

hipError_t launch_i8_quantize_weight(int dtype, const void *w, void *codes, float *scales, int64_t E,
                                     int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const int pairs = I8Dims(Kd, 8).KS / 2;
    auto k = dtype == 1 ? (pairs <= 4    ? quantize_weight_t<bf16, 4, 1>
                           : pairs <= 8  ? quantize_weight_t<bf16, 8, 1>
                           : pairs <= 16 ? quantize_weight_t<bf16, 8, 2>
                           : pairs <= 32 ? quantize_weight_t<bf16, 8, 4>
                                         : quantize_weight_t<bf16, 8, 0>)
                        : (pairs <= 4    ? quantize_weight_t<float, 4, 1>
                           : pairs <= 8  ? quantize_weight_t<float, 8, 1>
                           : pairs <= 16 ? quantize_weight_t<float, 16, 1>
                                         : quantize_weight_t<float, 8, 0>);
    return k(w, codes, scales, E, Kd, N, panels, s);
}

// with the pairs of k-steps spread over z, four a wave
static dim3 spread_grid(const I8Dims &d, int64_t E, int panels)
{
    dim3 grid = weight_grid(d, E, panels);
    grid.z = (unsigned)((d.KS / 2 + 4 * kI8Waves - 1) / (4 * kI8Waves));
    return grid;
}

hipError_t launch_i8_pack_weight(const void *w, const float *w_scales, void *codes, float *scales,
                                 int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    hipLaunchKernelGGL(i8_pack_weight_kernel, spread_grid(d, E, panels), dim3(64 * kI8Waves), 0, s,
                       static_cast<const int8_t *>(w), w_scales, static_cast<u32x4 *>(codes), scales,
                       (int)Kd, (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

template <typename T>
static hipError_t dequantize_weight_t(const void *codes, const float *scales, void *w, int64_t E,
                                      int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    const I8Dims d(Kd, N / panels);
    hipLaunchKernelGGL(i8_dequantize_weight_kernel<T>, spread_grid(d, E, panels), dim3(64 * kI8Waves),
                       0, s, static_cast<const u32x4 *>(codes), scales, static_cast<T *>(w), (int)Kd,
                       (int)N, panels, d.NT, d.KS);
    return hipGetLastError();
}

hipError_t launch_i8_dequantize_weight(int dtype, const void *codes, const float *scales, void *w,
                                       int64_t E, int64_t Kd, int64_t N, int panels, hipStream_t s)
{
    return dtype == 1 ? dequantize_weight_t<bf16>(codes, scales, w, E, Kd, N, panels, s)
                      : dequantize_weight_t<float>(codes, scales, w, E, Kd, N, panels, s);
}

template <typename T, int W> static auto rows_kernel(int steps)
{
    return steps <= 1   ? i8_quantize_rows_kernel<T, W, 1>
           : steps <= 2 ? i8_quantize_rows_kernel<T, W, 2>
           : steps <= 4 ? i8_quantize_rows_kernel<T, W, 4>
           : steps <= 8 ? i8_quantize_rows_kernel<T, W, 8>
                        : i8_quantize_rows_kernel<T, W, 0>;
}

template <typename T>
static hipError_t rows_t(const void *x, int64_t stride, void *codes, float *scales, int64_t M,
                         int64_t Kd, hipStream_t s)
{
    const I8Dims d(Kd, 8);
    const bool one = Kd <= 512 || (M >= 4096 && Kd <= 4096);
    const int64_t blocks = one ? (M + 3) / 4 : M;
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    auto k = one ? rows_kernel<T, 1>((int)((d.row() + 511) / 512))
                 : rows_kernel<T, 4>((int)((d.row() + 2047) / 2048));
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
