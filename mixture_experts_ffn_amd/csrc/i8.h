// i8.h — 8-bit integers with one scale a vector: layouts and device helpers
// shared by the quantisation kernels and the GEMMs.
//
// A vector v (a token's row, a weight's column) has scale s = max|v| / 127 rounded
// to fp32 and codes v / s rounded to nearest, ties to even, held to [-127, 127]
// (where s is so small that it lost bits, a quotient may lie above 127).
//
// One matrix instruction (32 x 32 x 32) covers a "k-step" of 32 values: lane l of
// either operand holds row l % 32 and k = 16 (l / 32) + [0, 16), 16 bytes.  k-steps
// come in pairs, 64 bytes of a token's row, so Kd is rounded up to 64 with codes 0.
//
// Packed weights [E][panel][column tile of 32][k-step][lane][16 bytes]: a k-step of
// a tile is 1024 consecutive bytes in the operand's own lane order.  Then the
// scales, fp32 [E][panel][32 per tile], zero past the panel's last column.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

struct I8Dims {
    int NT, KS; // column tiles of a panel, k-steps
    __host__ __device__ I8Dims(int64_t Kd, int64_t panel_cols)
        : NT((int)((panel_cols + 31) / 32)), KS((int)((Kd + 63) / 64 * 2))
    {
    }
    __host__ __device__ int64_t row() const { return (int64_t)KS * 32; } // bytes of a token's codes
};

__device__ inline uint32_t i8_abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The largest magnitude of a vector's values, as the bits of an fp32 number (as
// integers they order as the values do, infinities and NaN above all numbers).  bf16
// values two at a time.
template <typename T> struct I8Top;
template <> struct I8Top<float> {
    uint32_t t = 0;
    __device__ void add(float v) { t = max(t, i8_abs_bits(v)); }
    __device__ uint32_t bits() const { return t; }
};
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
struct I8Top2 { // of either half of dwords
    u16x2 t = {0, 0};
    __device__ void add(uint32_t v)
    {
        t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, v & 0x7fff7fffu));
    }
    __device__ uint32_t bits(int half) const { return (uint32_t)t[half] << 16; }
    __device__ uint32_t bits() const { return max(bits(0), bits(1)); }
};

// Scale and codes of a vector with the largest magnitude `top`.
struct I8Scale {
    float scale, inverse;
    float quick; // bf16: the factor of codes without a further look
    bool exact;  // every quotient by division in 64 bits
    bool ties;   // bf16: many quotients lie in the middle of two codes
};
template <typename T> __device__ inline I8Scale i8_scale(uint32_t top)
{
    I8Scale s{__uint_as_float(0x7fc00000u), 0.f, 0.f, false, false};
    if (top >= 0x7f800000u) // NaN or infinity: the scale says it, the codes are 0
        return s;
    const float largest = __uint_as_float(top);
    s.scale = largest / 127.0f;
    if (s.scale == 0.f)
        return s;
    // the reciprocal of a scale below 2^-126 overflows or has lost bits, of one near
    // 2^126 is subnormal
    s.exact = s.scale < 0x1p-100f || s.scale > 0x1p100f;
    s.inverse = 1.0f / s.scale;
    if constexpr (sizeof(T) == 2) {
        // v and largest have 8 bits: 254 v / largest is an odd integer (or within
        // 2^-23 of one, scale being rounded) only for v = largest / 2, whose side of
        // 63.5 the factor is moved to, and, among others, where largest is 127 times a
        // power of two; else it is 1 / 255 away, so that 2^-20 of error do no harm
        const float rest = fmaf(-63.5f, s.scale, 0.5f * largest); // exact (see i8_codes)
        s.quick = s.inverse * (rest >= 0.f ? 1.f + 0x1p-21f : 1.f - 0x1p-21f);
        s.ties = (top >> 16 & 0x7fu) == 0x7eu;
    }
    return s;
}

// Codes of N values (a multiple of 4), packed four to a dword, of a vector of T.  Each is
// made as code + 128 in its byte (rounded to nearest even by the conversion).
//
// t = v * inverse is within 2^-23 of v / scale, relatively (the reciprocal's and the
// product's rounding), so it never rounds past 127.  Where some quotient may lie on the
// other side of the middle of two codes than t, or on it, all N are compared with it
// by their rest e = v - code * scale, one multiply-add: where it decides, e is a
// multiple of half a unit in scale's last place, below 2^24 of them, so exact.  Of a
// vector with a NaN or an infinity (or of zeros) all codes are 0.
template <typename T, int N>
__device__ inline void i8_codes(const float *v, const I8Scale &s, uint32_t *out)
{
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            uint32_t u = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                u = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(v[4 * i + b], s.quick, 128.f), b, u);
            out[i] = s.quick == 0.f ? 0u : u ^ 0x80808080u;
        }
        if (!(s.exact || s.ties))
            return;
    }
    float r[N], near = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t = v[i] * s.inverse;
        r[i] = rintf(t);
        near = fmaxf(near, fabsf(t - r[i]));
    }
    if (s.exact) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            r[i] = fminf(fmaxf((float)rint((double)v[i] / (double)s.scale), -127.f), 127.f);
    } else if (near > 0.49998f) { // 127 * 2^-23 is 1.6e-5
        const float half = 0.5f * s.scale;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float e = fmaf(-r[i], s.scale, v[i]), a = fabsf(e);
            if (a > half || (a == half && ((int)r[i] & 1)))
                r[i] += copysignf(1.f, e);
        }
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        uint32_t u = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
            u = __builtin_amdgcn_cvt_pk_u8_f32(r[4 * i + b] + 128.f, b, u);
        out[i] = s.inverse == 0.f ? 0u : u ^ 0x80808080u;
    }
}

// Token rows by workgroups of WAVES waves, of which this is number `block` of `blocks`.
// W waves a row: one where there are many rows, or rows that it covers in one step,
// else four, which then exchange their maxima.  Rows of up to HELD steps (of 512 W
// values) stay in registers between the maximum and the codes; 0: longer ones, read
// twice.  24576 x 1408 bf16 18 us (5.7 TB/s), 8192 x 7168 28 (6.3), 65536 x 2048 fp32 129
// (5.2).
template <typename T> struct I8Eight {
    u32x4 v[sizeof(T) / 2]; // eight values
};
template <typename T, int W, int HELD, int WAVES>
__device__ inline void i8_quantize_rows(const T *x, int64_t stride, uint8_t *codes, float *scales,
                                        int64_t M, int Kd, int row_bytes, int64_t block,
                                        int64_t blocks)
{
    __shared__ uint32_t s_top[WAVES];
    constexpr int G = WAVES / W; // rows at a time
    constexpr int STEP = 512 * W;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, group = wave / W;
    const int me = ((wave - group * W) * 64 + lane) * 8; // Kd is a multiple of 8
    for (int64_t base = block * G; base < M; base += blocks * G) {
        const int64_t m = base + group < M ? base + group : M - 1; // the last row, again
        const T *row = x + m * stride;
        I8Eight<T> held[HELD ? HELD : 1];
        auto load = [&](int k, I8Eight<T> &d) {
            d = I8Eight<T>{};
            if (k < Kd)
                d = *reinterpret_cast<const I8Eight<T> *>(row + k);
        };
        std::conditional_t<sizeof(T) == 2, I8Top2, I8Top<float>> tops;
        auto maximum = [&](const I8Eight<T> &d) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) * 2; ++i)
                if constexpr (sizeof(T) == 2)
                    tops.add(d.v[0][i]);
                else
                    tops.add(__uint_as_float(d.v[i >> 2][i & 3]));
        };
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                load(me + i * STEP, held[i]);
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                maximum(held[i]);
        } else {
            for (int k = me; k < Kd; k += STEP) {
                load(k, held[0]);
                maximum(held[0]);
            }
        }
        uint32_t top = tops.bits();
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1)
            top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
        if constexpr (W > 1) {
            __syncthreads(); // the last rows' maxima are read
            if (lane == 0)
                s_top[wave] = top;
            __syncthreads();
            top = s_top[group * W];
#pragma unroll
            for (int w = 1; w < W; ++w)
                top = max(top, s_top[group * W + w]);
        }
        const I8Scale s = i8_scale<T>(top);
        if (me == 0)
            scales[m] = s.scale;
        uint8_t *out = codes + m * row_bytes;
        auto store = [&](int k, const I8Eight<T> &d) {
            const T *p = reinterpret_cast<const T *>(&d);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = to_f32<T>(p[i]); // zeros behind Kd
            u32x2 c;
            i8_codes<T, 8>(v, s, reinterpret_cast<uint32_t *>(&c));
            if (k < row_bytes)
                *reinterpret_cast<u32x2 *>(out + k) = c;
        };
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                store(me + i * STEP, held[i]);
        } else {
            for (int k = me; k < row_bytes; k += STEP) {
                load(k, held[0]);
                store(k, held[0]);
            }
        }
    }
}

} // namespace moe
