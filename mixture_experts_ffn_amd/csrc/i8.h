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

// Scale and codes of a vector from the bits of its largest magnitude (as integers
// they order as the values do, infinities and NaN above all numbers).
struct I8Scale {
    float scale, inverse;
    bool exact; // every quotient by division in 64 bits
};
__device__ inline I8Scale i8_scale(uint32_t top)
{
    I8Scale s;
    if (top >= 0x7f800000u) { // NaN or infinity: the scale says it, the codes are 0
        s.scale = __uint_as_float(0x7fc00000u);
        s.inverse = 0.f;
        s.exact = false;
        return s;
    }
    s.scale = (float)((double)__uint_as_float(top) / 127.0);
    // the reciprocal of a scale below 2^-126 overflows or has lost bits, of one near
    // 2^126 is subnormal
    s.exact = s.scale < 0x1p-100f || s.scale > 0x1p100f;
    s.inverse = s.scale > 0.f ? 1.0f / s.scale : 0.f;
    if (s.scale == 0.f)
        s.exact = false;
    return s;
}

// The code of v.  v * inverse is within 2^-23 of v / scale, relatively (the
// reciprocal's and the product's rounding), 1.6e-5 at 127: a quotient that lies
// within 4e-5 of the middle of two codes is formed again in 64 bits, where a middle
// is told from its neighbours (v and scale are fp32, so that a quotient beside a
// middle is 2^-32 away at least).
__device__ inline int i8_code(float v, const I8Scale &s)
{
    float t = v * s.inverse;
    float r = rintf(t);
    if (s.exact || fabsf(t - r) > 0.49996f)
        r = s.inverse == 0.f ? 0.f : (float)rint((double)v / (double)s.scale);
    // a NaN or an infinity among v: codes 0
    return s.inverse == 0.f ? 0 : (int)fminf(fmaxf(r, -127.f), 127.f);
}

__device__ inline uint32_t i8_pack4(int a, int b, int c, int d)
{
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 |
           (uint32_t)d << 24;
}

} // namespace moe
