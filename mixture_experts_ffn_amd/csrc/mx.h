// mx.h — block-scaled (microscaled) formats of the MXFP4 expert FFN: layouts
// and device helpers shared by the quantisation kernels and the GEMMs.
//
// A block is 32 consecutive values along the contraction axis with one shared
// power of two X = 2^(code - 127), kept as the 8-bit code (E8M0).  For the
// block's largest magnitude m the code is floor(log2 m) - 2 + 127, not below
// 0; each element is v / X rounded to nearest, ties to even, and saturated:
//   e2m1 (MXFP4): 0, .5, 1, 1.5, 2, 3, 4, 6
//   e2m3 (MXFP6): steps of 1/8 up to 2, 1/4 up to 4, 1/2 up to 7.5
// A block that holds a NaN or an infinity has code 255 (NaN): every product
// with it is NaN.  The rule, the formats and the NaN code are those of the OCP
// microscaling formats specification 1.0.
//
// Why e2m3 and not e4m3 for the finer activations: within a block whose
// largest element is scaled to [4, 8) both have three fraction bits where it
// matters; e2m3 moves a quarter fewer bytes and runs at the rate of e2m1
// (measured with registers only, random data: 6.3 PFLOP/s for e2m1 x e2m1,
// 5.5 for e2m1 x e2m3, 3.9 for e2m1 x e4m3); and every product of e2m1 and
// e2m3 is a multiple of 1/16 below 64, which the matrix unit adds up exactly,
// while sums with e4m3 products were off by up to 2^-11 of the largest one.
//
// One matrix instruction (32 x 32 x 64, scaled) covers a "k-step" of 64
// values, two blocks; lane l of either operand holds row l % 32 and k-block
// l / 32, k ascending from the lowest bits: 16 bytes of e2m1 or 24 of e2m3.
// The lane's scale code is one byte of a dword, selected by an immediate, so a
// dword carries four k-steps.
//
// Packed weights of a stack [E, Kd, N] whose columns form `panels` equal
// panels (up_proj: gate and up; down_proj: one), NT = ceil(N / panels / 32)
// column tiles each, KS = 2 ceil(Kd / 128) k-steps, KC = ceil(KS / 4) chunks:
//   codes  [E][panels][NT][KS][64 lanes][16 bytes]
//   scales [E][panels][NT][KC][64 lanes][4 k-steps]      (256-byte aligned)
// so that one wave's operand of a k-step is 1024 contiguous bytes, straight
// from memory into registers, and a column tile's whole contraction is one
// contiguous stream.  Columns and k past the ends are zero (an even number of
// k-steps: the tile kernel's loop takes them in pairs).
//
// Activations are row-major: the first 16 bytes of every block's codes
// [rows][2 KS][16], for e2m3 the other 8 in an array of their own
// [rows][2 KS][8] (both then load as whole vectors), and the scales
// [rows][KC rounded up to even][2 k-blocks][4 k-steps] (whole 16 bytes a row).
#pragma once

#include "common.h"
#include "kernels.h"

namespace moe {

constexpr int kMxNan = 255;  // E8M0 code of NaN

struct MxDims {
    int NT, KS, KC;
    MxDims() = default;
    __host__ __device__ MxDims(int64_t Kd, int64_t panel_cols)
        : NT((int)((panel_cols + 31) / 32)), KS((int)((Kd + 127) / 128) * 2), KC((KS + 3) / 4)
    {
    }
    // bytes of an activation row: first 16 and last 8 bytes of the blocks, scales
    __host__ __device__ int code_row() const { return KS * 32; }
    __host__ __device__ int tail_row(int bits) const { return bits == 6 ? KS * 16 : 0; }
    __host__ __device__ int scale_row() const { return (KC + 1) / 2 * 16; }
};

// place of k-block b's scale byte in an activation row's scales
__host__ __device__ inline int mx_scale_at(int b)
{
    const int ks = b >> 1;
    return (ks >> 2) * 8 + (b & 1) * 4 + (ks & 3);
}

// Scale code of a block from the bits of its largest magnitude (the integer
// maximum of |v|'s bits: NaN > inf > every number, so non-finite values win).
__device__ inline int mx_scale_code(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 2;
    return amax_bits >= 0x7f800000u ? kMxNan : e > 0 ? e : 0;
}
// 1 / X: 2^(127 - code), exact and normal for every code a finite fp32 block
// can have (at most 252); zero for the NaN code
__device__ inline float mx_inverse(int code)
{
    return code == kMxNan ? 0.f : __uint_as_float((uint32_t)(254 - code) << 23);
}
__device__ inline float mx_scale_value(int code)
{
    // 2^(code - 127); code 0 is the fp32 subnormal 2^-127
    return code == kMxNan ? __uint_as_float(0x7fc00000u)
                          : __uint_as_float(code ? (uint32_t)code << 23 : 0x00400000u);
}
__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));

// eight already scaled values -> eight e2m1 codes, value 0 in the low nibble
// (the conversion rounds to nearest even and saturates at 6)
__device__ inline uint32_t mx_pack8_fp4(const float *v)
{
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
    return r;
}
// N (16 or 32) scaled values -> e2m3 codes, value 0 in the lowest bits: the
// first N 6 / 32 dwords.  The conversion takes two vectors and interleaves
// them; it rounds to nearest even and saturates at 7.5.
template <int N> __device__ inline u32x6 mx_pack_fp6(const float *v)
{
    f32x16 even, odd;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        even[i] = 2 * i < N ? v[2 * i] : 0.f;
        odd[i] = 2 * i < N ? v[2 * i + 1] : 0.f;
    }
    return __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(even, odd, 1.0f);
}

// value of an e2m1 code
__device__ inline float mx_fp4_value(uint32_t code)
{
    const int m = code & 7;
    // 0, .5, then (1 + (m & 1) / 2) 2^((m >> 1) - 1)
    const float a = m < 2 ? 0.5f * m
                          : __uint_as_float((uint32_t)(((m >> 1) + 126) << 23 | (m & 1) << 22));
    return code & 8 ? -a : a;
}

// Block i of the token rows (block i % (2 KS) of row i / (2 KS)): a lane owns
// it, so its maximum needs no other lane and its codes are whole vectors.  The
// row is padded with zeros to whole k-steps.
template <int BITS> __device__ inline void mx_quantize_block(const MxRows &r, int64_t i)
{
    const int64_t t = i / (2 * r.KS);
    const int b = (int)(i - t * (2 * r.KS));
    const bf16 *x = static_cast<const bf16 *>(r.x) + t * r.H + b * 32;
    float v[32];
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        u32x4 raw = {0u, 0u, 0u, 0u};
        if (b * 32 + q * 8 < r.H) // H is a multiple of 8
            raw = *reinterpret_cast<const u32x4 *>(x + q * 8);
        const bf16 *vv = reinterpret_cast<const bf16 *>(&raw);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[q * 8 + j] = static_cast<float>(vv[j]);
            top = max(top, abs_bits(v[q * 8 + j]));
        }
    }
    const int code = mx_scale_code(top);
    const float inv = mx_inverse(code);
#pragma unroll
    for (int j = 0; j < 32; ++j)
        v[j] *= inv;
    u32x4 *codes = static_cast<u32x4 *>(r.codes);
    if constexpr (BITS == 4) {
        codes[i] = u32x4{mx_pack8_fp4(v), mx_pack8_fp4(v + 8), mx_pack8_fp4(v + 16),
                         mx_pack8_fp4(v + 24)};
    } else {
        const u32x6 c = mx_pack_fp6<32>(v);
        codes[i] = u32x4{c[0], c[1], c[2], c[3]};
        static_cast<u32x2 *>(r.tails)[i] = u32x2{c[4], c[5]};
    }
    static_cast<uint8_t *>(r.scales)[t * r.srow + mx_scale_at(b)] = (uint8_t)code;
}

} // namespace moe
