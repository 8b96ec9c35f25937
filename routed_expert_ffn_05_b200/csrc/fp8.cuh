// FP8 matrices with one fp32 scale per block of 128: the block rule shared by
// the quantiser, the norm and the shared expert's hidden row.
//
// A block (128 consecutive elements of an activation row, or 128 x 128 of a
// weight matrix) with largest magnitude amax stores
//     m = max(amax, 2^-100),  scale = m / 448,  code = E4M3(v * r), r = 448 / m
// (E4M3 rounding to nearest even, saturating); with power-of-two scales, scale
// is the least power of two not below m / 448 and r = 1 / scale (exact). Every
// quotient and product is one fp32 operation rounded to nearest. The floor
// keeps r finite; values a hundred binades below one quantise to zero codes.
// amax is taken over the magnitudes' bit patterns as integers, so a NaN is
// larger than every number: it makes its block's scale NaN and its codes NaN
// (0x7F), and an infinity makes them Inf and (for finite values) zero.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;

struct BlockScale {
    float scale, r;
};

// From the bit pattern of amax (sign cleared).
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, bool pow2) {
    constexpr uint32_t kFloor = 27u << 23;  // 2^-100
    const float m = __uint_as_float(max(amax_bits, kFloor));
    BlockScale b;
    b.scale = __fdiv_rn(m, 448.f);
    b.r = __fdiv_rn(448.f, m);
    if (pow2 && amax_bits < 0x7F800000u) {
        // round the exponent up unless the mantissa is zero; m / 448 <= 2^120, so no overflow
        const uint32_t u = (__float_as_uint(b.scale) + 0x7FFFFFu) & 0x7F800000u;
        b.scale = __uint_as_float(u);
        b.r = __uint_as_float((254u << 23) - u);
    }
    return b;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Two fp32 -> two E4M3 codes (lo in the low byte), nearest even, saturating; NaN -> 0x7F.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
    return f32x2_to_e4m3x2(a, b) | f32x2_to_e4m3x2(c, d) << 16;
}

// Two fp32 -> bf16x2 (lo in the low half), nearest even.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace moe
