// The scale of a block of 128 FP8 values and the quotients its codes are rounded
// from: the rule shared by the quantiser, the norm and the shared expert's hidden
// row. Nothing but arithmetic, so that it also compiles for the host in a test.
//
// A block (128 consecutive elements of an activation row, or 128 x 128 of a
// weight matrix) with largest magnitude amax stores
//     m = max(amax, 2^-100),  scale = m / 448,  code = E4M3(v / scale)
// (E4M3 rounding to nearest even, saturating); with power-of-two scales, scale
// is the least power of two not below m / 448. Every quotient is one fp32
// operation rounded to nearest. Values a hundred binades below one quantise to
// zero codes. amax is taken over the magnitudes' bit patterns as integers, so a
// NaN is larger than every number: it makes its block's scale NaN and its codes
// NaN, and an infinity makes them Inf and (for finite values) zero.
//
// v / scale is not v * (448 / m): the reciprocal's rounding moves quotients over
// the borders between codes (0.03% of the codes of normal bf16 values), exact
// ties among them. Nor is it a division here: one per value made the quantiser 6
// to 20% slower. The reciprocal is kept in two words, 1 / scale = hi + lo (to
// 2^-45), and the quotient is fma(v, hi, v * lo), in pairs as many instructions
// as a product. It can differ from the rounded quotient in the last bit, and so
// give another code only if the exact quotient lies within 2^-21 ulp of the middle
// between a border of E4M3 and one of its fp32 neighbours. A border has five
// significant bits at most, so such a scale's 24-bit mantissa lies within a few
// units of a multiple of 2^20. Trying every mantissa with every border found
// three, all with the mantissa's upper half set, and none with lo one unit larger
// for those (two in the lower half then): hence the unit added below. A test goes
// over all of them.
#pragma once

#include <stdint.h>

namespace moe {

struct BlockScale {
    float scale;
    float hi, lo;  // 1 / (scale * pre) = hi + lo
    float pre;     // 1, or 2^-64 for scales too large for lo
};

// m / 448, rounded to nearest, for m >= 2^-100: the product's error is exact, and
// its correction right for every mantissa (the test goes over them too).
__device__ __forceinline__ float over_448(float m) {
    const float c = 1.f / 448.f, q = m * c;
    const float s = __fmaf_rn(__fmaf_rn(-448.f, q, m), c, q);
    return __float_as_uint(m) < 0x7F800000u ? s : q;  // infinity, NaN: themselves
}

__device__ __forceinline__ BlockScale with_reciprocal(float scale) {
    const uint32_t u = __float_as_uint(scale);
    BlockScale b;
    b.scale = scale;
    b.pre = u >= (227u << 23) ? 0x1p-64f : 1.f;
    const float s = scale * b.pre;
    const float h = reciprocal_approx(s);  // off by one unit at most
    b.hi = __fmaf_rn(__fmaf_rn(-s, h, 1.f), h, h);
    float e = __fmaf_rn(-s, b.hi, 1.f);  // exact, as is the next one
    if (e < 0.f) {                       // hi not above 1 / s: lo is never negative, and -0 keeps its sign
        b.hi = __uint_as_float(__float_as_uint(b.hi) - 1u);
        e = __fmaf_rn(-s, b.hi, 1.f);
    }
    b.lo = __uint_as_float(__float_as_uint(e * b.hi) + (u >> 22 & 1u));
    if (u >= 0x7F800000u) b.hi = b.lo = h;  // infinity: 0; NaN: NaN
    return b;
}

// From the bit pattern of amax (sign cleared).
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, bool pow2) {
    constexpr uint32_t kFloor = 27u << 23;  // 2^-100
    const float scale = over_448(__uint_as_float(max(amax_bits, kFloor)));
    if (!pow2 || amax_bits >= 0x7F800000u) return with_reciprocal(scale);
    // round the exponent up unless the mantissa is zero; m / 448 <= 2^120, so no overflow
    return with_reciprocal(__uint_as_float((__float_as_uint(scale) + 0x7FFFFFu) & 0x7F800000u));
}

// v / scale of each value, as far as codes go (see above).
template <int N>
__device__ __forceinline__ void scale_pairs(float2 (&v)[N], const BlockScale &b) {
    if (b.pre != 1.f)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = make_float2(v[i].x * b.pre, v[i].y * b.pre);
    const float2 hi = make_float2(b.hi, b.hi), lo = make_float2(b.lo, b.lo);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __ffma2_rn(v[i], hi, __fmul2_rn(v[i], lo));
}
template <int N>
__device__ __forceinline__ void scale_values(float (&v)[N], const BlockScale &b) {
    float2 p[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = make_float2(v[2 * i], v[2 * i + 1]);
    scale_pairs(p, b);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        v[2 * i] = p[i].x;
        v[2 * i + 1] = p[i].y;
    }
}

}  // namespace moe
