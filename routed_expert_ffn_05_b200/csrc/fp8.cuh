// FP8 matrices with one fp32 scale per block of 128 (the block rule: fp8_scale.h).
#pragma once

#include "common.cuh"

namespace moe {

__device__ __forceinline__ float reciprocal_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace moe

#include "fp8_scale.h"

namespace moe {

constexpr int kFp8Block = 128;

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
