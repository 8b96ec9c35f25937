"""The FP8 block scale and the quotients that codes are rounded from (csrc/fp8_scale.h),
compiled for the host: every mantissa that a scale can have, with values around every
border between two E4M3 codes, against fp32 division; the ends of the range; and the
plain step-by-step form of the quantiser against v / scale in 64 bits."""
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_ffn_05_b200", "csrc")

PROG = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#define __device__
#define __forceinline__ inline
struct float2 { float x, y; };
static inline float2 make_float2(float x, float y) { return {x, y}; }
static inline uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
static inline float __uint_as_float(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static inline uint32_t __float_as_uint(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static inline float __fmaf_rn(float a, float b, float c) { return fmaf(a, b, c); }
static int off_by;  // the approximate reciprocal's error, in units: -1 .. 1
static inline float reciprocal_approx(float x) {
    const float r = (float)(1.0 / (double)x);
    return isfinite(x) ? __uint_as_float(__float_as_uint(r) + off_by) : r;
}
static inline float2 __fmul2_rn(float2 a, float2 b) { return {a.x * b.x, a.y * b.y}; }
static inline float2 __ffma2_rn(float2 a, float2 b, float2 c) { return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
#include "fp8_scale.h"
using namespace moe;

int main() {
    float t[16];
    for (int i = 0; i < 8; ++i) t[i] = (float)(2 * i + 1) * ldexpf(1.f, -10), t[8 + i] = 1.f + (float)(2 * i + 1) / 16.f;
    long wrong = 0, by_reciprocal = 0;
    for (off_by = -1; off_by <= 1; ++off_by) {
#pragma omp parallel for reduction(+ : wrong, by_reciprocal)
        for (uint32_t S = 0; S < 1u << 23; ++S) {
            const float m = __uint_as_float(127u << 23 | S);
            wrong += over_448(m) != m / 448.f;
            const BlockScale b = with_reciprocal(m);
            for (int k = 0; k < 16; ++k) {
                const uint32_t c = __float_as_uint((float)((double)t[k] * m));
                float v[6], q[6];
                for (int d = 0; d < 6; ++d) v[d] = q[d] = __uint_as_float(c + d - 3);
                scale_values(q, b);
                for (int d = 0; d < 6; ++d) {
                    const float want = v[d] / m, r = v[d] * (1.f / m);
                    wrong += (q[d] < t[k]) != (want < t[k]) || (q[d] > t[k]) != (want > t[k]);
                    by_reciprocal += (r < t[k]) != (want < t[k]) || (r > t[k]) != (want > t[k]);
                }
            }
        }
    }
    off_by = 0;
    // the ends: the smallest scale, large ones, infinite and NaN ones, zeros of either sign
    const uint32_t amax[] = {0, 1, 27u << 23, (27u << 23) + 1, 0x42000000, 0x7F7FFFFF, 0x7F800000, 0x7FC00000};
    for (uint32_t a : amax)
        for (int pow2 = 0; pow2 < 2; ++pow2) {
            const BlockScale b = block_scale(a, pow2);
            const float m = __uint_as_float(a);
            float vs[] = {0.f, -0.f, m, -m, m / 3, -m / 7, m / 999, 1e-44f}, q[8];
            memcpy(q, vs, sizeof q);
            scale_values(q, b);
            for (int i = 0; i < 8; ++i) {
                const float w = vs[i] / b.scale;
                wrong += isnan(q[i]) != isnan(w) || (!isnan(w) && signbit(q[i]) != signbit(w)) ||
                         fabsf(q[i] - w) > fabsf(w) * 1.2e-7f + 1e-30f;
            }
        }
    printf("%ld %ld\n", wrong, by_reciprocal);
}
"""


def test_quotients_fall_on_the_same_side_of_every_border_as_a_division():
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "q.cpp"), os.path.join(d, "q")
        with open(src, "w") as f:
            f.write(PROG)
        r = subprocess.run(["g++", "-std=c++17", "-O2", "-march=native", "-ffp-contract=off", "-fopenmp", "-Wno-unknown-pragmas",
                            "-I", CSRC, src, "-o", exe], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        wrong, by_reciprocal = map(int, subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split())
    assert wrong == 0
    assert by_reciprocal > 10 ** 6  # what is tested does matter


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_codes_are_nearest_to_value_over_scale(dt, block, pow2):
    """The quotient in fp32 is off by 2^-24 relative at most, so a code is as near to v / scale in 64 bits as any
    other to within that; where v / scale is a border exactly, fp32 has it exactly, and the even code is taken."""
    v = torch.randn(512, 1024, generator=torch.Generator().manual_seed(5)).to(dt)
    v[:128, 128:256] = torch.arange(-63, 65) * 2.0 ** -6 + 0.75 * torch.sign(torch.arange(-63, 65))
    v[:128, 128] = 1.75  # scale 2^-8: v / scale is a multiple of 4, many of them exact ties
    q, s = ref.quantise(v, block, pow2)
    x = v.double() / ref.spread(s, 512, 1024, block)
    got = q.view(torch.float8_e4m3fn).double()
    want, step, border = ref.e4m3(x)
    near = border <= x.abs() * 2.0 ** -24
    assert torch.equal(got[~near], want[~near])
    assert ((got - x).abs() <= step / 2 + x.abs() * 2.0 ** -24).all()
    tie = border == 0
    assert tie.sum() >= 20 and torch.equal(got[tie], want[tie])


def test_an_exact_tie_goes_to_the_even_code():
    """-1.3671875 / 0.0068359375 is -200, halfway between -192 and -208; times 448 / m it is a little more."""
    v = torch.zeros(1, 128)
    v[0, 0], v[0, 1] = -1.3671875, 448 * 0.0068359375
    q, s = ref.quantise(v, 1, False)
    assert s.item() == 0.0068359375
    assert q.view(torch.float8_e4m3fn).float()[0, 0] == -192
    m = np.float32(448 * 0.0068359375)
    assert np.float32(-1.3671875) * (np.float32(448) / m) < -200
