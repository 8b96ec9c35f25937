"""Plain 64-bit forms of the FP8 operators and the error bounds their tests use.

Tolerances (u = 2^-24, half a step of fp32 relative to the value):

* Quantiser: every step is one correctly rounded fp32 operation, so codes and
  scales are compared bit for bit with the same steps in numpy.
* Norm: the sum of squares of d <= 32768 non-negative terms is a chain of at
  most 64 fmas per lane and two five-step trees: relative error <= 74 u; the
  mean, + eps, square root and quotient add 4 u at most, and the root halves
  what came before: below 42 u. s has one rounding (u), which enters n directly
  and through the sum (u each); the two products add 2 u. In all below 46 u,
  within 2^-18 = 64 u relative to n, which tests allow, plus half a step of the
  output type.
* Matrix product: a sum of 128 products of E4M3 codes (exact in fp32) in any
  order, rounded or truncated, is within 128 * 2^-23 of the sum of magnitudes; the
  scale product, one fma per K block and at most 8 adds over a cluster stay
  within (nkb + 10) u of it.
* Shared expert: the bound of the matrix product on g and u carries over to h
  (|silu'| < 1.1, |silu(g)| <= |g|, 2^-19 relative for SiLU's exponential and
  quotient); a code of h may move by one step where h / scale lies that near to a
  rounding border, and by the scale's own error elsewhere; the second product
  weighs those moves with |W2| and adds its own bound.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def quantise(v, block_rows, pow2):
    """Codes (uint8) and scales of fp32 v, step by step in fp32 (numpy, CPU)."""
    v = v.detach().float().cpu().numpy()
    r, c = v.shape
    nr, nc = -(-r // block_rows), -(-c // 128)
    p = np.zeros((nr * block_rows, nc * 128), np.float32)
    p[:r, :c] = v
    with np.errstate(all="ignore"):
        m = np.abs(p).reshape(nr, block_rows, nc, 128).max(axis=(1, 3))  # a NaN carries through
        m = np.where(np.isnan(m), m, np.maximum(m, np.float32(2.0 ** -100)))
        s = (m / np.float32(448)).astype(np.float32)
        if pow2:
            fin = np.isfinite(s)
            man, ex = np.frexp(np.where(fin, s, np.float32(1)))
            pw = np.ldexp(np.float32(1), np.where(man == 0.5, ex - 1, ex)).astype(np.float32)
            s = np.where(fin, pw, s)
        q = p / np.repeat(np.repeat(s, block_rows, 0), 128, 1)
    q = torch.from_numpy(np.clip(q, -448, 448)[:r, :c].copy())
    return q.to(torch.float8_e4m3fn).view(torch.uint8), torch.from_numpy(s)


def spread(scales, rows, cols, block_rows):
    s = scales.double().repeat_interleave(block_rows, 0)[:rows] if block_rows > 1 else scales.double()
    return s.repeat_interleave(128, 1)[:, :cols]


def values(codes, scales, cols, block_rows):
    """fp64 values of codes [rows][ld] and their scales."""
    c = codes[:, :cols].contiguous().view(torch.float8_e4m3fn).double()
    return c * spread(scales, c.shape[0], cols, block_rows)


def held(codes, pad=16, fill=0x7F):
    """Codes in rows of a multiple of `pad` bytes; what lies between is filled with NaN codes."""
    r, c = codes.shape
    p = torch.full((r, -(-c // pad) * pad), fill, dtype=torch.uint8, device=codes.device)
    p[:, :c] = codes
    return p


def gemm_bound(a_abs, w_abs, K):
    nkb = -(-K // 128)
    return (128 * 2.0 ** -23 + (nkb + 10) * U) * (a_abs @ w_abs.t())


def e4m3(v):
    """Nearest E4M3 value of fp64 v, ties to even, saturating; and the distance to the nearest border."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -6))).clamp_min(-6)
    step = torch.exp2(e - 3)
    q = torch.clamp(torch.round(v / step) * step, -448, 448)
    t = a / step
    border = ((t - torch.floor(t)) - 0.5).abs() * step
    return q, step, border


def block_scales(h, pow2):
    r, c = h.shape
    nc = -(-c // 128)
    p = torch.nn.functional.pad(h, (0, nc * 128 - c)).view(r, nc, 128)
    m = p.abs().amax(2).clamp_min(2.0 ** -100)
    s = m / 448
    return (torch.exp2(torch.ceil(torch.log2(s.float().double()))) if pow2 else s), p


def ffn(x, w1, w3, w2, pow2):
    """(y, bound) of the shared expert on fp64 values, before the output's rounding."""
    d, F = x.shape[1], w1.shape[0]
    g, u = x @ w1.t(), x @ w3.t()
    bg, bu = gemm_bound(x.abs(), w1.abs(), d), gemm_bound(x.abs(), w3.abs(), d)
    sg = g * torch.sigmoid(g)
    h = sg * u
    dh = 1.1 * bg * (u.abs() + bu) + sg.abs() * bu + 2.0 ** -19 * h.abs() + 1e-30
    s, p = block_scales(h, pow2)
    # relative error of a scale: that of the block's largest magnitude (0 for powers of two, chosen in tests
    # so that no scale is near a border of its own)
    ds, _ = block_scales(dh, False)
    rel = torch.zeros_like(s) if pow2 else ds / s + 4 * U
    sf = s.repeat_interleave(128, 1)[:, :F]
    relf = rel.repeat_interleave(128, 1)[:, :F]
    v = h / sf
    q, step, border = e4m3(v)
    near = dh / sf + v.abs() * (relf + 4 * U)
    move = torch.where(border <= near, step * 1.0001, torch.zeros_like(step)) + q.abs() * relf
    hv = q * sf
    y = hv @ w2.t()
    bound = (move * sf) @ w2.abs().t() * 1.01 + gemm_bound(hv.abs() + move * sf, w2.abs(), F)
    return y, bound
