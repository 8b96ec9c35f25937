"""Codes of the FP8 kernels where v / scale lies at a border between two of them."""
import numpy as np
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import no_error, quantise

pytestmark = pytest.mark.gpu

BORDERS = np.array([(2 * i + 1) * 2.0 ** -10 for i in range(8)] + [1 + (2 * i + 1) / 16 for i in range(8)])


def maxima():
    """Largest magnitudes of blocks: those whose scale's mantissa lies next to a multiple of 2^20, and others."""
    m = (np.arange(1 << 23, dtype=np.uint32) | np.uint32(127 << 23)).view(np.float32)
    off = (m / np.float32(448)).view(np.uint32) & 0xFFFFF
    odd = m[np.minimum(off, (1 << 20) - off) <= 16]
    return np.concatenate([odd, m[:: 1 << 15], np.float32([1.75, 1.0, 1.5])])


@pytest.mark.parametrize("exponent", [-96, -30, 0, 90, 110])
@pytest.mark.parametrize("offset", [0, 1])  # 1: rows at no multiple of 16 bytes, the scalar kernels
@pytest.mark.parametrize("block", [1, 128])
def test_codes_around_every_border(exponent, offset, block):
    m = maxima()
    s = m / np.float32(448)
    c = (BORDERS[None, :] * s[:, None].astype(np.float64)).astype(np.float32)  # [row][16]
    near = (c.view(np.uint32)[:, :, None] + np.arange(-3, 4).astype(np.uint32)).view(np.float32).reshape(len(m), -1)
    v = np.zeros((len(m), 128), np.float32)
    v[:, :112] = near * np.where(np.arange(112) % 3 == 1, np.float32(-1), np.float32(1))
    v[:, 112], v[:, 113] = m, -0.0
    v = np.ldexp(v, exponent)
    if block == 128:  # one block of 128 equal rows for each of some maxima
        v = np.repeat(v[:: max(1, len(m) // 100)], 128, 0)
    x = torch.zeros(v.shape[0], 128 + offset, device="cuda")
    x[:, offset:] = torch.from_numpy(v).cuda()
    x = x[:, offset:]
    q, sc = quantise(x, block, False)
    no_error()
    rq, rs = ref.quantise(x, block, False)
    assert torch.equal(sc.cpu(), rs) and torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantiser_against_64_bits(dt, block, pow2):
    """As near to v / scale as any code to within the fp32 quotient's half step, exact ties to the even code."""
    v = torch.randn(512, 1024, generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    v[:128, 128:256] = (torch.arange(-63, 65) * 2.0 ** -6 + 0.75 * torch.sign(torch.arange(-63, 65))).cuda()
    v[:128, 128] = 1.75
    q, s = quantise(v, block, pow2)
    x = v.double() / ref.spread(s, 512, 1024, block)
    got = q.view(torch.float8_e4m3fn).double()
    want, step, border = ref.e4m3(x)
    away = border > x.abs() * 2.0 ** -24
    assert torch.equal(got[away], want[away])
    assert ((got - x).abs() <= step / 2 + x.abs() * 2.0 ** -24).all()
    tie = border == 0
    assert tie.sum() >= 20 and torch.equal(got[tie], want[tie])
