"""The norm at the widths where the units per warp change: one up to 8192 elements, two up to
16384 (whose last warp may have one), four beyond."""
import pytest

from test_gpu_fp8 import DT, check_norm, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [8191, 8192, 8193, 8200, 8704, 9216, 12288, 16383, 16384, 16392, 16896])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("f32", None), ("bf16", None)])
def test_norm(d, xt, rt):
    g = gen(d)
    x = randn(g, 3, d).to(DT[xt])
    res = (4 * randn(g, 3, d)).to(DT[rt]) if rt else None
    check_norm(x, res, (1 + 0.2 * randn(g, d)).to(DT["bf16" if d % 3 else "f32"]), 1e-6, d % 2 == 0)


@pytest.mark.parametrize("d", [8200, 12288, 16384])
def test_norm_of_unaligned_rows(d):
    """The scalar kernels at widths that the vector ones would take."""
    g = gen(d)
    x = randn(g, 4, d + 1)[:, 1:]
    res = randn(g, 4, d + 3).bfloat16()[:, 3:]
    check_norm(x, res, None, 1e-6, False, pad=1)
    check_norm(x, res.contiguous(), randn(g, d), 1e-6, True, in_place=True)
