"""What the binding takes for a buffer of a call: elements of the right type, rows where the descriptor
looks for them, and all of them within the tensor. Through the C part and the ctypes one, with CPU
tensors and an entry point that only records its arguments (CPU)."""
import ctypes

import pytest
import torch

import routed_expert_ffn_05_b200 as M
from routed_expert_ffn_05_b200 import marshal_py

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
TYPE, LAYOUT = 1000, 2000


class Sub(torch.Tensor):
    pass


@pytest.fixture(params=[("c", False), ("c", True), ("py", False)], ids=["c", "c-subclass", "ctypes"])
def marshal(request):
    kind, sub = request.param
    m = marshal_py if kind == "py" else M._marshal
    m.bind(torch.Tensor, torch.nn.Parameter)
    wrap = lambda t: t.as_subclass(Sub) if sub and isinstance(t, torch.Tensor) else t  # noqa: E731

    def call(structs, op, tensors, weights=None, ws=0):
        """0 when the entry point is reached, else the refusal's code."""
        n = len(structs) + len(tensors) + 1
        got = []
        fn = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * n)(lambda *a: got.append(a) or 0)
        r = m.call(ctypes.cast(fn, ctypes.c_void_p).value, -1, 0, structs, tuple(map(wrap, tensors)), op,
                   None if weights is None else tuple(map(wrap, weights)), ws)
        if r is None:
            want = [None if t is None else t.data_ptr() or None for t in tensors]
            assert list(got[0][len(structs):-1]) == want
            return 0
        assert not got
        return r[1]
    call.m = m
    return call


def norm_args(T=4, d=256, **kw):
    a = dict(x=torch.zeros(T, d, dtype=BF), res=torch.zeros(T, d, dtype=BF), w=torch.zeros(d, dtype=BF),
             out=torch.zeros(T, d, dtype=BF), y=torch.zeros(T, d, dtype=BF), q=torch.zeros(T, d, dtype=U8),
             s=torch.zeros(T, -(-d // 128)))
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("i,name,bad,good", [
    (0, "x", [F32, torch.float16, torch.int64, torch.int32, torch.bool, torch.float8_e4m3fn], [torch.int16, torch.uint16]),
    (2, "w", [F32, torch.float16], [torch.int16]),
    (4, "y", [F32, torch.float16, torch.float8_e5m2], [torch.int16]),
    (5, "q", [BF, torch.float8_e5m2, torch.bool], [torch.int8, torch.float8_e4m3fn]),
    (6, "s", [BF, torch.float64, torch.int64], [torch.int32])])
def test_types(marshal, i, name, bad, good):
    desc = (M.make_norm(4, 256),)
    base = norm_args()[i]
    for dt, code in [(t, TYPE + i) for t in bad] + [(t, 0) for t in good]:
        t = torch.zeros(8, *base.shape[1:] or base.shape, dtype=dt)  # enough bytes, whatever the type
        assert marshal(desc, marshal.m.NORM, norm_args(**{name: t})) == code, dt
    raw = torch.zeros(base.numel() * base.element_size(), dtype=U8)
    assert marshal(desc, marshal.m.NORM, norm_args(**{name: raw})) == 0  # a buffer of bytes
    assert marshal(desc, marshal.m.NORM, norm_args(**{name: raw[1:]})) == 2 * i + 2


def test_types_follow_the_descriptor(marshal):
    desc = (M.make_norm(4, 256, x_type=M.MOE_T_F32, res_type=M.MOE_T_F32, w_type=M.MOE_T_F32),)
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    assert marshal(desc, marshal.m.NORM, norm_args(x=f(4, 256), res=f(4, 256), w=f(256), out=f(4, 256))) == 0
    assert marshal(desc, marshal.m.NORM, norm_args(x=f(4, 256), res=f(4, 256), w=f(256))) == 2 * 3 + 2  # out: bf16 of fp32 rows
    assert marshal(desc, marshal.m.NORM, norm_args(x=torch.zeros(8, 256, dtype=BF), res=f(4, 256), w=f(256), out=f(4, 256))) == TYPE
    g = (M.make_fp8_gemm(4, 256, 128, M.MOE_T_F32),)
    a, w = torch.zeros(4, 128, dtype=U8), torch.zeros(256, 128, dtype=torch.float8_e4m3fn)
    assert marshal(g, marshal.m.GEMM, (a, f(4, 1), w, f(2, 1), f(4, 256))) == 0
    assert marshal(g, marshal.m.GEMM, (a, f(4, 1), w, f(2, 1), torch.zeros(8, 256, dtype=BF))) == TYPE + 4
    assert marshal(g, marshal.m.GEMM, (a, f(4, 1), f(256, 128), f(2, 1), f(4, 256))) == TYPE + 2


def test_layouts(marshal):
    T = d = 256
    op, at = marshal.m.NORM, lambda **kw: (M.make_norm(T, d, **kw),)
    z = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    args = lambda **kw: norm_args(T, d, **kw)  # noqa: E731
    assert marshal(at(), op, args(x=z(T, d))) == 0
    assert marshal(at(), op, args(x=z(d, T).t())) == LAYOUT                      # transposed
    assert marshal(at(), op, args(x=z(T, 2 * d)[:, ::2])) == LAYOUT
    assert marshal(at(), op, args(x=z(2 * T, d)[::2])) == LAYOUT                 # every second row, ld says every one
    assert marshal(at(ldx=2 * d), op, args(x=z(2 * T, d)[::2])) == 0
    assert marshal(at(), op, args(x=z(T, d + 8)[:, 8:])) == LAYOUT               # rows d + 8 apart, ld says d
    assert marshal(at(ldx=d + 8), op, args(x=z(T, d + 8)[:, 8:])) == 0
    assert marshal(at(ldx=d + 8), op, args(x=z(T + 1, d + 8)[:T, :d - 1])) == 2  # a row ends before d elements
    assert marshal(at(ldx=d + 8), op, args(x=z(T + 1, d + 8)[:, :d - 1])) == LAYOUT
    assert marshal(at(), op, args(x=z(2, T // 2, d))) == 0                       # any shape of the same dense memory
    assert marshal(at(), op, args(x=z(T * d))) == 0
    assert marshal(at(ldx=d + 8), op, args(x=z(2, T // 2, d + 8)[..., :d])) == 0
    assert marshal(at(ldx=d + 8), op, args(x=z(2, T, d + 8)[:, ::2, :d])) == LAYOUT
    assert marshal(at(), op, args(x=z(1, T, 1, d)[:, :, 0])) == 0
    assert marshal(at(), op, args(w=z(2 * d)[::2])) == LAYOUT + 2
    assert marshal(at(), op, args(s=torch.zeros(T, 4)[:, :2])) == LAYOUT + 6     # the table is dense
    assert marshal(at(), op, args(s=torch.zeros(2, T).t())) == LAYOUT + 6
    one = M.make_norm(1, d, ldx=999)
    for x in (z(1, 999)[:, :d], z(5, 2 * d)[:1, :d], z(5, 2 * d)[:, :d], z(5, d, 2)[:, :, 0].t().contiguous().t()[:, :d]):
        code = marshal((one,), op, norm_args(1, d, x=x))
        assert code == (0 if x.stride(-1) == 1 else LAYOUT)                      # one row: how far the next is does not matter
    assert marshal(at(), op, args(x=torch.zeros(1, 1, dtype=BF).expand(T, d))) == 2


def test_a_view_does_not_reach_beyond_itself(marshal):
    big = torch.zeros(8, 256, dtype=U8)
    desc = (M.make_fp8_quant(5, 256),)
    v, s = torch.zeros(5, 256, dtype=BF), torch.zeros(5, 2)
    assert marshal(desc, marshal.m.QUANTIZE, (v, big[:5], s)) == 0
    assert marshal(desc, marshal.m.QUANTIZE, (v, big[:4], s)) == 4  # four rows, though memory goes on behind them
    assert marshal(desc, marshal.m.QUANTIZE, (v, big[3:], s)) == 0
    assert marshal(desc, marshal.m.QUANTIZE, (v, big[4:], s)) == 4
    assert marshal((M.make_fp8_quant(0, 256),), marshal.m.QUANTIZE, (v[:0], big[:0], s[:0])) == 0


def test_weights_of_the_shared_expert(marshal):
    T, d, F = 3, 256, 384
    u, f = lambda *s: torch.zeros(*s, dtype=U8), torch.zeros  # noqa: E731
    good = (u(F, d), f(3, 2), u(F, d), f(3, 2), u(d, F), f(2, 3))
    desc = M.make_fp8_ffn(T, d, F)
    ws = torch.zeros(M.moe_fp8_ffn_workspace_size(desc), dtype=U8)
    bufs = (u(T, d), f(T, 2), torch.zeros(T, d, dtype=BF), ws)
    go = lambda w, b=bufs: marshal((desc, M.make_fp8_ffn_weights(*good)), marshal.m.FFN, b, w)  # noqa: E731
    assert go(good) == 0
    for i, bad, code in ((0, u(d, F).t(), LAYOUT), (1, f(2, 3).t(), LAYOUT), (2, f(F, d), TYPE), (3, f(3, 2).double(), TYPE),
                         (4, u(d, F + 16)[:, :F], LAYOUT), (5, torch.zeros(8, 3, dtype=BF), TYPE)):
        assert go(good[:i] + (bad,) + good[i + 1:]) == code + len(bufs) + i
    assert go(good[:4] + (u(d - 1, F), good[5])) == 2 * (len(bufs) + 4) + 2
    assert go(good, bufs[:3] + (ws[::2],)) == 8
    assert go(good, bufs[:3] + (torch.zeros(2 * len(ws), dtype=U8)[::2],)) == LAYOUT + 3


def test_the_block(marshal):
    T, d, Fs = 4, 256, 512
    dims = M.make_dims(T, d, 256, 8, 2, d_ff_shared=Fs)
    u, f, b = lambda *s: torch.zeros(*s, dtype=U8), torch.zeros, lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    good = (u(Fs, d), f(4, 2), u(Fs, d), f(4, 2), u(d, Fs), f(2, 4))
    shared, norm = M.make_fp8_ffn_weights(*good), M.make_norm(T, d, x_type=M.MOE_T_F32)
    n = M.moe_block_workspace_size(dims)
    bufs = (f(T, d), b(T, d), b(d), b(T, d), torch.zeros(T, dtype=torch.int32), f(T, d), u(n))
    w = M.make_weights(None, None, None)
    go = lambda t=bufs, ww=good, st=(dims, w, norm, shared): marshal(st, marshal.m.BLOCK, t, ww, n)  # noqa: E731
    assert go() == 0 and go(st=(dims, w, norm, None), ww=None) == 0
    for i, bad, code in ((0, b(2 * T, d), TYPE), (1, f(T, d), TYPE), (2, f(d), TYPE), (3, b(d, T).t(), LAYOUT),
                         (4, torch.zeros(T, dtype=torch.int64), TYPE), (4, torch.zeros(2 * T, dtype=torch.int32)[::2], LAYOUT),
                         (5, b(2 * T, d), TYPE), (5, f(T, 2 * d)[:, :d], LAYOUT)):
        assert go(bufs[:i] + (bad,) + bufs[i + 1:]) == code + i, i
    assert go(bufs[:6] + (u(n - 1),)) == 14
    assert go(ww=(f(Fs, d),) + good[1:]) == TYPE + 7
    for st in ((dims, w, None, shared), (dims, w, dims, shared), (norm, w, norm, shared)):
        with pytest.raises(TypeError):
            go(st=st)


def test_what_the_error_says():
    for code, why in ((1, "not on the current device"), (4, "fewer than 77 bytes"), (TYPE + 3, "type"), (LAYOUT + 3, "strides")):
        with pytest.raises(M.MoeError, match=why) as e:
            M._refuse("moe_rms_norm", code, 77)
        assert e.value.status == M.MOE_ERR_INVALID_ARG and f"argument {(code - 1) // 2 if code < 9 else 3}" in str(e.value)
