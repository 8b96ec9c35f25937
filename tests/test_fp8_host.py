"""The FP8 operators' argument checks (host only: nothing is launched) and the
binding's structs."""
import pytest

import routed_expert_ffn_05_b200 as M
from test_abi import header_struct_fields

A = 0x10000  # an aligned, never dereferenced address
B, C, D, E, F, G = (A + (i << 32) for i in range(1, 7))  # far apart


def refused(f, status=M.MOE_ERR_INVALID_ARG):
    with pytest.raises(M.MoeError) as e:
        f()
    assert e.value.status == status


def test_structs_match_the_header():
    for n in ("moe_norm_desc", "moe_fp8_quant_desc", "moe_fp8_gemm_desc", "moe_fp8_ffn_desc", "moe_fp8_ffn_weights"):
        assert [f for f, _ in getattr(M, n)._fields_] == header_struct_fields(n), n


def norm(T=4, d=256, x=A, res=B, w=C, sum_=D, y=E, q=F, s=G, **kw):
    M.moe_rms_norm(M.make_norm(T, d, **kw), x, res, w, sum_, y, q, s, stream=0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(x=None), dict(sum_=None, y=None, q=None, s=None), dict(s=None), dict(q=None),
    dict(res=None), dict(x_type=2), dict(res_type=-1), dict(w_type=5), dict(scale_mode=2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=255), dict(ldr=100), dict(ldy=1), dict(ldq=255),
    dict(x=A + 1), dict(res=B + 1), dict(w=C + 1), dict(y=E + 1), dict(s=G + 2), dict(sum_=D + 1),
    dict(x_type=1, x=A + 2), dict(ldx=1 << 40),
    dict(y=A), dict(y=A + 64), dict(q=B), dict(sum_=A), dict(sum_=B + 2), dict(s=E), dict(q=D + 8), dict(y=C),
])
def test_norm_refuses(kw):
    refused(lambda: norm(**kw))


def test_norm_refuses_rows_beyond_its_registers():
    refused(lambda: norm(d=32769), M.MOE_ERR_UNSUPPORTED)


@pytest.mark.parametrize("f", [
    lambda n: norm(T=n), lambda n: quant(rows=n, v_type=0), lambda n: quant(cols=n), lambda n: quant(rows=1 << 21, cols=1 << 19),
    lambda n: gemm(T=n), lambda n: gemm(N=n, ldy=1 << 29), lambda n: gemm(K=n), lambda n: ffn(T=n), lambda n: ffn(F_=n),
])
def test_sizes_beyond_the_indices_are_refused(f):
    refused(lambda: f((1 << 28) + 16), M.MOE_ERR_UNSUPPORTED)


def test_nothing_to_do_is_ok_without_a_gpu():
    norm(T=0)
    M.moe_fp8_quantize(M.make_fp8_quant(0, 128), A, B, C, stream=0)
    M.moe_fp8_gemm(M.make_fp8_gemm(0, 128, 128), A, B, C, D, E, stream=0)
    w = M.make_fp8_ffn_weights(A, B, A, B, C, D)
    M.moe_shared_ffn_fp8(M.make_fp8_ffn(0, 128, 256), w, E, F, G, A, stream=0)


def quant(rows=4, cols=256, v=A, q=B, s=C, **kw):
    M.moe_fp8_quantize(M.make_fp8_quant(rows, cols, **kw), v, q, s, stream=0)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=0), dict(v=None), dict(q=None), dict(s=None), dict(v_type=3), dict(block_rows=64),
    dict(scale_mode=9), dict(ldv=255), dict(ldq=255), dict(v=A + 1), dict(s=C + 1), dict(q=A), dict(q=A + 100),
    dict(s=B + 512), dict(s=A + 4),
])
def test_quantiser_refuses(kw):
    refused(lambda: quant(**kw))


def gemm(T=4, N=128, K=256, a=A, sa=B, w=C, sw=D, y=E, **kw):
    M.moe_fp8_gemm(M.make_fp8_gemm(T, N, K, **kw), a, sa, w, sw, y, stream=0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(N=0), dict(K=0), dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None),
    dict(y_type=2), dict(accumulate=2, y_type=1), dict(accumulate=1), dict(lda=255), dict(lda=264), dict(ldw=248),
    dict(K=250, lda=250), dict(ldy=127), dict(a=A + 8), dict(w=C + 1), dict(sa=B + 2), dict(y=E + 1),
    dict(y_type=1, y=E + 2), dict(y=A), dict(y=C + 16), dict(y=B), dict(y=D), dict(ldw=1 << 40),
])
def test_gemm_refuses(kw):
    refused(lambda: gemm(**kw))


def ffn(T=4, d=256, F_=512, x=A, xs=B, y=C, ws=D, w=None, **kw):
    w = M.make_fp8_ffn_weights(*(w or (E, E + 0x1000000, E, E + 0x1000000, F, F + 0x1000000)))
    M.moe_shared_ffn_fp8(M.make_fp8_ffn(T, d, F_, **kw), w, x, xs, y, ws, stream=0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(d=0), dict(F_=0), dict(x=None), dict(xs=None), dict(y=None), dict(ws=None), dict(ws=D + 16),
    dict(x=A + 8), dict(y=C + 1), dict(y_type=7), dict(accumulate=1), dict(accumulate=3, y_type=1),
    dict(scale_mode=-1), dict(ldx=255), dict(ld13=264), dict(ld2=500), dict(ldy=255),
    dict(w=(None, E, F, G, F, G)), dict(w=(E, None, F, G, F, G)), dict(w=(E + 1, F, E, F, F, G)),
    dict(y=A), dict(ws=C), dict(ws=A), dict(ws=E), dict(y=F),
])
def test_ffn_refuses(kw):
    refused(lambda: ffn(**kw))


def test_ffn_workspace_holds_h_and_its_scales():
    for T, F_ in ((1, 2048), (77, 700), (16384, 2048)):
        n = M.moe_fp8_ffn_workspace_size(M.make_fp8_ffn(T, 256, F_, ld2=-(-F_ // 16) * 16))
        assert n % 256 == 0 and n >= T * F_ + 4 * T * -(-F_ // 128)


def block(T=4, d=256, Fs=512, norm_kw=None, x=A, res=B, nw=C, rout=None, y=D, ws=E, shared=True, tok=None, route=0,
          wr=G):
    dims = M.make_dims(T, d, 256, 8, 2, route=route, d_ff_shared=Fs)
    w = M.make_weights(F, F, F, w_router=wr)
    sh = M.make_fp8_ffn_weights(*[F + (i << 24) for i in range(1, 7)]) if shared else None
    M.moe_block(dims, w, M.make_norm(T, d, **(norm_kw or {})), sh, x, res, nw, rout, tok, y, ws, stream=0)


@pytest.mark.parametrize("kw", [
    dict(shared=False), dict(ws=None), dict(ws=E + 64), dict(y=None), dict(y=D + 4), dict(norm_kw=dict(eps=-1.0)),
    dict(norm_kw=dict(ldx=100)), dict(x=None), dict(res=None, rout=G), dict(wr=None), dict(route=1), dict(y=A),
    dict(ws=D), dict(d=200), dict(Fs=100), dict(y=B), dict(x=A + 1), dict(nw=D),
])
def test_block_refuses(kw):
    refused(lambda: block(**kw))


def test_block_refuses_a_norm_of_another_shape():
    dims = M.make_dims(4, 256, 256, 8, 2)
    w = M.make_weights(F, F, F, w_router=G)
    for n in (M.make_norm(3, 256), M.make_norm(4, 128)):
        refused(lambda: M.moe_block(dims, w, n, None, A, B, C, None, None, D, E, stream=0))


@pytest.mark.parametrize("T,d,F_,pad", [(1, 128, 16, 0), (3, 300, 700, 0), (77, 1000, 4095, 32), (5, 1, 1, 7)])
def test_what_each_buffer_has_to_hold(T, d, F_, pad):
    """Every buffer one byte short is refused, and all at their sizes reach the entry point."""
    import ctypes
    import torch
    M._marshal.bind(torch.Tensor, torch.nn.Parameter)
    up, nb = lambda n: -(-n // 16) * 16, lambda n: -(-n // 128)  # noqa: E731
    rows = lambda n, ld, cols, size=1: ((n - 1) * ld + cols) * size  # noqa: E731
    ld, k, f = d + pad, up(d) + 16 * pad, up(F_)
    fd = M.make_fp8_ffn(T, d, F_, M.MOE_T_F32, ldx=k, ld13=k, ld2=f, ldy=ld)
    wt = [torch.zeros(n, dtype=torch.uint8) for n in (rows(F_, k, d), 4 * nb(F_) * nb(d)) * 2 + (rows(d, f, F_), 4 * nb(F_) * nb(d))]
    cases = [
        ((M.make_norm(T, d, 1e-6, M.MOE_T_F32, M.MOE_T_BF16, M.MOE_T_F32, ldx=ld, ldr=ld, ldy=ld, ldq=ld),), M._marshal.NORM,
         (rows(T, ld, d, 4), rows(T, ld, d, 2), 4 * d, rows(T, ld, d, 2), rows(T, ld, d, 2), rows(T, ld, d), 4 * T * nb(d))),
        ((M.make_fp8_quant(T, d, M.MOE_T_BF16, 1, ldv=ld, ldq=k),), M._marshal.QUANTIZE,
         (rows(T, ld, d, 2), rows(T, k, d), 4 * T * nb(d))),
        ((M.make_fp8_quant(T, d, M.MOE_T_F32, 128, ldv=ld, ldq=k),), M._marshal.QUANTIZE,
         (rows(T, ld, d, 4), rows(T, k, d), 4 * nb(T) * nb(d))),
        ((M.make_fp8_gemm(T, F_, d, M.MOE_T_BF16, lda=k, ldw=k, ldy=F_ + pad),), M._marshal.GEMM,
         (rows(T, k, d), 4 * T * nb(d), rows(F_, k, d), 4 * nb(F_) * nb(d), rows(T, F_ + pad, F_, 2))),
        ((fd, M.make_fp8_ffn_weights(*wt)), M._marshal.FFN,
         (rows(T, k, d), 4 * T * nb(d), rows(T, ld, d, 4), M.moe_fp8_ffn_workspace_size(fd)))]
    for structs, op, needs in cases:
        n = len(structs) + len(needs) + 1
        probe = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * n)(lambda *a: 0)
        weights = tuple(wt) if op == M._marshal.FFN else None
        go = lambda t, w=weights: M._marshal.call(  # noqa: E731
            ctypes.cast(probe, ctypes.c_void_p).value, -1, 0, structs, t, op, w)
        full = tuple(torch.zeros(m, dtype=torch.uint8) for m in needs)
        assert go(full) is None
        for i, m in enumerate(needs):
            short = full[:i] + (torch.zeros(m - 1, dtype=torch.uint8),) + full[i + 1:]
            assert go(short) == (0, 2 * i + 2, m), (op, i)
        for i in range(6 if weights else 0):
            short = weights[:i] + (weights[i][:-1].clone(),) + weights[i + 1:]
            assert go(full, short) == (0, 2 * (len(needs) + i) + 2, wt[i].numel())


def test_another_descriptor_is_refused():
    w = M.make_fp8_ffn_weights(A, B, A, B, C, D)
    for f in (lambda: M.moe_fp8_gemm(M.make_fp8_quant(4, 256), A, B, C, D, E, stream=0),
              lambda: M.moe_rms_norm(None, A, B, C, D, E, F, G, stream=0),
              lambda: M.moe_shared_ffn_fp8(M.make_fp8_ffn(4, 256, 512), M.make_norm(4, 256), A, B, C, D, stream=0),
              lambda: M.moe_block(M.make_dims(4, 256, 256, 8, 2), w, M.make_norm(4, 256), w, A, B, C, None, None, D, E, stream=0)):
        with pytest.raises(TypeError):
            f()


def test_sizes_beyond_63_bits_hold_in_no_tensor():
    import torch
    t = torch.zeros(64, dtype=torch.uint8)
    refused(lambda: quant(rows=1 << 30, cols=1 << 30, ldv=1 << 62, v=t))


def test_tensors_off_the_device_or_too_small_are_refused():
    import torch
    t = torch.zeros(4, 256, dtype=torch.uint8)
    check = M._marshal.check
    assert check(0, (None, t), (9, 16)) == 3            # a CPU tensor is on no device
    assert check(-1, (t,), (4 * 256 + 1,)) == 2         # one byte short
    assert check(-1, (t[1:, :16], 5), (3 * 256, 9)) == 0  # a view counts what lies behind it
    assert check(-1, (t[1:, :16],), (3 * 256 + 1,)) == 2
    refused(lambda: quant(rows=5, v=t))                 # through an entry point
    for bad in (lambda: check(0, [t], (1,)), lambda: check(0, (t,), ()), lambda: check(0, (object(),), (1,))):
        with pytest.raises((TypeError, AttributeError)):
            bad()


def test_expanded_tensors_count_their_memory():
    import torch
    check = M._marshal.check
    one = torch.ones(1)
    assert check(-1, (one.expand(4, 256),), (4 * 4 * 256,)) == 2  # 1024 elements, 4 bytes
    assert check(-1, (one.expand(4, 256),), (4,)) == 0
    assert check(-1, (torch.ones(4, 1).expand(4, 2),), (17,)) == 2
    assert check(-1, (torch.ones(4, 8).t(),), (128,)) == 0
    assert check(-1, (torch.ones(0),), (0,)) == 0


def test_cpu_tensors_are_refused_whatever_the_stream():
    import torch
    refused(lambda: quant(v=torch.zeros(4, 256, dtype=torch.bfloat16)))


class Sub:
    """Wraps a tensor into a subclass, which is looked at through its methods instead of the exchange table."""
    def __new__(cls, t):
        import torch

        class Wrapped(torch.Tensor):
            pass
        return t.as_subclass(Wrapped)


@pytest.mark.parametrize("wrap", [lambda t: t, Sub, lambda t: __import__("torch").nn.Parameter(t, False)])
def test_what_a_tensor_holds(wrap):
    import torch
    assert M._marshal.bind(torch.Tensor, torch.nn.Parameter)
    check = M._marshal.check
    base = torch.zeros(8, 64)
    for t, n in ((base, 2048), (base[1:], 1792), (base[:, 8:16], 2048 - 32), (base[6:, 60:], 512 - 240),
                 (base.t(), 2048), (base.view(torch.uint8), 2048), (base.bfloat16(), 1024), (base[3], 1280),
                 (base.to(torch.float8_e4m3fn), 512), (torch.ones(1).expand(4, 256), 4), (torch.zeros(0, 5), 0),
                 (torch.ones(3, 1).expand(3, 9), 12), (torch.tensor(1.0), 4)):
        t = wrap(t)
        assert check(-1, (t,), (n,)) == 0 and check(-1, (t,), (n + 1,)) == 2 and check(0, (t,), (0,)) == 1
        assert check(-1, (t,), (-5,)) == 0
    given_back = torch.zeros(64)
    given_back.untyped_storage().resize_(0)
    assert check(-1, (wrap(given_back),), (4,)) == 2 and check(-1, (wrap(given_back),), (0,)) == 0


def test_the_exchange_table_gives_the_address():
    """Through an entry point that refuses overlapping buffers: it sees the addresses the tensors have."""
    import ctypes
    import torch
    M._marshal.bind(torch.Tensor, torch.nn.Parameter)
    got = []
    probe = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 5)(lambda *a: got.append(a) or 0)
    t = torch.zeros(8, 64)
    desc = M.make_fp8_quant(8, 64)
    for x in (t, t[3:, 5:], Sub(t[2]), torch.nn.Parameter(t)):
        M._marshal.call(ctypes.cast(probe, ctypes.c_void_p).value, -1, 77, (desc,), (x, None, 12345), (4, 4, 4))
        assert got.pop() == (ctypes.addressof(desc), x.data_ptr(), None, 12345, 77)
    assert M._marshal.addresses((t, None, t[3, 5:], 7, Sub(t[1]))) == (
        t.data_ptr(), None, t[3, 5:].data_ptr(), 7, t[1].data_ptr())
    for bad in ((t, "x"), [t]):
        with pytest.raises((TypeError, AttributeError)):
            M._marshal.addresses(bad)
