"""The FP8 operators against their plain 64-bit forms (tolerances: fp8_ref.py)."""
import numpy as np
import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def lib():
    import routed_expert_ffn_05_b200 as M
    return M


def ty(dt):
    M = lib()
    return M.MOE_T_BF16 if dt in ("bf16", torch.bfloat16) else M.MOE_T_F32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def no_error():
    assert lib().moe_get_device_error() == 0


# ---------------------------------------------------------------- quantiser

def quantise(v, block, pow2, ldq=None):
    M = lib()
    r, c = v.shape
    ldq = ldq or c
    q = torch.full((r, ldq), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-r // block), -(-c // 128)), -7.0, device="cuda")
    desc = M.make_fp8_quant(r, c, ty(v.dtype), block, M.MOE_SCALE_POW2 if pow2 else M.MOE_SCALE_F32, ldv=v.stride(0),
                            ldq=ldq)
    M.moe_fp8_quantize(desc, v, q, s)
    return q, s


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 127), (5, 129), (128, 128), (129, 260), (300, 1001),
                                       (257, 4096)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantiser_is_exact(rows, cols, dt, block, pow2):
    g = gen(rows * 7919 + cols)
    wide = torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    v = (randn(g, rows, cols + 5) * wide).to(DT[dt])[:, :cols]  # rows 5 elements apart, so unaligned for most
    q, s = quantise(v, block, pow2, ldq=cols + 3)
    rq, rs = ref.quantise(v, block, pow2)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q[:, :cols].cpu(), rq)
    assert (q[:, cols:] == 0x55).all()  # between the rows nothing is written
    a = v.contiguous()
    if cols % 4 == 0:                   # and the vector path gives the same
        q2, s2 = quantise(a, block, pow2)
        assert torch.equal(q2.cpu(), rq) and torch.equal(s2, s)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantiser_zero_tiny_and_non_finite_blocks(block, pow2):
    v = torch.randn(128, 1024, generator=torch.Generator().manual_seed(1))
    v[:, :128] = 0
    v[:, 128:256] = 1e-38 * torch.sign(v[:, 128:256])
    v[:, 256:384] = 2.0 ** -100 * 448 * torch.sign(v[:, 256:384])  # right at a power of two
    v[7, 400] = float("nan")
    v[9, 600] = float("inf")
    v[:, 640:768] = 3.4e38
    v[11, 800] = -float("inf")
    v[12, 801] = float("nan")
    q, s = quantise(v.cuda(), block, pow2)
    rq, rs = ref.quantise(v, block, pow2)
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(rs))
    assert torch.equal(s.cpu().nan_to_num(nan=0.0, posinf=-1.0), rs.nan_to_num(nan=0.0, posinf=-1.0))
    got, want = q.cpu() & 0x7F, rq & 0x7F  # a NaN code's sign is not part of the format
    nan = want == 0x7F
    assert torch.equal(got[nan], want[nan])
    assert torch.equal(q.cpu()[~nan], rq[~nan])


# --------------------------------------------------------------------- norm

def check_norm(x, res, w, eps, pow2, outs=("sum", "y", "q"), pad=0, in_place=False):
    M = lib()
    T, d = x.shape
    v = x.double() if res is None else x.double() + res.double()
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * (1 if w is None else w.double())
    total = None
    if res is not None and "sum" in outs:
        total = res.clone() if in_place else torch.empty_strided(res.shape, res.stride(), dtype=res.dtype,
                                                                 device="cuda")
    src = total if in_place else res
    y = torch.full((T, d + pad), 5.0, dtype=torch.bfloat16, device="cuda") if "y" in outs else None
    q = torch.full((T, d + pad), 0x33, dtype=torch.uint8, device="cuda") if "q" in outs else None
    s = torch.full((T, -(-d // 128)), -1.0, device="cuda") if "q" in outs else None
    desc = M.make_norm(T, d, eps, ty(x.dtype), ty(res.dtype) if res is not None else 0,
                       ty(w.dtype) if w is not None else 0, M.MOE_SCALE_POW2 if pow2 else M.MOE_SCALE_F32,
                       ldx=x.stride(0), ldr=res.stride(0) if res is not None else None, ldy=d + pad, ldq=d + pad)
    M.moe_rms_norm(desc, x, src, w, total, y, q, s)
    no_error()
    if total is not None:
        assert torch.equal(total, (x.float() + res.float()).to(res.dtype))
    e = 2.0 ** -18
    if y is not None:
        assert ((y[:, :d].double() - n).abs() <= n.abs() * (2.0 ** -8 + e) + 2.0 ** -133).all()
        assert (y[:, d:] == 5.0).all()
    if q is not None:
        m = torch.nn.functional.pad(n.abs(), (0, -d % 128)).view(T, -1, 128).amax(2).clamp_min(2.0 ** -100) / 448
        if pow2:
            assert (torch.frexp(s)[0] == 0.5).all()
            assert (s.double() >= m * (1 - e)).all() and (s.double() / 2 < m * (1 + e)).all()
        else:
            assert ((s.double() - m).abs() <= m * e).all()
        sv = ref.spread(s, T, d, 1)
        assert ((ref.values(q, s, d, 1) - n).abs() <= n.abs() * (2.0 ** -4 * (1 + e) + e) + 2.0 ** -10 * sv * (1 + e)).all()
        assert (q[:, d:] == 0x33).all()


@pytest.mark.parametrize("T,d", [(1, 4096), (3, 256), (8, 4096), (5, 1), (2, 130), (7, 127), (4, 1000), (33, 1001),
                                 (2, 8192), (1, 32768), (3, 20001)])
@pytest.mark.parametrize("xt,rt,wt", [("bf16", "bf16", "bf16"), ("f32", "bf16", "f32"), ("f32", "f32", None),
                                      ("bf16", None, "bf16")])
@pytest.mark.parametrize("pow2", [False, True])
def test_norm(T, d, xt, rt, wt, pow2):
    g = gen(T * 31 + d)
    x = randn(g, T, d).to(DT[xt])
    res = (4 * randn(g, T, d)).to(DT[rt]) if rt else None
    w = (1 + 0.2 * randn(g, d)).to(DT[wt]) if wt else None
    check_norm(x, res, w, 1e-6, pow2)


@pytest.mark.parametrize("outs", [("sum",), ("y",), ("q",), ("sum", "q"), ("sum", "y")])
def test_norm_any_output_alone(outs):
    g = gen(3)
    check_norm(randn(g, 6, 512), randn(g, 6, 512).bfloat16(), None, 1e-5, False, outs)


@pytest.mark.parametrize("pad", [1, 2, 8])
def test_norm_strided_rows_and_in_place_residual(pad):
    g = gen(4)
    x = randn(g, 9, 640 + pad)[:, pad:]
    res = randn(g, 9, 640 + 3 * pad).bfloat16()[:, :640]
    check_norm(x, res, randn(g, 640).bfloat16(), 1e-6, False, pad=pad)
    check_norm(x, res.contiguous(), randn(g, 640), 1e-6, True, pad=pad, in_place=True)


def test_norm_of_zero_large_and_non_finite_rows():
    M = lib()
    x = torch.randn(5, 512, generator=torch.Generator().manual_seed(2)).cuda()
    x[0] = 0
    x[1] *= 1e15
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y = torch.empty(5, 512, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(5, 512, dtype=torch.uint8, device="cuda")
    s = torch.empty(5, 4, device="cuda")
    M.moe_rms_norm(M.make_norm(5, 512, 1e-6, M.MOE_T_F32), x, None, None, None, y, q, s)
    n = x.double() / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-6)
    assert (y[0] == 0).all() and ((q[0] & 0x7F) == 0).all()
    for t in (1, 4):
        assert ((y[t].double() - n[t]).abs() <= n[t].abs() * (2.0 ** -8 + 2.0 ** -18)).all()
    assert torch.isnan(y[2]).all() and torch.isnan(s[2]).all() and ((q[2] & 0x7F) == 0x7F).all()
    assert torch.isnan(y[3, 7]) and (y[3, :7] == 0).all() and torch.isnan(s[3, 0]) and not torch.isnan(s[3, 1:]).any()


# ----------------------------------------------------------- matrix product

def fp8_mat(g, rows, cols, block, scale=1.0, pad=16):
    codes, s = ref.quantise(scale * randn(g, rows, cols), block, False)
    return ref.held(codes.cuda(), pad), s.cuda()


def run_gemm(T, N, K, a, sa, w, sw, yt, acc=False, ldy=None, y=None):
    M = lib()
    ldy = ldy or N
    if y is None:
        y = torch.full((T, ldy), 3.0, dtype=DT[yt], device="cuda")
    M.moe_fp8_gemm(M.make_fp8_gemm(T, N, K, ty(yt), int(acc), lda=a.stride(0), ldw=w.stride(0), ldy=ldy), a, sa, w, sw, y)
    return y


def check_gemm(T, N, K, yt, acc=False, pad=16, ldy=None, seed=0):
    g = gen(T * 3 + N * 5 + K * 7 + seed)
    a, sa = fp8_mat(g, T, K, 1, 1.0, pad)
    w, sw = fp8_mat(g, N, K, 128, 0.02, pad)
    y0 = randn(g, T, N) if acc else None
    y = run_gemm(T, N, K, a, sa, w, sw, yt, acc, ldy, y0.clone() if acc else None)
    no_error()
    av, wv = ref.values(a, sa, K, 1), ref.values(w, sw, K, 128)
    want = av @ wv.t() + (y0.double() if acc else 0)
    bound = ref.gemm_bound(av.abs(), wv.abs(), K) + want.abs() * ref.HALF_STEP[DT[yt]] * 1.01
    err = (y[:, :N].double() - want).abs()
    print(f"T={T} N={N} K={K} {yt}: max err / bound {(err / bound).max().item():.3f}, "
          f"rel {(err.norm() / want.norm()).item():.2e}")
    assert (err <= bound).all()
    assert (y[:, N:] == 3.0).all()
    return a, sa, w, sw, y


SIZES = [(1, 128, 128), (1, 4096, 2048), (1, 1, 1), (2, 130, 16), (3, 100, 127), (8, 256, 129), (16, 384, 1111),
         (17, 129, 512), (32, 1003, 4096), (33, 512, 640), (64, 4096, 4096), (65, 200, 1000), (100, 2048, 256),
         (128, 1024, 2048), (129, 300, 700), (200, 128, 8192), (333, 1003, 1111), (512, 512, 512), (1000, 2048, 2048),
         (1500, 257, 385)]


@pytest.mark.parametrize("T,N,K", SIZES)
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_gemm(T, N, K, yt):
    check_gemm(T, N, K, yt)


# The choice of kernel and split goes by the grid (148 SMs): each is met by some of these.
GRIDS = [(1, 20000, 256),     # 16-token tiles, unsplit
         (16, 9000, 130), (32, 5000, 300),  # 32-token tiles
         (24, 12000, 520), (50, 16500, 200),  # 32 and 64, unsplit
         (300, 2300, 1500),   # 64-token tiles, one CTA per SM
         (257, 8192, 130), (1111, 2500, 1111), (2500, 1003, 385), (3000, 4096, 256), (5000, 700, 128),  # pairs of SMs
         (769, 3333, 77)]


@pytest.mark.parametrize("T,N,K", GRIDS)
@pytest.mark.parametrize("yt,acc", [("bf16", False), ("f32", False), ("f32", True)])
def test_gemm_every_grid(T, N, K, yt, acc):
    check_gemm(T, N, K, yt, acc)


@pytest.mark.parametrize("T", [900, 1700])
def test_gemm_pairs_strided_rows_and_the_same_bits(T):
    check_gemm(T, 2050, 500, "bf16", pad=64, ldy=2057)
    a, sa, w, sw, y = check_gemm(T, 2050, 700, "f32", ldy=2052)
    for _ in range(2):
        assert torch.equal(run_gemm(T, 2050, 700, a, sa, w, sw, "f32", ldy=2052), y)


@pytest.mark.parametrize("T", [1, 16, 40, 150, 600])
def test_gemm_adds_to_y(T):
    check_gemm(T, 320, 900, "f32", acc=True)


@pytest.mark.parametrize("T", [3, 64, 300])
def test_gemm_strided_rows(T):
    check_gemm(T, 250, 500, "bf16", pad=64, ldy=257)
    check_gemm(T, 250, 500, "f32", pad=1024, ldy=256)


@pytest.mark.parametrize("T", [1, 20, 64, 200, 700])
def test_gemm_is_the_same_every_time_and_for_every_batch(T):
    """Same call, same bits."""
    a, sa, w, sw, y = check_gemm(T, 640, 1536, "f32")
    for _ in range(3):
        assert torch.equal(run_gemm(T, 640, 1536, a, sa, w, sw, "f32"), y)


@pytest.mark.parametrize("T,N", [(5, 300), (300, 300), (50, 16500), (1500, 2300)])
def test_gemm_non_finite_scales_and_codes_stay_in_their_rows_and_columns(T, N):
    K = 520
    g = gen(9)
    a, sa = fp8_mat(g, T, K, 1)
    w, sw = fp8_mat(g, N, K, 128, 0.02)
    y = run_gemm(T, N, K, a, sa, w, sw, "f32")
    a2, sa2, w2, sw2 = a.clone(), sa.clone(), w.clone(), sw.clone()
    a2[2, 7] = 0x7F
    sa2[4, 1] = float("inf")
    w2[140, 300] = 0xFF
    sw2[2, 0] = float("nan")
    z = run_gemm(T, N, K, a2, sa2, w2, sw2, "f32")
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[2] = bad[4] = True
    bad[:, 140] = True
    bad[:, 256:384] = True
    assert torch.isnan(z[2]).all() and torch.isnan(z[:, 140]).all() and torch.isnan(z[:, 256:384]).all()
    assert not torch.isfinite(z[4]).any()
    assert torch.equal(z[~bad], y[~bad])


# ------------------------------------------------------------ shared expert

def ffn_weights(g, d, F, pow2=False):
    M = lib()
    t = []
    for shape in ((F, d), (F, d), (d, F)):
        codes, s = ref.quantise(0.02 * 64 / np.sqrt(shape[1]) * randn(g, *shape), 128, pow2)
        t += [ref.held(codes.cuda()), s.cuda()]
    return t, M.make_fp8_ffn_weights(*t)


def run_ffn(T, d, F, x, xs, w, yt="bf16", pow2=False, acc=False, y=None, ws=None):
    M = lib()
    desc = M.make_fp8_ffn(T, d, F, ty(yt), M.MOE_SCALE_POW2 if pow2 else M.MOE_SCALE_F32, int(acc),
                          ldx=x.stride(0), ld13=-(-d // 16) * 16, ld2=-(-F // 16) * 16)
    y = torch.empty(T, d, dtype=DT[yt], device="cuda") if y is None else y
    ws = torch.full((M.moe_fp8_ffn_workspace_size(desc),), 0x7F, dtype=torch.uint8, device="cuda") if ws is None else ws
    M.moe_shared_ffn_fp8(desc, w, x, xs, y, ws)
    return y


def ffn_want(x, xs, t, d, F, pow2):
    return ref.ffn(ref.values(x, xs, d, 1), ref.values(t[0], t[1], d, 128), ref.values(t[2], t[3], d, 128),
                   ref.values(t[4], t[5], F, 128), pow2)


@pytest.mark.parametrize("T,d,F", [(1, 4096, 2048), (8, 4096, 2048), (1, 128, 128), (2, 16, 1), (3, 100, 130),
                                   (16, 1000, 700), (17, 640, 128), (32, 256, 512), (64, 512, 384), (77, 1000, 700),
                                   (130, 384, 260), (300, 1024, 520), (700, 512, 1100), (24, 384, 2600),
                                   (60, 260, 5000), (1000, 2600, 1300), (2100, 300, 2050)])
@pytest.mark.parametrize("yt,pow2", [("bf16", False), ("f32", False), ("bf16", True)])
def test_ffn(T, d, F, yt, pow2):
    g = gen(T + d + F)
    x, xs = fp8_mat(g, T, d, 1)
    t, w = ffn_weights(g, d, F, pow2)
    y = run_ffn(T, d, F, x, xs, w, yt, pow2)
    no_error()
    want, bound = ffn_want(x, xs, t, d, F, pow2)
    bound = bound + want.abs() * ref.HALF_STEP[DT[yt]] * 1.01
    err = (y.double() - want).abs()
    print(f"T={T} d={d} F={F} {yt}: max err / bound {(err / bound).max().item():.3f}, "
          f"rel {(err.norm() / want.norm()).item():.2e}")
    assert (err <= bound).all()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_ffn_adds_to_y_and_repeats(T):
    d, F = 512, 640
    g = gen(T)
    x, xs = fp8_mat(g, T, d, 1)
    t, w = ffn_weights(g, d, F)
    y = run_ffn(T, d, F, x, xs, w, "f32")
    y0 = randn(g, T, d)
    z = run_ffn(T, d, F, x, xs, w, "f32", acc=True, y=y0.clone())
    assert torch.equal(z, y0 + y)  # one fp32 addition on the same sum
    assert torch.equal(run_ffn(T, d, F, x, xs, w, "f32"), y)


def test_ffn_non_finite_token_stays_alone():
    T, d, F = 6, 256, 384
    g = gen(1)
    x, xs = fp8_mat(g, T, d, 1)
    t, w = ffn_weights(g, d, F)
    y = run_ffn(T, d, F, x, xs, w, "f32")
    x[3, 0] = 0x7F
    z = run_ffn(T, d, F, x, xs, w, "f32")
    keep = torch.arange(T, device="cuda") != 3
    assert torch.isnan(z[3]).all() and torch.equal(z[keep], y[keep])


# ------------------------------------------------------- bounds of the buffers

@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (5, 300, 200), (40, 9000, 256), (60, 16500, 128), (300, 2300, 300),
                                   (1000, 4000, 200), (257, 8200, 128)])
@pytest.mark.parametrize("yt", ["bf16", "f32"])
def test_gemm_writes_its_rows_and_columns_only(T, N, K, yt):
    g = gen(T)
    a, sa = fp8_mat(g, T, K, 1)
    w, sw = fp8_mat(g, N, K, 128, 0.02)
    ldy = N + (8 if N % 8 == 0 else 3)
    y = torch.full((T + 140, ldy), -5.0, dtype=DT[yt], device="cuda")
    run_gemm(T, N, K, a, sa, w, sw, yt, ldy=ldy, y=y[:T])
    assert (y[T:] == -5.0).all() and (y[:, N:] == -5.0).all()
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("T,d,F", [(1, 256, 256), (9, 100, 130), (70, 1000, 700), (1000, 1300, 1100)])
def test_ffn_writes_its_rows_and_its_workspace_only(T, d, F):
    M = lib()
    g = gen(T)
    x, xs = fp8_mat(g, T, d, 1)
    t, w = ffn_weights(g, d, F)
    y = torch.full((T + 140, d), -5.0, device="cuda")
    n = M.moe_fp8_ffn_workspace_size(M.make_fp8_ffn(T, d, F, ldx=x.stride(0), ld13=-(-d // 16) * 16, ld2=-(-F // 16) * 16))
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    run_ffn(T, d, F, x, xs, w, "f32", y=y[:T], ws=ws[:n])
    assert (y[T:] == -5.0).all() and (ws[n:] == 0x5A).all()


@pytest.mark.parametrize("T,d", [(3, 640), (5, 1001)])
def test_norm_and_quantiser_write_their_rows_only(T, d):
    M = lib()
    g = gen(T)
    x, res = randn(g, T + 2, d), randn(g, T + 2, d).bfloat16()
    y = torch.full((T + 2, d), -5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T + 2, d), -5.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((T + 2, d), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 2, -(-d // 128)), -5.0, device="cuda")
    M.moe_rms_norm(M.make_norm(T, d, x_type=M.MOE_T_F32), x, res, None, out, y, q, s)
    for b in (1, 128):
        q2, s2 = torch.full_like(q, 0x5A), torch.full_like(s, -5.0)
        M.moe_fp8_quantize(M.make_fp8_quant(T, d, M.MOE_T_F32, b), x, q2, s2)
        assert (q2[T:] == 0x5A).all() and (s2[T if b == 1 else 1:] == -5.0).all()
    for t, v in ((y, -5.0), (out, -5.0), (q, 0x5A), (s, -5.0)):
        assert (t[T:] == v).all()


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in every large operand; rows at the ends and in the middle are checked."""
    M = lib()
    T, d = 67000, 32768
    rows = torch.tensor([0, 1, 33333, 65535, 65536, T - 1], device="cuda")
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(0))
    q = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, d // 128, device="cuda")
    M.moe_fp8_quantize(M.make_fp8_quant(T, d), x, q, s)
    rq, rs = ref.quantise(x[rows], 1, False)
    assert torch.equal(q[rows].cpu(), rq) and torch.equal(s[rows].cpu(), rs)
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    M.moe_rms_norm(M.make_norm(T, d), x, None, None, None, y, q, s)
    v = x[rows].double()
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    assert ((y[rows].double() - n).abs() <= n.abs() * (2.0 ** -8 + 2.0 ** -18)).all()
    assert ((ref.values(q[rows], s[rows], d, 1) - n).abs() <=
            n.abs() * (2.0 ** -4 + 2.0 ** -17) + 2.0 ** -10 * ref.spread(s[rows], len(rows), d, 1) * 1.001).all()
    # a product that reads those codes (2^31 bytes and more) and one that writes 2^31 outputs
    w, sw = fp8_mat(gen(1), 200, d, 128, 0.02)
    z = run_gemm(T, 200, d, q, s, w, sw, "f32")
    av, wv = ref.values(q[rows], s[rows], d, 1), ref.values(w, sw, d, 128)
    assert ((z[rows].double() - av @ wv.t()).abs() <= ref.gemm_bound(av.abs(), wv.abs(), d)).all()
    K = 48
    w, sw = fp8_mat(gen(2), d, K, 128, 0.1)
    run_gemm(T, d, K, q, s, w, sw, "bf16", y=y)  # rows of q are d bytes apart; K of each are read
    # (scales: one per row and 128 columns of K, so the first T entries of s, densely)
    sa = s.flatten()[:T].view(T, 1)
    av, wv = ref.values(q[rows], sa[rows], K, 1), ref.values(w, sw, K, 128)
    want = av @ wv.t()
    assert ((y[rows].double() - want).abs() <= ref.gemm_bound(av.abs(), wv.abs(), K) + want.abs() * 2.0 ** -8 * 1.01).all()
    no_error()


# ------------------------------------------------- streams, graphs, the block

def chain(T, d, F, seed):
    """norm -> FP8 shared expert, as one program's step: returns a closure and its output."""
    M = lib()
    g = gen(seed)
    h = randn(g, T, d)
    res = randn(g, T, d).bfloat16()
    t, w = ffn_weights(g, d, F)
    q = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    s = torch.empty(T, -(-d // 128), device="cuda")
    desc = M.make_fp8_ffn(T, d, F, M.MOE_T_BF16)
    ws = torch.empty(M.moe_fp8_ffn_workspace_size(desc), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    nd = M.make_norm(T, d, x_type=M.MOE_T_F32)

    def step(stream=None):
        M.moe_rms_norm(nd, h, res, None, None, None, q, s, stream)
        M.moe_shared_ffn_fp8(desc, w, q, s, y, ws, stream)
    return step, y, (h, res, t, w, q, s, ws)


@pytest.mark.parametrize("T", [1, 8, 70, 400])
def test_two_streams_at_once(T):
    a, ya, ka = chain(T, 1024, 1024, 1)
    b, yb, kb = chain(T + 3, 1024, 512, 2)
    a(), b()
    torch.cuda.synchronize()
    wa, wb = ya.clone(), yb.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ya.zero_(), yb.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        a(s1), b(s2)
    torch.cuda.synchronize()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)
    no_error()


@pytest.mark.parametrize("T", [1, 70, 400])
def test_captured_and_replayed(T):
    step, y, keep = chain(T, 1024, 768, 5)
    step()
    torch.cuda.synchronize()
    want = y.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
            step()
    y.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    keep[0].neg_()  # new inputs in the same buffers
    keep[1].neg_()
    graph.replay()
    torch.cuda.synchronize()
    got = y.clone()
    step()
    assert torch.equal(got, y)
    no_error()


@pytest.mark.parametrize("T,d,F,act,route,Fs", [
    (1, 256, 512, "bf16", 0, 512), (4, 256, 512, "bf16", 0, 512), (4, 256, 512, "bf16", 0, 0),
    (40, 256, 512, "mxfp8", 0, 256), (300, 256, 512, "mxfp8", 1, 512),
    (1, 4096, 2048, "bf16", 0, 2048), (8, 4096, 2048, "bf16", 0, 1024)])  # the decode dims: the fused decode kernels
def test_block_runs_its_parts(T, d, F, act, route, Fs):
    """moe_block gives the bits of norm, layer and shared expert called one after the other."""
    M = lib()
    E, k = 8, 2
    g = gen(T)
    dims = M.make_dims(T, d, F, E, k, route, M.MOE_A_MXFP8 if act == "mxfp8" else M.MOE_A_BF16, d_ff_shared=Fs)
    packed = {}
    for which, (n, kk) in {M.MOE_MAT_W1: (F, d), M.MOE_MAT_W3: (F, d), M.MOE_MAT_W2: (d, F)}.items():
        canon = torch.empty(E * n * kk * 17 // 32, dtype=torch.uint8, device="cuda")
        M.moe_quantize_weights(dims, which, 1.6 / kk ** 0.5 * randn(g, E, n, kk), canon)
        packed[which] = torch.empty(M.moe_packed_size(dims, which), dtype=torch.uint8, device="cuda")
        M.moe_pack_weights(dims, which, canon, packed[which])
    router = randn(g, E, d).bfloat16().view(torch.int16)
    w = M.make_weights(packed[M.MOE_MAT_W1], packed[M.MOE_MAT_W3], packed[M.MOE_MAT_W2], w_router=router)
    t, shared = ffn_weights(g, d, Fs) if Fs else (None, None)
    x, res = randn(g, T, d), randn(g, T, d).bfloat16()
    nw = (1 + 0.1 * randn(g, d)).bfloat16()
    tok = torch.arange(T, dtype=torch.int32, device="cuda") * 977 if route else None
    norm = M.make_norm(T, d, 1e-6, M.MOE_T_F32)
    y, out = torch.empty(T, d, device="cuda"), torch.empty_like(res)
    ws = torch.empty(M.moe_block_workspace_size(dims), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        M.moe_block(dims, w, norm, shared, x, res, nw, out, tok, y, ws)
    no_error()
    xn = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, d // 128, device="cuda")
    out2, y2 = torch.empty_like(res), torch.empty_like(y)
    M.moe_rms_norm(norm, x, res, nw, out2, xn, q, s)
    dl = M.make_dims(T, d, F, E, k, route, dims.act)
    wl = torch.empty(M.moe_workspace_size(dl), dtype=torch.uint8, device="cuda")
    M.moe_layer(dl, w, xn.view(torch.int16), tok, y2, wl)
    routed = y2.clone()
    if Fs:
        run_ffn(T, d, Fs, q, s, shared, "f32", acc=True, y=y2)
    assert torch.equal(out, out2) and torch.equal(y, y2)
    assert torch.isfinite(y).all()
    if Fs:  # and the shared part is what the 64-bit form gives
        want, bound = ffn_want(q, s, t, d, Fs, False)
        b = bound + ref.U * 2 * (y.double().abs() + routed.double().abs())
        assert ((y.double() - routed.double() - want).abs() <= b).all()


def captured_block(T, seed):
    """A MoE block at the decode dims, captured into a graph of its own workspace: (graph, y, what it uses)."""
    M = lib()
    d, F, E, k, Fs = 4096, 2048, 8, 2, 1024
    g = gen(seed)
    dims = M.make_dims(T, d, F, E, k, 0, M.MOE_A_BF16, d_ff_shared=Fs)
    packed = {}
    for which, (n, kk) in {M.MOE_MAT_W1: (F, d), M.MOE_MAT_W3: (F, d), M.MOE_MAT_W2: (d, F)}.items():
        canon = torch.empty(E * n * kk * 17 // 32, dtype=torch.uint8, device="cuda")
        M.moe_quantize_weights(dims, which, 1.6 / kk ** 0.5 * randn(g, E, n, kk), canon)
        packed[which] = torch.empty(M.moe_packed_size(dims, which), dtype=torch.uint8, device="cuda")
        M.moe_pack_weights(dims, which, canon, packed[which])
    router = randn(g, E, d).bfloat16().view(torch.int16)
    w = M.make_weights(packed[M.MOE_MAT_W1], packed[M.MOE_MAT_W3], packed[M.MOE_MAT_W2], w_router=router)
    t, shared = ffn_weights(g, d, Fs)
    x, res = randn(g, T, d), randn(g, T, d).bfloat16()
    norm = M.make_norm(T, d, 1e-6, M.MOE_T_F32)
    y, out = torch.empty(T, d, device="cuda"), torch.empty_like(res)
    ws = torch.empty(M.moe_block_workspace_size(dims), dtype=torch.uint8, device="cuda")

    def run():
        M.moe_block(dims, w, norm, shared, x, res, None, out, None, y, ws)
    run()
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
        run()
    return graph, y, want, (w, shared, t, packed, router, x, res, out, ws)


@pytest.mark.parametrize("Ta,Tb", [(1, 8), (40, 3)])
def test_two_captured_blocks_replayed_at_once(Ta, Tb):
    ga, ya, wa, ka = captured_block(Ta, 1)
    gb, yb, wb, kb = captured_block(Tb, 2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ya.zero_(), yb.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
    torch.cuda.synchronize()
    no_error()
    assert torch.equal(ya, wa) and torch.equal(yb, wb)
