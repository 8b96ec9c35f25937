"""Calls of the FP8 operators as programs make them: captured before any other call, across streams that
wait for one another, from two threads, rows in batches of different sizes."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import captured_block, chain, fp8_mat, ffn_weights, gen, lib, no_error, quantise, randn, run_ffn, run_gemm

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import sys; sys.path.insert(0, 'tests')
import torch, test_gpu_fp8 as t
T, d, F = {T}, 1024, 1536
step, y, keep = t.chain(T, d, F, 1)
g = t.gen(2)
v, q, s = t.randn(g, 130, 512), torch.empty(130, 512, dtype=torch.uint8, device='cuda'), torch.empty(2, 4, device='cuda')
M = t.lib()
def all_of_it():
    step()
    M.moe_fp8_quantize(M.make_fp8_quant(130, 512, M.MOE_T_F32, 128), v, q, s)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    all_of_it()
y.fill_(float('nan')); q.zero_(); s.zero_()
graph.replay()
torch.cuda.synchronize()
a = y.clone(), q.clone(), s.clone()
all_of_it()
torch.cuda.synchronize()
assert all(torch.equal(i, j) for i, j in zip(a, (y, q, s))) and torch.isfinite(y).all()
assert M.moe_get_device_error() == 0
print('the same')
"""


@pytest.mark.parametrize("T", [1, 40, 1500])
def test_captured_before_any_other_call(T):
    r = subprocess.run([sys.executable, "-c", FIRST.format(T=T)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "the same" in r.stdout, r.stderr[-3000:]


@pytest.mark.parametrize("T", [1, 8, 70, 900])
def test_streams_that_wait_for_one_another(T):
    """The norm on one stream, the shared expert on another, with events between: every step has its own input."""
    M = lib()
    d, F, n = 1024, 1536, 6
    _, y, (h, res, t, w, q, s, ws) = chain(T, d, F, 3)
    xs = [randn(gen(10 + i), T, d) for i in range(n)]
    nd, fd = M.make_norm(T, d, x_type=M.MOE_T_F32), M.make_fp8_ffn(T, d, F, M.MOE_T_BF16)
    want = []
    for x in xs:
        M.moe_rms_norm(nd, x, res, None, None, None, q, s)
        M.moe_shared_ffn_fp8(fd, w, q, s, y, ws)
        want.append(y.clone())
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        outs, used = [], None
        for x in xs:
            if used is not None:
                a.wait_event(used)  # q and s are read until here
            M.moe_rms_norm(nd, x, res, None, None, None, q, s, a)
            ready = a.record_event()
            b.wait_event(ready)
            out = torch.empty_like(y)
            M.moe_shared_ffn_fp8(fd, w, q, s, out, ws, b)
            used = b.record_event()
            outs.append(out)
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(outs, want))
    no_error()


def in_a_new_thread(f):
    got = []

    def run():
        try:
            got.append(f())
        except BaseException as e:  # noqa: BLE001 (raised again in the caller's thread)
            got.append(e)
    th = threading.Thread(target=run)
    th.start()
    th.join()
    if isinstance(got[0], BaseException):
        raise got[0]
    return got[0]


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("what", ["product", "shared expert", "quantiser", "norm and shared expert"])
def test_the_first_call_of_a_thread(what, T):
    """A new thread has no device context before a call needs one."""
    g = gen(T)
    a, sa = fp8_mat(g, T, 1024, 1)
    w, sw = fp8_mat(g, 1003, 1024, 128, 0.02)
    y = torch.empty(T, 1003, device="cuda")
    t, fw = ffn_weights(g, 1024, 768)
    z = torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(2 * T * 1024, dtype=torch.uint8, device="cuda")
    v = randn(g, T, 1024)
    step, out, keep = chain(T, 1024, 768, 4)
    f = {"product": lambda: run_gemm(T, 1003, 1024, a, sa, w, sw, "f32", y=y),
         "shared expert": lambda: run_ffn(T, 1024, 768, a, sa, fw, y=z, ws=ws),
         "quantiser": lambda: quantise(v, 1, False)[0],
         "norm and shared expert": lambda: (step(), out)[1]}[what]
    want = f().clone()
    torch.cuda.synchronize()
    for _ in range(2):
        got = in_a_new_thread(f)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    no_error()


@pytest.mark.parametrize("T", [1, 40])
def test_the_block_in_a_new_thread(T):
    M = lib()
    d, F, E, k, Fs = 4096, 2048, 8, 2, 1024
    _, y, want, (w, shared, t, packed, router, x, res, out, ws) = captured_block(T, 1)
    dims = M.make_dims(T, d, F, E, k, 0, M.MOE_A_BF16, d_ff_shared=Fs)
    y.zero_()
    in_a_new_thread(lambda: M.moe_block(dims, w, M.make_norm(T, d, 1e-6, M.MOE_T_F32), shared, x, res, None, out, None, y, ws))
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    no_error()


def test_two_threads_at_once():
    T, N, K = (5, 600), 1003, 1024
    M = lib()
    cases = []
    for t in T:
        g = gen(t)
        a, sa = fp8_mat(g, t, K, 1)
        w, sw = fp8_mat(g, N, K, 128, 0.02)
        cases.append((t, a, sa, w, sw, run_gemm(t, N, K, a, sa, w, sw, "f32").clone()))
    torch.cuda.synchronize()
    wrong = []

    def work(case, stream):
        t, a, sa, w, sw, want = case
        desc = M.make_fp8_gemm(t, N, K, M.MOE_T_F32, lda=a.stride(0), ldw=w.stride(0))
        ys = [torch.empty(t, N, device="cuda") for _ in range(50)]
        for y in ys:
            M.moe_fp8_gemm(desc, a, sa, w, sw, y, stream)
        stream.synchronize()
        wrong.append(sum(not torch.equal(y, want) for y in ys))
    threads = [threading.Thread(target=work, args=(c, torch.cuda.Stream())) for c in cases]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert wrong == [0, 0]
    no_error()


@pytest.mark.parametrize("N,K", [(640, 1536), (4096, 512)])
def test_a_row_is_the_same_in_every_batch_to_within_the_bounds(N, K):
    """The order of the sums goes by the shape, so the bits may differ: each is within its bound of the same value."""
    g = gen(N)
    a, sa = fp8_mat(g, 700, K, 1)
    w, sw = fp8_mat(g, N, K, 128, 0.02)
    av, wv = ref.values(a, sa, K, 1), ref.values(w, sw, K, 128)
    bound = 2 * ref.gemm_bound(av.abs(), wv.abs(), K) + 2 * ref.U * 1.01 * (av @ wv.t()).abs()
    full = run_gemm(700, N, K, a, sa, w, sw, "f32")
    for T in (1, 16, 17, 40, 64, 65, 200):
        y = run_gemm(T, N, K, a[:T], sa[:T].contiguous(), w, sw, "f32")
        assert ((y.double() - full[:T].double()).abs() <= bound[:T]).all()
