"""The FP8 products' bounded waits: one that runs out ends the kernel with an error status,
within about its limit, and the next call is clean."""
import time

import pytest
import torch

from test_gpu_fp8 import ffn_weights, fp8_mat, gen, lib, no_error, run_ffn, run_gemm

pytestmark = pytest.mark.gpu


def gives_up(call, where, y):
    """`call` with waits of 1 ms that run out: the error word, the time, and the same bits as before afterwards."""
    M = lib()
    want = call().clone()
    no_error()
    try:
        M.moe_debug_set_fp8_wait(1_000_000, where)
        t0 = time.perf_counter()
        call()
        code = M.moe_get_device_error()
        dt = time.perf_counter() - t0
    finally:
        M.moe_debug_set_fp8_wait()
    print(f"gave up after {dt * 1e3:.1f} ms")
    assert code == M.MOE_DEVERR_TIMEOUT
    assert dt < 1.0
    y.fill_(float("nan"))
    assert torch.equal(call(), want)
    no_error()


# One CTA per tile of each width (no split along K), and pairs of SMs. K blocks of a tile: far more than the
# accumulators in flight, so that most of them come after the wait that gave up.
@pytest.mark.parametrize("T,N,K", [(1, 20000, 1024), (1, 20000, 8192), (24, 12000, 4096), (50, 16500, 4096), (3000, 4096, 2048)])
def test_a_wait_that_runs_out(T, N, K):
    g = gen(T)
    a, sa = fp8_mat(g, T, K, 1)
    w, sw = fp8_mat(g, N, K, 128, 0.02)
    y = torch.empty(T, N, dtype=torch.float32, device="cuda")
    gives_up(lambda: run_gemm(T, N, K, a, sa, w, sw, "f32", y=y), 1, y)


# Clusters of two and four CTAs along K: a rank that gives up still sends what it has, and none leaves while
# another may send to it.
@pytest.mark.parametrize("T,N,K", [(8, 512, 8192), (1, 4096, 4096), (24, 1100, 8192), (60, 1003, 8192), (16, 8000, 2048)])
@pytest.mark.parametrize("where", [1, 2])
def test_a_wait_that_runs_out_in_a_cluster(T, N, K, where):
    g = gen(T)
    a, sa = fp8_mat(g, T, K, 1)
    w, sw = fp8_mat(g, N, K, 128, 0.02)
    y = torch.empty(T, N, dtype=torch.float32, device="cuda")
    gives_up(lambda: run_gemm(T, N, K, a, sa, w, sw, "f32", y=y), where, y)


@pytest.mark.parametrize("T,d,F,where", [(3, 4096, 2048, 1), (3, 4096, 2048, 2), (40, 4096, 4096, 1), (40, 2048, 1024, 2),
                                         (1500, 2048, 2048, 1)])
def test_a_shared_expert_whose_waits_run_out(T, d, F, where):
    g = gen(T)
    x, xs = fp8_mat(g, T, d, 1)
    t, w = ffn_weights(g, d, F)
    y = torch.empty(T, d, dtype=torch.float32, device="cuda")
    gives_up(lambda: run_ffn(T, d, F, x, xs, w, "f32", y=y), where, y)


def test_the_hook_refuses_other_places():
    M = lib()
    with pytest.raises(M.MoeError):
        M.moe_debug_set_fp8_wait(0, 7)
