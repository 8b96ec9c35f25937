#!/usr/bin/env python
"""Benchmark of the routed MoE FFN layer: MoE-layer tokens/s on B200.

Default workload: the decode layer (d_model 4096, d_ff 2048, 256 MXFP4 routed
experts, top-8 softmax routing, bf16 activations, one bf16 shared expert of
d_ff 2048) at T = 8 tokens. One step = one moe_layer call (route -> permute ->
expert FFN + shared expert -> combine) on one batch; batches rotate over 8
seeded inputs and L2 is flushed (256 MB write) between steps, outside the
timed events. Other configurations are measured in the same run and reported
under "breakdown".

    python bench.py [--gpus N] [--steps K] [--warmup W] [--impl ours|reference]
                    [--config decode|prefill|hash|q2k|tiny] [--T T] [--E E] [--ep]

With N > 1 (torchrun) every rank runs an independent replica on its own
batches (the path partitions by token batch; no data-path collective) and the
job value is the sum over ranks of tokens over the slowest rank's time. With
--ep the N ranks instead split one layer's routed experts (moe_layer_ep on a
contiguous share each, the shared expert on rank 0, NCCL all-reduce of y):
one batch per step, strong scaling.
--impl reference times the oracle (plain C, host cores) on the same workload.
"""
from __future__ import annotations

import argparse
import json
import math
import os
import statistics
import subprocess
import sys
import tempfile
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import synth  # noqa: E402

METRIC = "MoE-layer tokens/sec (decode T<=8, prefill T=4096); % HBM / FP4-TC roofline"
UNIT = "tokens/s"
FLUSH_BYTES = 256 << 20
NBATCH = 8


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def peaks(sustained=False):
    """(HBM GB/s, bf16 TFLOP/s, source): the measured figures, the bf16 one as a
    burst or (sustained=True) as a seconds-long loop under the power cap."""
    p = os.path.join(ROOT, "MEASURED_PEAKS.json")
    if os.path.exists(p):
        with open(p) as f:
            j = json.load(f)
        if sustained and "bf16_tflops_sustained" in j:
            return float(j["hbm_gbs"]), float(j["bf16_tflops_sustained"]), "measured sustained"
        return float(j["hbm_gbs"]), float(j["bf16_tflops"]), "measured"
    return 6650.0, (1400.0 if sustained else 1590.0), "fallback sustained" if sustained else "fallback"


# ---- device setup (product path only: no oracle here) -------------------------

class DeviceLayer:
    """Weights of one layer config on the device, built with the library's own
    quantiser and packer from the seeded generator's fp32 normals."""

    def __init__(self, M, torch, cfg, seed=0, experts=None):
        """experts: (begin, end) to hold only those routed experts (one rank of
        the expert-parallel layer); default all."""
        self.M, self.torch, self.cfg = M, torch, cfg
        dev = torch.device("cuda")
        self.dims = self.dims_for(cfg.T)
        self.ebegin, self.eend = experts if experts else (0, cfg.E)
        nE = self.eend - self.ebegin
        local = M.make_dims(cfg.T, cfg.d, cfg.F, nE, cfg.k, self.dims.route, self.dims.act, self.dims.wfmt, 0)
        self.packed = {}
        chunk = 16
        for tid, which in ((synth.W1, M.MOE_MAT_W1), (synth.W3, M.MOE_MAT_W3), (synth.W2, M.MOE_MAT_W2)):
            N, K = (cfg.F, cfg.d) if tid != synth.W2 else (cfg.d, cfg.F)
            q2k = cfg.wfmt == "q2k"
            per_e_a = N * K // 256 * 84 if q2k else N * K // 2
            per_e_b = 0 if q2k else N * K // 32
            canon = torch.empty(nE * (per_e_a + per_e_b), dtype=torch.uint8, device=dev)
            f32 = torch.empty(chunk * N * K, dtype=torch.float32, device=dev)
            tmp = torch.empty(chunk * (per_e_a + per_e_b), dtype=torch.uint8, device=dev)
            for e0 in range(0, nE, chunk):
                ne = min(chunk, nE - e0)
                for j in range(ne):  # expert ids are the layer's: a rank's experts draw the same weights
                    synth.normal_f32_device(seed, tid, self.ebegin + e0 + j, N * K, 0.0, cfg.w_std,
                                            out=f32[j * N * K:(j + 1) * N * K])
                cd = M.make_dims(1, cfg.d, cfg.F, ne, 1, wfmt=self.dims.wfmt)
                M.moe_quantize_weights(cd, which, f32, tmp)
                canon[e0 * per_e_a:(e0 + ne) * per_e_a].copy_(tmp[:ne * per_e_a])
                if per_e_b:
                    base = nE * per_e_a
                    canon[base + e0 * per_e_b: base + (e0 + ne) * per_e_b].copy_(
                        tmp[ne * per_e_a: ne * (per_e_a + per_e_b)])
            out = torch.empty(M.moe_packed_size(local, which), dtype=torch.uint8, device=dev)
            M.moe_pack_weights(local, which, canon, out)
            self.packed[which] = out
            del canon, f32, tmp
        to16 = lambda a: torch.from_numpy(a.astype(np.int16)).to(dev)
        self.wr = to16(synth.make_router(cfg, seed)) if cfg.has_router else None
        b = synth.make_bias(cfg, seed)
        self.bias = torch.from_numpy(b).to(dev) if b is not None else None
        sh = synth.shared_weights_bf16(cfg, seed)
        self.sh = [to16(a) for a in sh] if sh is not None else [None] * 3
        self.weights = M.make_weights(self.packed[M.MOE_MAT_W1], self.packed[M.MOE_MAT_W3],
                                      self.packed[M.MOE_MAT_W2], *self.sh, self.wr, self.bias)
        torch.cuda.synchronize()

    def dims_for(self, T):
        M, cfg = self.M, self.cfg
        return M.make_dims(T, cfg.d, cfg.F, cfg.E, cfg.k,
                           M.MOE_ROUTE_HASH if cfg.route == "hash" else M.MOE_ROUTE_SOFTMAX_TOPK,
                           {"mxfp8": M.MOE_A_MXFP8, "mxfp4": M.MOE_A_MXFP4}.get(cfg.act, M.MOE_A_BF16),
                           M.MOE_W_Q2K if cfg.wfmt == "q2k" else M.MOE_W_MXFP4,
                           cfg.Fs if cfg.Fs else 0)

    def with_weights(self, cfg):
        """The same routed experts under another config of equal dims and format."""
        other = object.__new__(DeviceLayer)
        other.__dict__.update(self.__dict__)
        other.cfg = cfg
        other.dims = other.dims_for(cfg.T)
        M, torch = self.M, self.torch
        dev = torch.device("cuda")
        to16 = lambda a: torch.from_numpy(a.astype(np.int16)).to(dev)
        other.wr = to16(synth.make_router(cfg)) if cfg.has_router else None
        b = synth.make_bias(cfg)
        other.bias = torch.from_numpy(b).to(dev) if b is not None else None
        other.sh = self.sh if cfg.Fs else [None] * 3
        other.weights = M.make_weights(self.packed[M.MOE_MAT_W1], self.packed[M.MOE_MAT_W3],
                                       self.packed[M.MOE_MAT_W2], *other.sh, other.wr, other.bias)
        return other


def touched_experts(M, torch, layer, x_d, tok_d, T):
    dims = layer.dims_for(T)
    ws = torch.empty(M.moe_workspace_size(dims), dtype=torch.uint8, device="cuda")
    idx = torch.empty((T, layer.cfg.k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, layer.cfg.k), dtype=torch.float32, device="cuda")
    M.moe_route(dims, x_d, layer.weights, tok_d, idx, w, ws)
    return idx.cpu().numpy()


def algorithmic_ffn_bytes(cfg, n_experts_touched):
    """Weight bytes one layer call's expert FFN must read: the touched routed
    experts' codes + scales (once each) and the bf16 shared expert."""
    if cfg.wfmt == "q2k":
        per = 3 * cfg.F * cfg.d // 256 * 84
    else:
        per = 3 * (cfg.F * cfg.d // 2 + cfg.F * cfg.d // 32)
    return per * n_experts_touched + 3 * cfg.Fs * cfg.d * 2


# DRAM traffic (dram__bytes_read.sum + dram__bytes_write.sum) from one-pass ncu
# captures of full-size launches, one record per workload. Each figure belongs
# to the sources it was taken on: their SHA-256 is checked before it is
# reported, and the field is null once any of them has changed.
#  - decode T=8: one decode_ffn_kernel launch on batch 0 (58 experts touched);
#    command and figures in profiles/decode_ffn_kernel_traffic_decode_T8.md.
#  - prefill T=4096 (w4a8): the gate/up and the down tc_ffn_kernel launches of
#    one layer call (batch 2), summed: 1,672.6 + 1,053.9 MB; command and figures
#    in profiles/tc_ffn_kernel_traffic_prefill_T4096.md.
_DECODE_SOURCES = ["routed_expert_ffn_05_b200/csrc/decode.cu", "routed_expert_ffn_05_b200/csrc/common.cuh",
                   "routed_expert_ffn_05_b200/csrc/kernels.h", "routed_expert_ffn_05_b200/csrc/ptx.cuh",
                   "routed_expert_ffn_05_b200/csrc/tma.h", "routed_expert_ffn_05_b200/csrc/tma.cu",
                   "routed_expert_ffn_05_b200/csrc/layout.h", "include/moe.h"]
_PREFILL_SOURCES = ["routed_expert_ffn_05_b200/csrc/prefill.cu", "routed_expert_ffn_05_b200/csrc/tc.cuh",
                    "routed_expert_ffn_05_b200/csrc/common.cuh", "routed_expert_ffn_05_b200/csrc/kernels.h",
                    "routed_expert_ffn_05_b200/csrc/ptx.cuh", "routed_expert_ffn_05_b200/csrc/tma.h",
                    "routed_expert_ffn_05_b200/csrc/tma.cu", "routed_expert_ffn_05_b200/csrc/layout.h",
                    "include/moe.h"]
TRAFFIC = [
    {"config": "decode", "T": 8, "E": 256, "act": "bf16", "dram_bytes": 830_643_968,
     "kernels": "decode_ffn_kernel<MXFP4>", "sources": _DECODE_SOURCES,
     "sources_sha256": "5a1e26552c03b6fa6f1ad24a129d268caafb2524cc858f6f9e099430c058b196"},
    {"config": "prefill", "T": 4096, "E": 256, "act": "mxfp8", "dram_bytes": 2_726_514_944,
     "kernels": "tc_ffn_kernel gate/up + down", "sources": _PREFILL_SOURCES,
     "sources_sha256": "80180ea0ee9c86470c7c5c9f529eb485fb50fb8faabbdff0ec42ef913d9b59d0"},
]


def sources_sha256(files):
    import hashlib
    h = hashlib.sha256()
    for f in files:
        with open(os.path.join(ROOT, f), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def captured_traffic(cfg, T):
    """The captured per-launch DRAM bytes (and the kernels they cover) when this
    run is a captured workload on the captured sources, else (None, None)."""
    for rec in TRAFFIC:
        base = synth.CONFIGS[rec["config"]]
        if (cfg.wfmt == base.wfmt and cfg.act == rec["act"] and cfg.route == base.route and T == rec["T"]
                and cfg.E == rec["E"] and cfg.d == base.d and cfg.F == base.F and cfg.Fs == base.Fs
                and cfg.zipf_s == base.zipf_s):
            if sources_sha256(rec["sources"]) == rec["sources_sha256"]:
                return rec["dram_bytes"], rec["kernels"]
    return None, None


def hbm_fraction(M, torch, layer, cfg, T, r, hbm, rank):
    """The decode roofline of one breakdown entry, as for the headline line:
    experts touched by batch 0's routing, its algorithmic bytes over the mean
    FFN time of the batch-0 steps, as a fraction of the HBM peak."""
    xb = torch.from_numpy(synth.make_x(cfg, 0, 1000 * rank).astype(np.int16)).cuda()
    U = len(np.unique(touched_experts(M, torch, layer, xb, None, T)))
    f0 = statistics.mean(r["ffn_ms"][::NBATCH])
    gbs = algorithmic_ffn_bytes(cfg, U) / (f0 / 1000.0) / 1e9
    return {"experts_touched": U, "ffn_hbm_gbs": gbs, "ffn_hbm_frac": gbs / hbm}


def measure(M, torch, layer, T, steps, warmup, rank, world, batches=NBATCH, e2e=False, ep=False):
    """Times `steps` moe_layer calls; returns a dict of per-step times (ms).
    ep: every rank runs its share of one expert-parallel layer on the same
    batch (moe_layer_ep on its experts, then the all-reduce of y)."""
    cfg = layer.cfg
    dev = torch.device("cuda")
    dims = layer.dims_for(T)
    ws = torch.empty(M.moe_workspace_size(dims), dtype=torch.uint8, device=dev)
    xs, toks = [], []
    src_rank = 0 if ep else rank  # expert parallelism: one batch, replicated on every rank
    for b in range(batches):
        c = cfg.with_T(T)
        xs.append(torch.from_numpy(synth.make_x(c, 0, batch_index(src_rank, b)).astype(np.int16)).to(dev))
        toks.append(torch.from_numpy(synth.make_token_ids(c, 0, batch_index(src_rank, b))).to(dev)
                    if cfg.route == "hash" else None)
    y = torch.empty((T, cfg.d), dtype=torch.float32, device=dev)
    flush = torch.empty(FLUSH_BYTES, dtype=torch.uint8, device=dev)
    if e2e:
        xh = [torch.empty((T, cfg.d), dtype=torch.int16).pin_memory() for _ in range(batches)]
        for b in range(batches):
            xh[b].copy_(xs[b].cpu())
        th = [t.cpu().pin_memory() if t is not None else None for t in toks]
        yh = torch.empty((T, cfg.d), dtype=torch.float32).pin_memory()
        xd = torch.empty((T, cfg.d), dtype=torch.int16, device=dev)
        td = torch.empty(T, dtype=torch.int32, device=dev) if cfg.route == "hash" else None
    stream = torch.cuda.current_stream()
    ev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(steps)]
    fev = [(torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)) for _ in range(steps)]
    for a, b in fev:  # torch creates the CUDA event on first record; the library needs live handles
        a.record(stream)
        b.record(stream)

    def layer_call(x, tok):
        if ep:
            M.moe_layer_ep(dims, layer.weights, layer.ebegin, layer.eend, rank == 0, x, tok, y, ws)
            if world > 1:
                torch.distributed.all_reduce(y)
        else:
            M.moe_layer(dims, layer.weights, x, tok, y, ws)

    def step(i, timed, ffn_events=False):
        b = i % batches
        flush.fill_(i & 0xFF)
        if timed:
            ev[i][0].record(stream)
            if ffn_events:
                M.moe_debug_set_ffn_events(fev[i][0], fev[i][1])
        if e2e:
            xd.copy_(xh[b], non_blocking=True)
            if td is not None:
                td.copy_(th[b], non_blocking=True)
            layer_call(xd, td)
            yh.copy_(y, non_blocking=True)
        else:
            layer_call(xs[b], toks[b])
        if timed:
            if ffn_events:
                M.moe_debug_set_ffn_events(None, None)
            ev[i][1].record(stream)

    for i in range(warmup):
        step(i, False)
    barrier(torch, world)
    torch.cuda.synchronize()
    n0 = M.moe_debug_launch_count()
    for i in range(steps):
        step(i, True)
    torch.cuda.synchronize()
    n1 = M.moe_debug_launch_count()
    barrier(torch, world)
    if M.moe_get_device_error() != 0:
        raise RuntimeError("device error word set during the benchmark")
    times = [a.elapsed_time(b) for a, b in ev]
    out = {"ms": times, "launches": n1 - n0}
    if not e2e:
        # A second pass with the library's FFN events installed times the expert
        # FFN stage alone (for the roofline). The events split the launch chain
        # (no early start of the FFN kernel during routing), so the layer time
        # above comes from the first, uninstrumented pass.
        barrier(torch, world)
        torch.cuda.synchronize()
        for i in range(steps):
            step(i, True, ffn_events=True)
        torch.cuda.synchronize()
        barrier(torch, world)
        if M.moe_get_device_error() != 0:
            raise RuntimeError("device error word set during the benchmark")
        out["ffn_ms"] = [a.elapsed_time(b) for a, b in fev]
        out["ms_with_ffn_events"] = [a.elapsed_time(b) for a, b in ev]
    return out


def barrier(torch, world):
    if world > 1:
        torch.distributed.barrier()


def max_over_ranks(torch, world, v):
    """The slowest rank's value (every rank gets it); NCCL on GPUs, gloo on CPU."""
    if world == 1:
        return v
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    t = torch.tensor([v], dtype=torch.float64, device=dev)
    torch.distributed.all_reduce(t, op=torch.distributed.ReduceOp.MAX)
    return float(t.item())


def batch_index(rank, b):
    """Seeded batch id of rank `rank`'s b-th rotating batch: replicas never share inputs."""
    return 1000 * rank + b


def job_value(world, tokens_per_step, steps, max_seconds):
    """Whole-job tokens/s: every rank's tokens over the slowest rank's time."""
    return world * tokens_per_step * steps / max_seconds


class Clocks:
    """nvidia-smi sampling during the timed region."""

    def __init__(self):
        self.proc, self.path = None, None

    def start(self):
        try:
            fd, self.path = tempfile.mkstemp(suffix=".csv")
            os.close(fd)
            q = ("index,clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.active,"
                 "clocks_event_reasons.hw_slowdown,clocks_event_reasons.hw_thermal_slowdown,"
                 "clocks_event_reasons.sw_thermal_slowdown,clocks_event_reasons.sw_power_cap")
            dev = os.environ.get("CUDA_VISIBLE_DEVICES", "0").split(",")[0]
            self.proc = subprocess.Popen(["nvidia-smi", "-i", dev, f"--query-gpu={q}", "--format=csv,noheader,nounits",
                                          "-lms", "100"], stdout=open(self.path, "w"), stderr=subprocess.DEVNULL)
        except (OSError, ValueError):
            self.proc = None

    def stop(self):
        if self.proc is None:
            return None
        time.sleep(0.25)
        self.proc.terminate()
        self.proc.wait()
        rows = []
        for line in open(self.path):
            f = [x.strip() for x in line.split(",")]
            if len(f) >= 9:
                try:
                    rows.append((float(f[1]), float(f[2]), float(f[3]), f[5:9]))
                except ValueError:
                    pass
        os.remove(self.path)
        if not rows:
            return None
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        reasons = sorted({n for r in rows for n, v in zip(names, r[3]) if v.lower() == "active"})
        loaded = [r[0] for r in rows if r[2] > 150.0] or [r[0] for r in rows]
        return {"sm_mhz": statistics.median(loaded), "sm_max_mhz": max(r[1] for r in rows),
                "reasons": reasons, "samples": len(rows)}


# ---- CPU baseline: the oracle on the host cores ---------------------------------

def oracle_sample(cfg, T, n_tokens, min_seconds, seed=0, batch=0):
    """Times the oracle's layer on the first n_tokens of a batch; returns
    (tokens/s, threads, seconds, description)."""
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    import oracle
    from harness import host_weights
    c = cfg.with_T(T)
    x = synth.make_x(c, seed, batch)
    tok = synth.make_token_ids(c, seed, batch) if c.route == "hash" else None
    wr = synth.make_router(c, seed) if c.has_router else None
    bias = synth.make_bias(c, seed)
    sh = synth.shared_weights_bf16(c, seed)
    toks = np.arange(n_tokens, dtype=np.int32)
    if c.route == "hash":
        idx, _, _ = oracle.hash_route(tok[:n_tokens], c.E, c.k)
    else:
        idx, _ = oracle.topk_softmax(oracle.router_logits(x[:n_tokens], wr, bias), c.k)
    hw = host_weights(c, seed)
    hw.ensure(np.unique(idx))
    ow = hw.oracle_layer(c, wr, bias, sh)
    reps, t0 = 0, time.perf_counter()
    while True:
        oracle.layer_tokens(ow, x, toks, tok)
        reps += 1
        el = time.perf_counter() - t0
        if el >= min_seconds or reps >= 200:
            break
    return reps * n_tokens / el, oracle.num_threads(), el, \
        f"{reps} x oracle layer on {n_tokens} token(s) of the {cfg.name} T={T} batch"


# ---- main -------------------------------------------------------------------------

def workload_desc(cfg):
    fmt = "Q2_K" if cfg.wfmt == "q2k" else "MXFP4"
    route = "hash (SplitMix64 of the token id)" if cfg.route == "hash" else f"top-{cfg.k} softmax"
    if cfg.zipf_s:
        route += f", Zipf({cfg.zipf_s}) router bias"
    act = {"mxfp8": "MXFP8 activations (w4a8)", "mxfp4": "MXFP4 activations (w4a4)"}.get(cfg.act, "bf16 activations")
    sh = f", bf16 shared expert d_ff {cfg.Fs}" if cfg.Fs else ""
    return (f"{cfg.name} layer T={cfg.T}: d_model {cfg.d}, d_ff {cfg.F}, {cfg.E} {fmt} routed experts, "
            f"{route} routing, {act}{sh}")


def expert_flops(cfg, T):
    """Useful expert-FFN multiply-adds x 2 of one layer call (routed + shared)."""
    return 2 * T * cfg.k * 3 * cfg.d * cfg.F + 2 * T * 3 * cfg.d * cfg.Fs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--config", default="decode", choices=["decode", "prefill", "hash", "q2k", "tiny"],
                    help="timed workload (default: the decode layer)")
    ap.add_argument("--T", type=int, default=None, help="tokens per step (default: the config's)")
    ap.add_argument("--E", type=int, default=None, help="routed experts (smaller only for profiling captures)")
    ap.add_argument("--no-breakdown", action="store_true")
    ap.add_argument("--no-cpu", action="store_true")
    ap.add_argument("--no-e2e", action="store_true")
    ap.add_argument("--act", default=None, choices=["bf16", "mxfp8", "mxfp4"],
                    help="activation mode override (w4a16 / w4a8 / w4a4)")
    ap.add_argument("--ep", action="store_true",
                    help="expert parallelism: the N ranks split one layer's routed experts (one batch, "
                         "partial sums all-reduced) instead of running N replicas")
    args = ap.parse_args()
    assert args.warmup >= 3, "at least 3 warm-up steps"

    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    from dataclasses import replace
    base_cfg = synth.CONFIGS[args.config]
    E = args.E if args.E else base_cfg.E
    T = args.T if args.T else base_cfg.T
    cfg = replace(base_cfg.with_T(T), E=E)
    if args.act:
        cfg = replace(cfg, act=args.act)
    workload = workload_desc(cfg)
    n_cpu_tokens = min(T, 8)

    if args.impl == "reference":
        if rank != 0:
            return
        per_step = []
        for i in range(args.warmup + args.steps):
            tps, threads, el, desc = oracle_sample(cfg, T, n_cpu_tokens, 0.0, batch=i % NBATCH)
            if i >= args.warmup:
                per_step.append(n_cpu_tokens / tps)
        ms = 1000 * statistics.mean(per_step) * T / n_cpu_tokens
        val = T / (ms / 1000)
        print(json.dumps({
            "impl": "reference", "metric": METRIC, "value": val, "unit": UNIT, "n_gpus": args.gpus,
            "steps": args.steps, "warmup": args.warmup, "ms_per_step": ms, "higher_is_better": True,
            "scaling": "weak", "vs_baseline": None, "dtype": "f64", "data": "synthetic",
            "config": {"workload": workload, "T": T},
            "cpu_baseline": {"kind": "oracle", "value": val, "unit": UNIT, "cores": threads,
                             "sample": f"each step: oracle layer on {n_cpu_tokens} of the {T} tokens of one batch, "
                                       f"scaled to the batch"},
            "e2e": {"value": val, "unit": UNIT, "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0},
        }))
        return

    import torch
    if world > 1:
        import datetime
        torch.cuda.set_device(int(os.environ.get("LOCAL_RANK", "0")))
        torch.distributed.init_process_group("nccl", timeout=datetime.timedelta(seconds=120))
    import routed_expert_ffn_05_b200 as M

    t0 = time.time()
    ep = args.ep
    span = M.moe_ep_range(E, rank, world) if ep else None
    if cfg.wfmt == "q2k" or cfg.d != synth.CONFIGS["decode"].d:
        base = DeviceLayer(M, torch, cfg, experts=span)
    else:
        base = DeviceLayer(M, torch, replace(synth.CONFIGS["decode"], E=E), experts=span)
    log(f"[bench] {cfg.wfmt} layer built in {time.time() - t0:.1f}s")
    layer = base.with_weights(cfg)
    # replicas: every rank's tokens count; expert parallelism: the ranks share one batch
    job_ranks = 1 if ep else world

    clocks = Clocks()
    clocks.start()
    r = measure(M, torch, layer, T, args.steps, args.warmup, rank, world, ep=ep)
    ck = clocks.stop()
    total_s = max_over_ranks(torch, world, sum(r["ms"]) / 1000.0)
    value = job_value(job_ranks, T, args.steps, total_s)
    ms_per_step = 1000.0 * total_s / args.steps

    if not args.no_e2e:
        e = measure(M, torch, layer, T, args.steps, args.warmup, rank, world, e2e=True, ep=ep)
        e2e_s = max_over_ranks(torch, world, sum(e["ms"]) / 1000.0)
    else:
        e2e_s = float("nan")

    # roofline of the expert FFN (the dominant stage), per step
    hbm, bf16, src = peaks()
    ffn_ms = statistics.mean(r["ffn_ms"]) if r["ffn_ms"] else float("nan")
    if cfg.act in ("mxfp8", "mxfp4") or T > 8:  # a dense contraction at the FP8 / FP4 / bf16 tensor-core rate
        fl = expert_flops(cfg, T)
        achieved = fl / (ffn_ms / 1000.0) / 1e12
        ratio = {"mxfp8": 2.0, "mxfp4": 4.0}.get(cfg.act, 1.0)  # nominal dense ratios to bf16: FP8 2x, FP4 4x
        # a run that met the power cap is held to the sustained (power-capped) figure
        capped = bool(ck and "sw_power_cap" in ck.get("reasons", []))
        _, bf16_peak, psrc = peaks(sustained=capped)
        peak = ratio * bf16_peak
        roof = {"kernel": "expert FFN: plan + gather/quantise + gate/up GEMM + down GEMM (tcgen05)",
                "bound": "tensor", "achieved": achieved, "peak": peak, "unit": "TFLOP/s",
                "frac": achieved / peak,
                "peak_source": f"{psrc} bf16" + (f" x {ratio:g} ({'FP8' if ratio == 2 else 'FP4'} nominal ratio)"
                                                  if ratio != 1 else ""),
                "frac_of_burst_peak": achieved / (ratio * bf16),
                "frac_of_fp4_peak": achieved / (4.0 * bf16_peak),
                "traffic": captured_traffic(cfg, T)[0], "traffic_kernels": captured_traffic(cfg, T)[1],
                "algorithmic_flops": fl, "ffn_ms": ffn_ms}
    else:
        xb = torch.from_numpy(synth.make_x(cfg, 0, 1000 * (0 if ep else rank)).astype(np.int16)).cuda()
        idx = touched_experts(M, torch, layer, xb, None, T)
        if ep:  # this rank's experts (and the shared expert on rank 0 only)
            idx = idx[(idx >= layer.ebegin) & (idx < layer.eend)]
        U = len(np.unique(idx))
        ffn_ms = statistics.mean(r["ffn_ms"][::NBATCH]) if r["ffn_ms"] else float("nan")
        alg = algorithmic_ffn_bytes(cfg if not ep or rank == 0 else replace(cfg, Fs=0), U)
        achieved = alg / (ffn_ms / 1000.0) / 1e9
        roof = {"kernel": "expert FFN: routed + shared", "bound": "hbm",
                "achieved": achieved, "peak": hbm, "unit": "GB/s", "frac": achieved / hbm,
                "peak_source": src, "traffic": captured_traffic(cfg, T)[0],
                "algorithmic_bytes": alg, "experts_touched": U, "ffn_ms": ffn_ms}
    line = {
        "metric": METRIC, "value": value, "unit": UNIT, "n_gpus": world, "steps": args.steps,
        "warmup": args.warmup, "ms_per_step": ms_per_step, "higher_is_better": True,
        "scaling": "strong" if ep else "weak",
        "vs_baseline": None,
        "dtype": ("mxfp4 x mxfp8 -> fp32" if cfg.act == "mxfp8" else "mxfp4 x mxfp4 -> fp32" if cfg.act == "mxfp4"
                  else ("q2k x bf16 -> fp32" if cfg.wfmt == "q2k" else "mxfp4 x bf16 -> fp32")),
        "data": "synthetic",
        "config": {"workload": workload, "T": T, "batches": NBATCH,
                   "l2": "flushed between steps (256 MB write), flush outside the timed events",
                   "parallelism": (f"expert-parallel x{world} (experts {layer.ebegin}..{layer.eend - 1} on rank 0, "
                                   f"NCCL all-reduce of y)" if ep else
                                   f"replicas x{world}" if world > 1 else "single GPU")},
        "roofline": roof,
        "e2e": {"value": job_value(job_ranks, T, args.steps, e2e_s), "unit": UNIT,
                "h2d_bytes_per_step": T * cfg.d * 2 + (T * 4 if cfg.route == "hash" else 0),
                "d2h_bytes_per_step": T * cfg.d * 4},
        "gpu_launches": r["launches"], "gpu_launches_per_step": r["launches"] / args.steps,
        "clocks": ck,
    }

    if not args.no_breakdown and rank == 0 and not ep:
        bd = {}
        if cfg.wfmt == "mxfp4" and cfg.d == synth.CONFIGS["decode"].d:
            dec = replace(synth.CONFIGS["decode"], E=E)
            for Tb in (1, 2, 4, 8):
                lb = base.with_weights(dec.with_T(Tb))
                rr = measure(M, torch, lb, Tb, 20, 3, rank, 1)
                bd[f"decode_T{Tb}"] = {"tokens_per_s": Tb / (statistics.mean(rr["ms"]) / 1000),
                                       "ms": statistics.mean(rr["ms"]), "ffn_ms": statistics.mean(rr["ffn_ms"]),
                                       **hbm_fraction(M, torch, lb, dec.with_T(Tb), Tb, rr, hbm, rank)}
            for name, act in (("prefill", "mxfp8"), ("hash", "mxfp8"), ("prefill", "mxfp4"), ("hash", "mxfp4"),
                              ("prefill", "bf16")):
                c = replace(synth.CONFIGS[name], E=E, act=act)
                rr = measure(M, torch, base.with_weights(c), c.T, 3, 3, rank, 1, batches=2)
                fl = expert_flops(c, c.T)
                tf = fl / (statistics.mean(rr["ffn_ms"]) / 1000) / 1e12
                bd[name + {"mxfp8": "", "mxfp4": "_w4a4", "bf16": "_w4a16"}[act]] = {
                    "T": c.T, "act": act, "tokens_per_s": c.T / (statistics.mean(rr["ms"]) / 1000),
                    "ms": statistics.mean(rr["ms"]), "ffn_ms": statistics.mean(rr["ffn_ms"]), "ffn_tflops": tf,
                    "ffn_frac_of_own_peak": tf / ({"mxfp8": 2.0, "mxfp4": 4.0, "bf16": 1.0}[act] * bf16),
                    "ffn_frac_of_fp4_peak": tf / (4.0 * bf16)}
            del base
            torch.cuda.empty_cache()
            q2 = DeviceLayer(M, torch, replace(synth.CONFIGS["q2k"], E=E))
            for Tb in (1, 8):
                qc = replace(synth.CONFIGS["q2k"], E=E).with_T(Tb)
                lb = q2.with_weights(qc)
                rr = measure(M, torch, lb, Tb, 20, 3, rank, 1)
                bd[f"q2k_T{Tb}"] = {"tokens_per_s": Tb / (statistics.mean(rr["ms"]) / 1000),
                                    "ms": statistics.mean(rr["ms"]), "ffn_ms": statistics.mean(rr["ffn_ms"]),
                                    **hbm_fraction(M, torch, lb, qc, Tb, rr, hbm, rank)}
        line["breakdown"] = bd

    if not args.no_cpu and world == 1 and rank == 0:
        tps, threads, el, desc = oracle_sample(cfg, T, n_cpu_tokens, 10.0)
        line["cpu_baseline"] = {"value": tps, "unit": UNIT, "cores": threads, "kind": "oracle",
                                "sample": desc, "seconds": el}
        # the same oracle on one thread (a single-threaded C loop over the tokens)
        import oracle
        oracle.set_num_threads(1)
        tps1, threads1, el1, desc1 = oracle_sample(cfg, T, 1, 5.0)
        oracle.set_num_threads(threads)
        line["cpu_baseline"]["single_thread"] = {"value": tps1, "unit": UNIT, "cores": threads1,
                                                 "sample": desc1, "seconds": el1}
    if rank == 0:
        print(json.dumps(line))
    if world > 1:
        torch.distributed.destroy_process_group()


if __name__ == "__main__":
    main()
