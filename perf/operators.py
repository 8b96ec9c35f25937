"""Timed cases of the FP8 operators around the MoE layer: the residual RMS norm with
an FP8 output, the FP8 quantiser, the FP8 matrix product with 128-block scales and the
FP8 shared expert.

FP8 here: E4M3 codes with one fp32 scale for 128 elements along the input dimension
of an activation row, or for a 128 x 128 block of a weight matrix. A block's scale is
m / 448, m its largest magnitude but at least 2^-100 ("pow2": the least power of two
not below that); a code is the nearest E4M3 value of v / scale, ties to even.
"""
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before the MoE layer of one decoded token: the layer's fp32 sum joins the bf16 stream
        {"name": "norm_t1", "op": "norm", "T": 1, "d": 4096, "x": "f32", "res": "bf16", "pow2": False},
        # the same over the largest prompt batch (16384 tokens)
        {"name": "norm_t16384", "op": "norm", "T": 16384, "d": 4096, "x": "f32", "res": "bf16", "pow2": False},
        # a first norm without a residual, a width that is no multiple of anything, power-of-two scales
        {"name": "norm_ragged", "op": "norm", "T": 333, "d": 1001, "x": "bf16", "res": "", "pow2": True},
        # activations of a prompt batch quantised by rows
        {"name": "quant_rows", "op": "quant", "rows": 4096, "cols": 4096, "src": "bf16", "block": 1, "pow2": False},
        # a shared expert's W1 quantised from fp32 when a model is loaded
        {"name": "quant_weight", "op": "quant", "rows": 2048, "cols": 4096, "src": "f32", "block": 128, "pow2": False},
        # one decoded token through a down projection, fp32 out
        {"name": "gemm_t1", "op": "gemm", "T": 1, "N": 4096, "K": 2048, "y": "f32"},
        # a decode batch of 64 requests through a square projection
        {"name": "gemm_t64", "op": "gemm", "T": 64, "N": 4096, "K": 4096, "y": "bf16"},
        # a prompt batch
        {"name": "gemm_t4096", "op": "gemm", "T": 4096, "N": 4096, "K": 4096, "y": "bf16"},
        # odd sizes everywhere
        {"name": "gemm_ragged", "op": "gemm", "T": 333, "N": 1003, "K": 1111, "y": "bf16"},
        # the shared expert for the decode batch, for a prompt batch, and at odd sizes
        {"name": "ffn_t8", "op": "ffn", "T": 8, "d": 4096, "F": 2048, "pow2": False},
        {"name": "ffn_t4096", "op": "ffn", "T": 4096, "d": 4096, "F": 2048, "pow2": False},
        {"name": "ffn_ragged", "op": "ffn", "T": 77, "d": 1000, "F": 700, "pow2": True},
    ]


def _log(rng, lo, hi):
    v = int(round(2.0 ** rng.uniform(torch.tensor(float(lo)).log2().item(), torch.tensor(float(hi)).log2().item())))
    if rng.random() < 0.5:  # half of the sizes are round, half are whatever came
        v = v // 64 * 64 if v >= 128 else v
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "ffn"])
    pow2 = rng.random() < 0.3
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "d": _log(rng, 64, 8192), "x": rng.choice(["f32", "bf16"]),
                "res": rng.choice(["", "bf16", "f32"]), "pow2": pow2}
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 64, 8192), "src": rng.choice(["f32", "bf16"]),
                "block": rng.choice([1, 128]), "pow2": pow2}
    if op == "gemm":
        return {"op": op, "T": _log(rng, 1, 4096), "N": _log(rng, 64, 4096), "K": _log(rng, 64, 4096),
                "y": rng.choice(["bf16", "f32"])}
    return {"op": op, "T": _log(rng, 1, 4096), "d": _log(rng, 64, 4096), "F": _log(rng, 64, 2048), "pow2": pow2}


# ----------------------------------------------------------------- inputs

def _quantise(v, block, pow2):
    """(codes, scales) of fp32 v [rows][cols] by 1 x 128 or 128 x 128 blocks; codes as E4M3."""
    r, c = v.shape
    nr, nc = -(-r // block), -(-c // 128)
    p = torch.nn.functional.pad(v, (0, nc * 128 - c, 0, nr * block - r)).view(nr, block, nc, 128)
    m = p.abs().amax(dim=(1, 3)).clamp_min(2.0 ** -100)
    s = m / 448.0
    if pow2:
        man, ex = torch.frexp(s)
        s = torch.ldexp(torch.ones_like(s), torch.where(man == 0.5, ex - 1, ex))
    q = (p / s[:, None, :, None]).clamp(-448.0, 448.0).view(nr * block, nc * 128)[:r, :c]
    return q.to(torch.float8_e4m3fn), s


def _held(codes):
    """The codes in rows of a multiple of 16 bytes, as the matrix products read them."""
    r, c = codes.shape
    p = torch.zeros(r, -(-c // 16) * 16, dtype=torch.uint8, device=codes.device)
    p[:, :c] = codes.view(torch.uint8)
    return p


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    up16 = lambda n: -(-n // 16) * 16  # noqa: E731
    up128 = lambda n: -(-n // 128)  # noqa: E731
    c, op = case, case["op"]
    s = {"case": c}
    if op == "norm":
        T, d = c["T"], c["d"]
        s["x"] = normal(T, d).to(_DT[c["x"]])
        s["res"] = (4 * normal(T, d) * (1 + 8 * (torch.rand(d, generator=g, device="cuda") < 0.01))).to(_DT[c["res"]]) if c["res"] else None
        s["w"] = (1 + 0.2 * normal(d)).to(torch.bfloat16)
        s["sum"] = new(T, d, dt=_DT[c["res"]]) if c["res"] else None
        s["y"] = new(T, d, dt=torch.bfloat16)
        s["q"], s["qs"] = new(T, up16(d), dt=torch.uint8), new(T, up128(d))
    elif op == "quant":
        r, k = c["rows"], c["cols"]
        s["v"] = ((0.02 if c["block"] == 128 else 1.0) * normal(r, k)).to(_DT[c["src"]])
        s["q"], s["qs"] = new(r, up16(k), dt=torch.uint8), new(-(-r // c["block"]), up128(k))
    elif op == "gemm":
        T, N, K = c["T"], c["N"], c["K"]
        a, s["as"] = _quantise(normal(T, K), 1, False)
        w, s["ws"] = _quantise(0.02 * normal(N, K), 128, False)
        s["a"], s["w"] = _held(a), _held(w)
        s["y"] = new(T, N, dt=_DT[c["y"]])
    else:
        T, d, F = c["T"], c["d"], c["F"]
        x, s["xs"] = _quantise(normal(T, d), 1, c["pow2"])
        s["x"] = _held(x)
        for n, shape in (("w1", (F, d)), ("w3", (F, d)), ("w2", (d, F))):
            w, s[n + "s"] = _quantise(0.02 * normal(*shape), 128, c["pow2"])
            s[n] = _held(w)
        s["y"] = new(T, d, dt=torch.bfloat16)
        s["work"] = new(T * up16(F) + 4 * T * up128(F) + 4096, dt=torch.uint8)
    return s


# ------------------------------------------------------------- plain forms

def _values(codes, scales, cols, block):
    """fp32 values of held codes and their scales."""
    v = codes[:, :cols].view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(block, 0)[: v.shape[0]] if block > 1 else scales
    return v * s.repeat_interleave(128, 1)[:, :cols]


def _plain(s):
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        v = s["x"].float()
        if s["res"] is not None:
            v = v + s["res"].float()
        n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * s["w"].float()
        q, qs = _quantise(n, 1, c["pow2"])
        out = {"y": n.to(torch.bfloat16), "q": q, "qs": qs}
        if s["res"] is not None:
            out["sum"] = v.to(s["res"].dtype)
        return out
    if op == "quant":
        q, qs = _quantise(s["v"].float(), c["block"], c["pow2"])
        return {"q": q, "qs": qs}
    if op == "gemm":
        a, w = _values(s["a"], s["as"], c["K"], 1), _values(s["w"], s["ws"], c["K"], 128)
        return (a @ w.t()).to(_DT[c["y"]])
    x = _values(s["x"], s["xs"], c["d"], 1)
    g = x @ _values(s["w1"], s["w1s"], c["d"], 128).t()
    u = x @ _values(s["w3"], s["w3s"], c["d"], 128).t()
    q, qs = _quantise(g / (1 + torch.exp(-g)) * u, 1, c["pow2"])
    h = q.float() * qs.repeat_interleave(128, 1)[:, : c["F"]]
    return (h @ _values(s["w2"], s["w2s"], c["F"], 128).t()).to(torch.bfloat16)


def _library(s):
    import routed_expert_ffn_05_b200 as M
    c, op = s["case"], s["case"]["op"]
    ty = {"bf16": M.MOE_T_BF16, "f32": M.MOE_T_F32, "": M.MOE_T_BF16}
    mode = M.MOE_SCALE_POW2 if c.get("pow2") else M.MOE_SCALE_F32
    if op == "norm":
        desc = M.make_norm(c["T"], c["d"], 1e-6, ty[c["x"]], ty[c["res"]], M.MOE_T_BF16, mode, ldq=s["q"].shape[1])
        M.moe_rms_norm(desc, s["x"], s["res"], s["w"], s["sum"], s["y"], s["q"], s["qs"])
        out = {"y": s["y"], "q": s["q"][:, : c["d"]].view(torch.float8_e4m3fn), "qs": s["qs"]}
        if s["res"] is not None:
            out["sum"] = s["sum"]
        return out
    if op == "quant":
        desc = M.make_fp8_quant(c["rows"], c["cols"], ty[c["src"]], c["block"], mode, ldq=s["q"].shape[1])
        M.moe_fp8_quantize(desc, s["v"], s["q"], s["qs"])
        return {"q": s["q"][:, : c["cols"]].view(torch.float8_e4m3fn), "qs": s["qs"]}
    if op == "gemm":
        desc = M.make_fp8_gemm(c["T"], c["N"], c["K"], ty[c["y"]], lda=s["a"].shape[1], ldw=s["w"].shape[1])
        M.moe_fp8_gemm(desc, s["a"], s["as"], s["w"], s["ws"], s["y"])
        return s["y"]
    desc = M.make_fp8_ffn(c["T"], c["d"], c["F"], M.MOE_T_BF16, mode, ldx=s["x"].shape[1], ld13=s["w1"].shape[1], ld2=s["w2"].shape[1])
    w = M.make_fp8_ffn_weights(s["w1"], s["w1s"], s["w3"], s["w3s"], s["w2"], s["w2s"])
    M.moe_shared_ffn_fp8(desc, w, s["x"], s["xs"], s["y"], s["work"])
    return s["y"]


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    c, op = case, case["op"]
    b = {"bf16": 2, "f32": 4, "": 0}
    blocks = lambda n: -(-n // 128)  # noqa: E731
    if op == "norm":
        n = c["T"] * c["d"]
        return {"bytes": n * (b[c["x"]] + 2 * b[c["res"]] + 2 + 1) + 4 * c["T"] * blocks(c["d"]) + 2 * c["d"], "flops": 6 * n}
    if op == "quant":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (b[c["src"]] + 1) + 4 * -(-c["rows"] // c["block"]) * blocks(c["cols"]), "flops": 3 * n}
    if op == "gemm":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": T * K + N * K + 4 * (T + blocks(N)) * blocks(K) + T * N * b[c["y"]], "flops": 2 * T * N * K}
    T, d, F = c["T"], c["d"], c["F"]
    return {"bytes": T * d + 3 * F * d + 4 * (T * blocks(d) + 3 * blocks(F) * blocks(d)) + 2 * T * d, "flops": 6 * T * F * d}


# ------------------------------------------------------- 64-bit definition

def _spread(m, cols):
    """A [rows][blocks] table as one value for each of the columns."""
    return m.index_select(1, torch.arange(cols, device=m.device) // 128)


def _block_max(v):
    """Largest magnitude of each 128 columns of a row (the last may hold fewer)."""
    return torch.stack([part.abs().max(dim=1).values for part in torch.split(v, 128, dim=1)], dim=1)


def _scale64(m, pow2):
    s = torch.maximum(m, torch.full_like(m, 2.0 ** -100)) / 448
    # the power of two is chosen on the 32-bit quotient, as the format says
    return torch.exp2(torch.ceil(torch.log2(s.float().double()))) if pow2 else s


def _e4m3(v):
    """Nearest E4M3 value in 64 bits, ties to the even mantissa."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(v / step) * step, -448, 448)


def _read64(codes, scales, cols, tall):
    v = codes[:, :cols].contiguous().view(torch.float8_e4m3fn).double()
    s = _spread(scales.double(), cols)
    return v * (s.index_select(0, torch.arange(v.shape[0], device=v.device) // 128) if tall else s)


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "norm":
        v = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        n = v / torch.sqrt(v.pow(2).sum(dim=1, keepdim=True) / c["d"] + 1e-6) * s["w"].double()
        qs = _scale64(_block_max(n), c["pow2"])
        out = {"y": n, "q": n / _spread(qs, c["d"]), "qs": qs}
        if s["res"] is not None:
            out["sum"] = v
        return out
    if op == "quant":
        v = s["v"].double()
        m = _block_max(v)
        if c["block"] == 128:
            m = torch.stack([part.max(dim=0).values for part in torch.split(m, 128, dim=0)], dim=0)
        qs = _scale64(m, c["pow2"])
        at = torch.arange(c["rows"], device=v.device) // c["block"]
        return {"q": v / _spread(qs, c["cols"]).index_select(0, at), "qs": qs}
    if op == "gemm":
        return torch.einsum("tk,nk->tn", _read64(s["a"], s["as"], c["K"], False), _read64(s["w"], s["ws"], c["K"], True))
    x = _read64(s["x"], s["xs"], c["d"], False)
    g = torch.einsum("tk,nk->tn", x, _read64(s["w1"], s["w1s"], c["d"], True))
    u = torch.einsum("tk,nk->tn", x, _read64(s["w3"], s["w3s"], c["d"], True))
    h = g * torch.sigmoid(g) * u
    hs = _spread(_scale64(_block_max(h), c["pow2"]), c["F"])
    return torch.einsum("tk,nk->tn", _e4m3(h / hs) * hs, _read64(s["w2"], s["w2s"], c["F"], True))
