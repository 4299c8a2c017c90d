"""Cases of the 8-bit feed-forward operators: the residual's addition with an RMS norm and an output
in 8 bits, the FP8 x FP8 product with block scales, and the gate/up product with SwiGLU and an output
in 8 bits.  Sizes are those of this repository's workloads (K = 5120 with N = 5120 and 17408, D = 2048
and 2560, F = 768, prompts of 2048, 5268 and 21504 tokens) and of single-token decoding.

`own` false: plain torch operations in 32 bits; `own` true: the library's calls."""
import math

import torch

own = False

EPS = 1e-6
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one token of a decode step: the norm in front of a layer's projections; latency is what counts
        {"name": "norm_fp8_t1", "op": "norm", "out": "fp8", "T": 1, "D": 5120, "x": "bf16", "r": "bf16", "g": "bf16", "y": False},
        # a ragged batch of decode tokens, the first norm of a model (no residual yet), width not a multiple of 128
        {"name": "norm_fp8_t37_d2000", "op": "norm", "out": "fp8", "T": 37, "D": 2000, "x": "bf16", "r": "", "g": "f32", "y": False},
        # a 5268-token prompt behind the expert stage (fp32 rows), feeding the Q8_0 x q8_1 projections
        {"name": "norm_q8_1_t5268", "op": "norm", "out": "q8_1", "T": 5268, "D": 2048, "x": "f32", "r": "bf16", "g": "bf16", "y": False},
        # the largest prompt, fp32 expert output and fp32 residual stream, with the bf16 rows for the router beside the codes
        {"name": "norm_fp8_t21504", "op": "norm", "out": "fp8", "T": 21504, "D": 2560, "x": "f32", "r": "f32", "g": "bf16", "y": True},
        # one token against a square projection: the weights' bytes are all there is
        {"name": "gemm_m1", "op": "gemm", "M": 1, "K": 5120, "N": 5120, "y": "bf16"},
        # a small batch against a ragged projection (neither N nor K a multiple of 128), fp32 out
        {"name": "gemm_m19_ragged", "op": "gemm", "M": 19, "K": 2000, "N": 1000, "y": "f32"},
        # a batch of short prompts: too few rows to fill the card with full tiles
        {"name": "gemm_m300", "op": "gemm", "M": 300, "K": 5120, "N": 5120, "y": "bf16"},
        # a prompt against the square projection
        {"name": "gemm_m2048", "op": "gemm", "M": 2048, "K": 5120, "N": 5120, "y": "bf16"},
        # the largest: the down product of a long prompt
        {"name": "gemm_m5268_down", "op": "gemm", "M": 5268, "K": 17408, "N": 5120, "y": "bf16"},
        # one token through gate and up: 178 MB of weights
        {"name": "swiglu_m1", "op": "swiglu", "M": 1, "K": 5120, "F": 17408},
        # a small prompt through a narrow feed-forward (the expert stage's widths)
        {"name": "swiglu_m131_narrow", "op": "swiglu", "M": 131, "K": 2048, "F": 768},
        # a prompt through gate and up
        {"name": "swiglu_m2048", "op": "swiglu", "M": 2048, "K": 5120, "F": 17408},
    ]


def _log(rng, lo, hi, step=1):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(["norm", "gemm", "swiglu"])
    if op == "norm":
        out = rng.choice(["fp8", "fp8", "q8_1"])
        return {"op": op, "out": out, "T": _log(rng, 1, 21504), "D": _log(rng, 256, 8192, 16 if out == "fp8" else 32) if rng.random() < 0.7 else rng.choice([2048, 2560, 5120]),
                "x": rng.choice(["bf16", "f32"]), "r": rng.choice(["", "bf16", "f32"]), "g": rng.choice(["bf16", "f32"]), "y": rng.random() < 0.3}
    while True:
        M, K = _log(rng, 1, 8192), _log(rng, 256, 17408, 16) if rng.random() < 0.7 else rng.choice([2048, 2560, 5120])
        if op == "gemm":
            N = _log(rng, 64, 17408)
            if 2.0 * M * N * K <= 9e11:
                return {"op": op, "M": M, "K": K, "N": N, "y": rng.choice(["bf16", "f32"])}
        else:
            F = _log(rng, 128, 17408, 128)
            if 4.0 * M * F * K <= 7e11 and F * K <= 17408 * 5120:
                return {"op": op, "M": M, "K": K, "F": F}


def work(case):
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        size = {"bf16": 2, "f32": 4, "": 0}
        b = T * D * (size[case["x"]] + 2 * size[case["r"]] + 1 + (2 if case["y"] else 0)) + D * size[case["g"]]
        b += T * (-(-D // 128) * 4 if case["out"] == "fp8" else D // 32 * 4)
        return {"bytes": b, "flops": 6.0 * T * D}
    M, K = case["M"], case["K"]
    kb = -(-K // 128)
    if case["op"] == "gemm":
        N = case["N"]
        return {"bytes": (M + N) * K + 4 * kb * (M + -(-N // 128)) + M * N * (2 if case["y"] == "bf16" else 4), "flops": 2.0 * M * N * K}
    F = case["F"]
    return {"bytes": (M + 2 * F) * K + 4 * kb * (M + F // 64) + M * F + 4 * M * (F // 128), "flops": 4.0 * M * F * K}


def _pad(t, n, dim=-1):
    """t with zeros up to a multiple of n along dim."""
    k = -t.shape[dim] % n
    if not k:
        return t
    shape = list(t.shape)
    shape[dim] = k
    return torch.cat([t, torch.zeros(shape, dtype=t.dtype, device=t.device)], dim)


def _quant_rows(y):
    """(e4m3 codes, fp32 scales) of y's rows per 128 columns; s = max|y| / 448."""
    T, D = y.shape
    b = _pad(y, 128).view(T, -1, 128)
    s = b.abs().amax(-1) / 448.0
    q = (b / torch.where(s == 0, torch.ones_like(s), s)[..., None]).clamp(-448.0, 448.0)
    return q.to(F8).view(T, -1)[:, :D], s


def _quant_blocks(w):
    """(e4m3 codes, fp32 scales) of a weight matrix per block of 128 x 128."""
    N, K = w.shape
    b = _pad(_pad(w, 128), 128, 0)
    b = b.view(b.shape[0] // 128, 128, b.shape[1] // 128, 128)
    s = b.abs().amax((1, 3)) / 448.0
    q = (b / s[:, None, :, None]).clamp(-448.0, 448.0).to(F8)
    return q.view(q.shape[0] * 128, -1)[:N, :K].contiguous(), s


def _hidden(gen, T, D):
    """Rows as a residual stream has them: tokens of different size, some channels far larger than the rest."""
    channel = torch.ones(D, device="cuda")
    channel[torch.randint(0, D, (max(1, D // 256),), generator=gen, device="cuda")] = 20.0
    token = torch.exp(0.5 * torch.randn(T, 1, generator=gen, device="cuda"))
    return torch.randn(T, D, generator=gen, device="cuda") * token * channel


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    if case["op"] == "norm":
        T, D = case["T"], case["D"]
        st = {"op": "norm", "out": case["out"], "y": case["y"], "X": _hidden(gen, T, D).to(_TYPES[case["x"]]), "R": None, "Rout": None}
        if case["r"]:
            st["R"] = (2.0 * _hidden(gen, T, D)).to(_TYPES[case["r"]])
            st["Rout"] = torch.empty_like(st["R"])
        st["G"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(_TYPES[case["g"]])
        st["Y"] = torch.empty((T, D), dtype=BF16, device="cuda") if case["y"] else None
        if case["out"] == "fp8":
            st["Q"] = torch.empty((T, D), dtype=F8, device="cuda")
            st["S"] = torch.empty((T, -(-D // 128)), dtype=F32, device="cuda")
        return st
    M, K = case["M"], case["K"]
    Xq, Xs = _quant_rows(_hidden(gen, M, K))
    N = case["N"] if case["op"] == "gemm" else 2 * case["F"]
    W, S = _quant_blocks(torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K))
    st = {"op": case["op"], "Xq": Xq.contiguous(), "Xs": Xs, "W": W, "S": S}
    if case["op"] == "gemm":
        st["Y"] = torch.empty((M, N), dtype=_TYPES[case["y"]], device="cuda")
    else:
        st["Hq"] = torch.empty((M, N // 2), dtype=F8, device="cuda")
        st["Hs"] = torch.empty((M, N // 256), dtype=F32, device="cuda")
    return st


def _plain_norm(st):
    v = st["X"].float()
    out = {}
    if st["R"] is not None:
        out["r"] = (v + st["R"].float()).to(st["R"].dtype)
        v = out["r"].float()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * st["G"].float()
    if st["y"]:
        out["y"] = y.to(BF16)
    if st["out"] == "fp8":
        out["q"], out["s"] = _quant_rows(y)
        return out
    T, D = y.shape
    b = y.view(T, D // 32, 32)
    d = b.abs().amax(-1) / 127.0
    t = b / torch.where(d == 0, torch.ones_like(d), d)[..., None]
    q = (torch.sign(t) * torch.floor(t.abs() + 0.5)).clamp(-127.0, 127.0)
    out["d"], out["s"] = d.half(), (d * q.sum(-1)).half()
    out["v"] = (q * out["d"].float()[..., None]).half()
    return out


def _dequant(st, dtype):
    """Activations and weights as the values that their codes and scales stand for."""
    M, K = st["Xq"].shape
    N = st["W"].shape[0]
    x = st["Xq"].to(dtype) * st["Xs"].to(dtype).repeat_interleave(128, 1)[:, :K]
    w = st["W"].to(dtype) * st["S"].to(dtype).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x, w


def run(st):
    if not own:
        if st["op"] == "norm":
            return _plain_norm(st)
        x, w = _dequant(st, F32)
        y = x @ w.t()
        if st["op"] == "gemm":
            return y.to(st["Y"].dtype)
        g, u = y.chunk(2, 1)
        q, s = _quant_rows(g / (1.0 + torch.exp(-g)) * u)
        return {"q": q, "s": s}
    import block_quantized_weight_route_gb300 as qmm
    if st["op"] == "gemm":
        return qmm.qmm_fp8a8_blk128(st["Xq"], st["Xs"], st["W"], st["S"], out_dtype=st["Y"].dtype, Y=st["Y"])
    if st["op"] == "swiglu":
        Hq, Hs = qmm.qmm_fp8a8_swiglu_blk128(st["Xq"], st["Xs"], st["W"], st["S"], Hq=st["Hq"], Hs=st["Hs"])
        return {"q": Hq, "s": Hs}
    if st["out"] == "fp8":
        got = qmm.qmm_add_rmsnorm_fp8(st["X"], st["G"], R=st["R"], eps=EPS, Rout=st["Rout"], Q=st["Q"], S=st["S"], Y=st["Y"])
        out = {"q": got["Q"], "s": got["S"]}
    else:
        got = qmm.qmm_add_rmsnorm_q8_1(st["X"], st["G"], R=st["R"], eps=EPS, Rout=st["Rout"], Y=st["Y"])
        d = got["Yd"].view(torch.float16)
        # the values that the codes stand for: code times its block's d
        out = {"v": got["Yq"].view(d.shape[0], d.shape[1], 32) * d[..., None], "d": d, "s": got["Ys"].view(torch.float16)}
    if st["R"] is not None:
        out["r"] = got["R"]
    if st["y"]:
        out["y"] = got["Y"]
    return out


def _exact_groups(y, n):
    """(max|.| per n columns of each row, the rows in groups of n), zeros behind a short last group."""
    T, D = y.shape
    full = torch.zeros((T, -(-D // n) * n), dtype=torch.float64, device=y.device)
    full[:, :D] = y
    full = full.reshape(T, -1, n)
    return full.abs().max(-1).values, full


def exact(case, seed):
    """In 64 bits from the definitions.  Codes come unrounded: y / s."""
    st = prepare(case, seed)
    f64 = torch.float64
    if st["op"] == "norm":
        v = st["X"].to(f64)
        out = {}
        if st["R"] is not None:
            v = v + st["R"].to(f64)
            out["r"] = v
            v = v.to(st["R"].dtype).to(f64)  # the norm is of the stored sum
        D = v.shape[1]
        y = v / (v.pow(2).sum(1, keepdim=True) / D + EPS).sqrt() * st["G"].to(f64)
        if st["y"]:
            out["y"] = y
        if st["out"] == "fp8":
            top, full = _exact_groups(y, 128)
            out["s"] = top / 448
            out["q"] = (full * (448 / top)[..., None]).reshape(y.shape[0], -1)[:, :D].contiguous()
        else:
            top, full = _exact_groups(y, 32)
            out["d"], out["v"] = top / 127, full
            t = full * (127 / top)[..., None]
            out["s"] = top / 127 * torch.where(t < 0, -torch.floor(0.5 - t), torch.floor(0.5 + t)).sum(-1)
        return out
    M, K = st["Xq"].shape
    N = st["W"].shape[0]
    y = torch.zeros((M, N), dtype=f64, device="cuda")
    for n in range(0, N, 128):  # one block of weight rows at a time, its scales on the products' sums
        w = st["W"][n:n + 128].to(f64)
        scale = st["S"][n // 128].to(f64)
        x = st["Xq"].to(f64)
        for k in range(0, K, 128):
            x[:, k:k + 128] *= (st["Xs"][:, k // 128].to(f64) * scale[k // 128])[:, None]
        y[:, n:n + 128] = x @ w.t()
    if st["op"] == "gemm":
        return y
    F = N // 2
    h = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:]
    top, full = _exact_groups(h, 128)
    return {"q": (full * (448 / top)[..., None]).reshape(M, F), "s": top / 448}
