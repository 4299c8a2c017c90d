"""A stack of dense gated feed-forward blocks with FP8 weights and activations:

    r' = r + x;  X8 = fp8(rmsnorm(r') * g)      qmm_add_rmsnorm_fp8
    H8 = fp8(silu(X8 Wg^T) * (X8 Wu^T))         qmm_fp8a8_swiglu_blk128
    x' = H8 Wd^T                                qmm_fp8a8_blk128

    python examples/dense_ffn_fp8.py [--layers L] [--width D] [--ffn F] [--tokens T]

runs a prompt of T tokens and then single-token steps from a CUDA graph, checks the
prompt against the same blocks in plain fp32 torch on the dequantised weights, and
prints the times.  Weights are random.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_quantized_weight_route_gb300 as qmm  # noqa: E402

EPS = 1e-6


def quantize_blk128(w: torch.Tensor):
    """(E4M3 codes [N, K], fp32 scales [ceil(N/128), ceil(K/128)]) of a weight matrix."""
    N, K = w.shape
    b = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    b = b.view(b.shape[0] // 128, 128, b.shape[1] // 128, 128)
    s = b.abs().amax((1, 3)) / 448.0
    q = (b / s.clamp(min=1e-30)[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(q.shape[0] * 128, -1)[:N, :K].contiguous(), s


def dequantize_blk128(q: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    N, K = q.shape
    return q.float() * s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


class DenseFFN:
    """One block's weights: the norm's g, gate and up rows (gate first) and down rows."""

    def __init__(self, D: int, F: int, seed: int):
        gen = torch.Generator("cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")

        self.g = (1.0 + 0.1 * rand(D)).to(torch.bfloat16)
        self.Wgu, self.Sgu = quantize_blk128(rand(2 * F, D) / math.sqrt(D))
        self.Wd, self.Sd = quantize_blk128(rand(D, F) / math.sqrt(F))

    def __call__(self, x, r):
        """(the block's output, the residual stream with x added), both bf16 [T, D]; r in place."""
        n = qmm.qmm_add_rmsnorm_fp8(x, self.g, R=r, eps=EPS, Rout=r)
        Hq, Hs = qmm.qmm_fp8a8_swiglu_blk128(n["Q"], n["S"], self.Wgu, self.Sgu)
        return qmm.qmm_fp8a8_blk128(Hq, Hs, self.Wd, self.Sd, out_dtype=torch.bfloat16), r

    def plain(self, x, r):
        """The same in fp32 torch, activations not rounded to 8 bits."""
        r = (x.float() + r.float()).to(torch.bfloat16)
        v = r.float()
        n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * self.g.float()
        g, u = (n @ dequantize_blk128(self.Wgu, self.Sgu).t()).chunk(2, 1)
        return (torch.nn.functional.silu(g) * u) @ dequantize_blk128(self.Wd, self.Sd).t(), r


def run(layers, x, r):
    for f in layers:
        x, r = f(x, r)
    return x, r


def main(argv=None) -> float:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--width", type=int, default=5120)
    ap.add_argument("--ffn", type=int, default=17408)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args(argv)
    layers = [DenseFFN(a.width, a.ffn, seed) for seed in range(a.layers)]
    gen = torch.Generator("cuda").manual_seed(99)
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda").to(torch.bfloat16)
    r = torch.randn(a.tokens, a.width, generator=gen, device="cuda").to(torch.bfloat16)

    # the prompt, against plain torch
    y, _ = run(layers, x, r.clone())
    qmm.qmm_check_status()
    px, pr = x, r
    for f in layers:
        px, pr = f.plain(px, pr)
        px = px.to(torch.bfloat16)
    err = float((y.float() - px.float()).norm() / px.float().norm())

    def clock(f, n):
        f()
        a_, b_ = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a_.record()
        for _ in range(n):
            f()
        b_.record()
        torch.cuda.synchronize()
        return a_.elapsed_time(b_) / n

    buf = r.clone()
    prompt_ms = clock(lambda: run(layers, x, buf), 10)
    # single tokens: the blocks captured once, replayed for every step
    x1, r1 = x[:1].clone(), r[:1].clone()
    run(layers, x1, r1.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(layers, x1, r1)
    token_ms = clock(graph.replay, 50)
    qmm.qmm_check_status()
    print(f"{a.layers} blocks, width {a.width}, ffn {a.ffn}: prompt of {a.tokens} tokens {prompt_ms:.3f} ms, "
          f"one token {token_ms:.3f} ms; against fp32 activations rel {err:.3f}")
    return err


if __name__ == "__main__":
    main()
