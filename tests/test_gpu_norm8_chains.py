"""The 8-bit norms with the products that they feed, and the feed-forward example's graph."""
import os
import sys

import numpy as np
import pytest
import torch
from test_gpu_norm8 import formula, rows

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


@pytest.mark.parametrize("T,D,N,xt,rt", [(1, 256, 128, BF16, BF16), (37, 2048, 256, F32, BF16), (130, 512, 384, F32, None)])
def test_q8_1_rows_into_the_q8_0_product(q, T, D, N, xt, rt):
    """The product of the norm's q8_1 rows with Q8_0 weights.  Against its own operands: exact block
    dots, one rounding for each block's scaling and addition, (D/32 + 4) 2^-23 of the sum of magnitudes.  Against the
    unrounded rows: half a code step of each value, and the fp16 rounding of the block's d."""
    g = torch.Generator().manual_seed(T)
    X, R = rows(T, T, D, xt), rows(T + 1, T, D, rt, 2.0) if rt else None
    G = (1 + 0.3 * torch.randn(D, generator=g)).to(BF16).cuda()
    n = q.qmm_add_rmsnorm_q8_1(X, G, R=R)
    Wq = torch.randint(-127, 128, (N, D), generator=g, dtype=torch.int8).cuda()
    Wd = (0.01 * (1 + torch.rand(N, D // 32, generator=g))).half().cuda()
    Y = q.qmm_q8_0_q8_1(n["Yq"], n["Yd"], Wq, Wd.view(torch.int16), fp32_out=True)["Y"].double().cpu().numpy()
    q.qmm_check_status()
    w = (Wq.double() * Wd.double().repeat_interleave(32, 1)).cpu().numpy()
    d = n["Yd"].view(torch.float16).double().repeat_interleave(32, 1).cpu().numpy()
    x = n["Yq"].double().cpu().numpy() * d
    assert np.all(np.abs(Y - x @ w.T) <= (D // 32 + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))
    _, y = formula(X, G, R, 1e-6)
    off = 0.5 * d * (1 + 2.0 ** -10) + (2.0 ** -11 + 2.0 ** -17) * np.abs(y) + 2.0 ** -25 * 127
    assert np.all(np.abs(Y - y @ w.T) <= off @ np.abs(w).T + (D // 32 + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T))


def test_fp8_rows_into_the_product(q):
    """The norm's E4M3 rows through the product, against the unrounded rows: half a code step each."""
    T, D, N = 77, 640, 200
    g = torch.Generator().manual_seed(1)
    X, G = rows(1, T, D, BF16), torch.ones(D, device="cuda")
    n = q.qmm_add_rmsnorm_fp8(X, G)
    W = (torch.randn(N, D, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()
    S = (0.01 * (1 + torch.rand(-(-N // 128), D // 128, generator=g))).cuda()
    Y = q.qmm_fp8a8_blk128(n["Q"], n["S"], W, S, out_dtype=F32).double().cpu().numpy()
    w = (W.double() * S.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)).cpu().numpy()
    _, y = formula(X, G, None, 1e-6)
    s = n["S"].double().repeat_interleave(128, 1).cpu().numpy()
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y / s) * (1 + 2.0 ** -17), 1e-30))), -6) - 3)
    off = 0.5 * step * s + 2.0 ** -17 * np.abs(y)
    assert np.all(np.abs(Y - y @ w.T) <= off @ np.abs(w).T + (128 + 5 + 4) * 2.0 ** -23 * (np.abs(y) @ np.abs(w).T) * 1.1)


def test_the_examples_graph_gives_what_its_calls_give(q):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import dense_ffn_fp8 as m
    finally:
        sys.path.pop(0)
    layers = [m.DenseFFN(640, 384, seed) for seed in range(3)]
    g = torch.Generator("cuda").manual_seed(9)

    def fresh():
        return [torch.randn(1, 640, generator=g, device="cuda").to(BF16) for _ in range(2)]
    x, r = fresh()
    m.run(layers, x, r.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = m.run(layers, x, r)
    for _ in range(3):
        nx, nr = fresh()
        x.copy_(nx)
        r.copy_(nr)
        graph.replay()
        want, stream = m.run(layers, nx, nr)
        assert torch.equal(y, want) and torch.equal(r, stream)   # r: the residual stream, in place
