"""The 8-bit operators on slices of a batch's tokens.  The codes' rows are multiples of 16 bytes, their
scales' are not: with 768 columns a row of scales is 24 bytes, with 640 it is 20."""
import pytest
import torch
from test_gpu_fp8a8 import operands

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("K", [128, 640, 768])
@pytest.mark.parametrize("part", [slice(1, 2), slice(1, 6), slice(3, 9)])
def test_products(q, K, part):
    Xq, Xs, W, S = operands(K, 9, K, 512)
    whole = [t[part].clone() for t in (Xq, Xs)]
    assert Xs[part].data_ptr() % 16, "the slice is to start off a multiple of 16 bytes"
    ref = q.qmm_fp8a8_blk128(*whole, W, S, out_dtype=F32)
    assert torch.equal(q.qmm_fp8a8_blk128(Xq[part], Xs[part], W, S, out_dtype=F32), ref)
    # weights from the second block of 128 rows on
    ref = q.qmm_fp8a8_blk128(*whole, W[128:].clone(), S[1:].clone(), out_dtype=F32)
    assert torch.equal(q.qmm_fp8a8_blk128(Xq[part], Xs[part], W[128:], S[1:], out_dtype=F32), ref)
    hq, hs = q.qmm_fp8a8_swiglu_blk128(*whole, W, S)
    out_q, out_s = torch.zeros((9, 256), dtype=F8, device="cuda"), torch.full((9, 2), 7.0, device="cuda")
    got = q.qmm_fp8a8_swiglu_blk128(Xq[part], Xs[part], W, S, Hq=out_q[part], Hs=out_s[part])
    assert got[0].data_ptr() == out_q[part].data_ptr() and got[1].data_ptr() == out_s[part].data_ptr()
    assert same(out_q[part], hq) and torch.equal(out_s[part], hs)
    rest = [i for i in range(9) if i not in range(9)[part]]
    assert bool((out_s[rest] == 7).all()) and not out_q[rest].float().any()


@pytest.mark.parametrize("D", [128, 640, 768])
def test_norm_into_a_slice(q, D):
    g = torch.Generator().manual_seed(D)
    X, G = torch.randn(7, D, generator=g).to(BF16).cuda(), torch.ones(D, device="cuda")
    ref = q.qmm_add_rmsnorm_fp8(X, G)
    Q, S = torch.zeros((9, D), dtype=F8, device="cuda"), torch.full((9, D // 128), 7.0, device="cuda")
    assert S[1:8].data_ptr() % 16
    got = q.qmm_add_rmsnorm_fp8(X, G, Q=Q[1:8], S=S[1:8])
    assert got["S"].data_ptr() == S[1:8].data_ptr()
    assert same(Q[1:8], ref["Q"]) and torch.equal(S[1:8], ref["S"])
    assert bool((S[[0, 8]] == 7).all())


def test_slices_in_a_graph(q):
    """The copies are part of the call: a graph replayed on other values sees them."""
    Xq, Xs, W, S = operands(1, 4, 768, 256)
    Y, Hs = torch.zeros((3, 256), device="cuda"), torch.zeros((5, 1), device="cuda")
    Hq = torch.zeros((3, 128), dtype=F8, device="cuda")

    def call():
        q.qmm_fp8a8_blk128(Xq[1:], Xs[1:], W, S, out_dtype=F32, Y=Y)
        q.qmm_fp8a8_swiglu_blk128(Xq[1:], Xs[1:], W, S, Hq=Hq, Hs=Hs[1:4])
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for a, b in zip((Xq, Xs, W, S), operands(2, 4, 768, 256)):
        a.copy_(b)
    graph.replay()
    rows = Xq[1:].clone(), Xs[1:].clone()
    assert torch.equal(Y, q.qmm_fp8a8_blk128(*rows, W, S, out_dtype=F32))
    hq, hs = q.qmm_fp8a8_swiglu_blk128(*rows, W, S)
    assert same(Hq, hq) and torch.equal(Hs[1:4], hs) and not Hs[[0, 4]].any()
