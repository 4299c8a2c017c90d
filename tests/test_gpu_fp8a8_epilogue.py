"""qmm_fp8a8_epilogue_blk128 against the formula in 64 bits.

Tolerance: the product's (test_gpu_fp8a8), half a step for the bias' addition; an activation hands
an error on with a slope of at most 1.13 and adds 32 * 2^-24 of its argument (exponential, quotient, erfc, a
few ulp each); the residual's addition half a step, bf16 output half a bf16 step.
"""
import itertools

import numpy as np
import pytest
import torch
from test_gpu_fp8a8 import formula, half_bf16_step, operands

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def extras(seed, M, N, bias, res):
    """A bias and a residual of the product's size."""
    g = torch.Generator().manual_seed(seed + 1000)
    b = None if bias is None else (2 * torch.randn(N, generator=g)).to(bias).cuda()
    R = None if res is None else (3 * torch.randn(M, N, generator=g)).to(res).cuda()
    return b, R


def act64(v, act):
    t = torch.from_numpy(v)
    F = torch.nn.functional
    return {"none": lambda: t, "relu": lambda: F.relu(t), "silu": lambda: F.silu(t), "gelu": lambda: F.gelu(t),
            "gelu_tanh": lambda: F.gelu(t, approximate="tanh")}[act]().numpy()


def check(Y, ops, b, R, act, dt):
    y, tol = formula(*ops)
    if b is not None:
        y = y + b.double().cpu().numpy()
        tol = tol + 2.0 ** -24 * (np.abs(y) + tol)
    z = act64(y, act)
    if act not in ("none", "relu"):
        tol = 1.13 * tol + 32 * 2.0 ** -24 * np.abs(y)
    if R is not None:
        z = z + R.double().cpu().numpy()
        tol = tol + 2.0 ** -24 * (np.abs(z) + tol)
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(z) + tol)
    assert Y.dtype == dt and tuple(Y.shape) == z.shape
    assert np.all(np.abs(Y.double().cpu().numpy() - z) <= tol)


MS = [1, 2, 7, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513]
KS = [16, 128, 272, 1024, 2000, 400]
NS = [1, 8, 36, 127, 128, 130, 200, 256, 384, 1000, 1352, 999]
TYPES = [None, F32, BF16]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("i", range(36))
def test_epilogue(q, i, dt):
    M, K, N = MS[i % len(MS)], KS[i % len(KS)], NS[(5 * i) % len(NS)]
    ops = operands(i, M, K, N)
    bias, res, act = TYPES[i % 3], TYPES[(i // 3) % 3], ACTS[i % 5]
    b, R = extras(i, M, N, bias, res)
    Y = q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act=act, R=R, out_dtype=dt)
    q.qmm_check_status()
    check(Y, ops, b, R, act, dt)


PLANS = [(0, 0, tn, cs) for tn in (16, 32, 64, 128) for cs in (1, 2)] + [(1, bn, 0, 0) for bn in (128, 192, 256)]


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("N", [520, 517, 518])
def test_every_tiling(q, plan, N):
    M, K = 300, 640
    ops = operands(N, M, K, N)
    for n, (bias, res, dt) in enumerate(itertools.product(TYPES, TYPES, (F32, BF16))):
        b, R = extras(n, M, N, bias, res)
        act = ACTS[n % 5]
        Y = q.qmm_dbg_fp8a8_epilogue_blk128(*ops, (plan, (0, 0, 0, 0), N), bias=b, act=act, R=R, out_dtype=dt)
        q.qmm_check_status()
        check(Y, ops, b, R, act, dt)


def test_two_launches(q):
    """Columns of whole tiles in one launch, the rest in a second one, with bias and residual of their columns."""
    M, K, N = 300, 256, 700
    ops = operands(4, M, K, N)
    b, R = extras(4, M, N, F32, BF16)
    Y = q.qmm_dbg_fp8a8_epilogue_blk128(*ops, ((1, 256, 0, 0), (0, 0, 32, 2), 512), bias=b, act="silu", R=R, out_dtype=F32)
    q.qmm_check_status()
    check(Y, ops, b, R, "silu", F32)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 300])
def test_far_and_special_values(q, act, M):
    """Arguments from -200 to 200 by the bias alone, and NaN and infinities there."""
    N = 512
    ops = operands(1, M, 128, N)
    ops[1].zero_()   # the product is 0
    b = torch.linspace(-200, 200, N)
    b[5], b[6], b[7] = float("nan"), float("inf"), -float("inf")
    b[10], b[201] = float("nan"), -float("inf")   # (each beside a finite one)
    Y = q.qmm_fp8a8_epilogue_blk128(*ops, bias=b.cuda(), act=act, out_dtype=F32)
    q.qmm_check_status()
    want = act64(b.double().numpy(), act)
    y = Y.double().cpu().numpy()
    assert np.isnan(y[:, 5]).all() and (y[:, 6] == np.inf).all()
    assert (y[:, 7] == want[7]).all() or (np.isnan(want[7]) and np.isnan(y[:, 7]).all())
    keep = np.isfinite(b.numpy())
    assert np.all(np.abs(y - want)[:, keep] <= 32 * 2.0 ** -24 * np.abs(b.double().numpy())[keep])


@pytest.mark.parametrize("M,N", [(1, 512), (5, 130), (300, 512), (300, 301)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_the_residual_in_place_and_as_a_slice(q, M, N, dt):
    ops = operands(7, M, 256, N)
    b, R = extras(7, M, N, BF16, dt)
    want = q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act="silu", R=R, out_dtype=dt)
    x = R.clone()
    got = q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act="silu", R=x, out_dtype=dt, Y=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(x, want)
    for pitch, first in ((N + 24, 0), (N + 3, 1), (N + 8, 8)):   # rows that start at any element
        wide = torch.full((M + 1, pitch), 9.0, dtype=dt, device="cuda")
        wide[1:, first:first + N] = R if first + N <= pitch else R[:, :pitch - first]
        if first + N <= pitch:
            assert torch.equal(q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act="silu", R=wide[1:, first:first + N], out_dtype=dt), want)
    out = torch.full((M + 16, N), 9.0, dtype=dt, device="cuda")
    q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act="silu", R=R, out_dtype=dt, Y=out[8:8 + M])   # (rows of 8 are aligned)
    assert torch.equal(out[8:8 + M], want) and out[:8].eq(9).all() and out[8 + M:].eq(9).all()


def test_without_anything_to_add_it_is_the_product(q):
    ops = operands(3, 70, 512, 384)
    assert torch.equal(q.qmm_fp8a8_epilogue_blk128(*ops), q.qmm_fp8a8_blk128(*ops))
    empty = q.qmm_fp8a8_epilogue_blk128(ops[0][:0], ops[1][:0], ops[2], ops[3], act="silu")
    assert empty.shape == (0, 384)


def test_a_graph_and_another_stream(q):
    ops = operands(5, 33, 512, 256)
    b, R = extras(5, 33, 256, F32, BF16)
    call = lambda **kw: q.qmm_fp8a8_epilogue_blk128(*ops, bias=b, act="gelu", R=R, **kw)  # noqa: E731
    want = call()
    Y = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(Y=Y)
    s.synchronize()
    assert torch.equal(Y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(Y=Y)
    R.add_(1.0)
    want = call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_refusals(q):
    ops = operands(6, 4, 128, 64)
    with pytest.raises(ValueError):
        q.qmm_fp8a8_epilogue_blk128(*ops, act="tanh")
    with pytest.raises(ValueError):
        q.qmm_fp8a8_epilogue_blk128(*ops, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(TypeError):
        q.qmm_fp8a8_epilogue_blk128(*ops, bias=torch.zeros(64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        q.qmm_fp8a8_epilogue_blk128(*ops, R=torch.zeros(64, 4, device="cuda").t())
    with pytest.raises(ValueError):
        q.qmm_fp8a8_epilogue_blk128(*ops, R=torch.zeros(3, 64, device="cuda"))
    with pytest.raises(q.QmmError):   # a broadcast row has no pitch
        q.qmm_fp8a8_epilogue_blk128(*ops, R=torch.zeros(64, device="cuda").expand(4, 64))
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(q.QmmError):   # in place, of another type
        q.qmm_fp8a8_epilogue_blk128(*ops, R=x, Y=x.view(-1)[:128].view(BF16).view(4, 64))
