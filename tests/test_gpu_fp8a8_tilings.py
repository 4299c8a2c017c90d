"""Every kernel form of the FP8 x FP8 products against the formulas in 64 bits, by a
given tiling (qmm_dbg_fp8a8_*): which one a shape takes follows from estimated times, so
shapes alone say little about what they test.  Tolerances: as in test_gpu_fp8a8.py.

Sizes: more than two tiles for each of the 76 pairs of SMs (phases, ring of scales and
staging across tiles), 11 K blocks (no multiple of the ring's 4 and 8) or 40 (past the
stages and the ring, also of a half or a third of them), ragged ends on every side.
"""
import numpy as np
import pytest
import torch
from test_gpu_fp8a8 import check_swiglu, formula, half_bf16_step, operands

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NONE = (0, 0, 0, 0)


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def pair(bn):
    return (1, bn, 0, 0)


def narrow(tn, cs):
    return (0, 0, tn, cs)


def check_product(q, ops, plan, dt, ref=None):
    y, tol = ref or formula(*ops)
    M, N = y.shape
    big = torch.full((M + 1, N), 7.0, dtype=dt, device="cuda")
    q.qmm_dbg_fp8a8_blk128(*ops, plan, out_dtype=dt, Y=big[:M])
    q.qmm_check_status()
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(y) + tol)
    assert np.all(np.abs(big[:M].double().cpu().numpy() - y) <= tol)
    assert bool((big[M] == 7).all())   # nothing behind the rows


def check_gated(q, ops, plan, ref=None):
    Hq, Hs = q.qmm_dbg_fp8a8_swiglu_blk128(*ops, plan)
    q.qmm_check_status()
    check_swiglu(Hq, Hs, *(ref or formula(*ops)))


@pytest.mark.parametrize("extra", [40, 37, 38])   # rows of 16-byte pitch; odd; even
@pytest.mark.parametrize("bn", [256, 192, 128])
def test_pair_product(q, bn, extra):
    M, K, N = 2500, 1296, 16 * bn + extra
    ops = operands(bn + extra, M, K, N)
    ref = formula(*ops)
    for dt in (F32, BF16):
        check_product(q, ops, (pair(bn), NONE, N), dt, ref)


def test_pair_gate_up(q):
    M, K, F = 2500, 1296, 17 * 128
    check_gated(q, operands(1, M, K, 2 * F), (pair(256), NONE, F))


@pytest.mark.parametrize("cs", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tn", [16, 32, 64, 128])
def test_narrow_product(q, tn, cs):
    M, K = 2 * tn + tn // 2 + 1, 5104
    for N in (300, 301):
        ops = operands(tn + cs, M, K, N)
        ref = formula(*ops)
        for dt in (F32, BF16):
            check_product(q, ops, (narrow(tn, cs), NONE, N), dt, ref)


@pytest.mark.parametrize("cs", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("tn", [16, 32, 64, 128])
def test_narrow_gate_up(q, tn, cs):
    M, K, F = 2 * tn + tn // 2 + 1, 5104, 256
    check_gated(q, operands(tn + cs, M, K, 2 * F), (narrow(tn, cs), NONE, F))


@pytest.mark.parametrize("second", [pair(256), pair(192), pair(128), narrow(16, 3), narrow(32, 1), narrow(64, 2), narrow(128, 3)])
@pytest.mark.parametrize("first,split", [(pair(256), 512), (pair(192), 768), (pair(128), 384), (narrow(128, 2), 256)])
def test_two_launches(q, first, split, second):
    M, K = 300, 656
    for N in (split + 320, split + 129):
        ops = operands(split, M, K, N)
        ref = formula(*ops)
        for dt in (F32, BF16):
            check_product(q, ops, (first, second, split), dt, ref)


@pytest.mark.parametrize("second", [pair(256), narrow(16, 3), narrow(32, 1), narrow(64, 2), narrow(128, 3)])
@pytest.mark.parametrize("first", [pair(256), narrow(128, 2)])
def test_two_launches_gate_up(q, first, second):
    M, K, F, split = 300, 656, 640, 256
    check_gated(q, operands(3, M, K, 2 * F), (first, second, split))


@pytest.mark.parametrize("M,K,N,gated,first", [
    (1, 5120, 5120, False, narrow(16, 0)),            # single token
    (300, 5120, 5120, False, narrow(128, 1)),
    (2048, 5120, 5120, False, pair(256)),             # prompts
    (5268, 17408, 5120, False, pair(256)),
    (1, 5120, 17408, True, narrow(16, 0)),
    (100, 5120, 17408, True, narrow(128, 0)),
    (2048, 5120, 17408, True, pair(256)),
])
def test_what_the_rule_takes(q, M, K, N, gated, first):
    """The kernel and tile that the sizes of the workloads take (cs 0 here: any split of K)."""
    got = q.qmm_dbg_fp8a8_plan(M, K, N, gated)
    assert got[0][:3] == first[:3] and (not first[3] or got[0][3] == first[3]), got
    if (M, N) == (2048, 5120):
        assert got[2] == 4864, got   # the 256 columns past two whole waves in a launch of their own


def test_the_rule_takes_only_what_is_tested_here(q):
    for gated in (False, True):
        for M in (1, 3, 17, 40, 65, 129, 200, 300, 513, 1000, 2048, 5268, 21504):
            for K in (16, 128, 400, 2000, 5120, 17408):
                for N in (128, 640, 1408, 5120, 17408):
                    first, second, split = q.qmm_dbg_fp8a8_plan(M, K, N, gated)
                    for pl in (first, second) if split < N else (first,):
                        if pl[0]:
                            assert pl[1] in ((256,) if gated else (128, 192, 256))
                        else:
                            assert pl[2] in (16, 32, 64, 128) and 1 <= pl[3] <= min(8, -(-K // 128))


def test_the_public_call_is_the_planned_one(q):
    for M, K, N in [(1, 5120, 1024), (100, 640, 512), (2048, 512, 5120)]:
        ops = operands(M, M, K, N)
        plan = q.qmm_dbg_fp8a8_plan(M, K, N)
        assert torch.equal(q.qmm_fp8a8_blk128(*ops, out_dtype=F32), q.qmm_dbg_fp8a8_blk128(*ops, plan, out_dtype=F32))


def test_tilings_that_do_not_fit_are_refused(q):
    ops = operands(0, 4, 256, 256)
    for plan in [((1, 64, 0, 0), NONE, 256), (narrow(8, 1), NONE, 256), (narrow(16, 3), NONE, 256), (narrow(16, 0), NONE, 256),
                 (pair(192), pair(128), 128), (pair(256), NONE, 128), (pair(256), NONE, 512), (pair(256), NONE, 0)]:
        with pytest.raises(q.QmmError, match="no such tiling"):
            q.qmm_dbg_fp8a8_blk128(*ops, plan)
    with pytest.raises(q.QmmError, match="no such tiling"):
        q.qmm_dbg_fp8a8_swiglu_blk128(*operands(0, 4, 256, 512), (pair(128), NONE, 256))
