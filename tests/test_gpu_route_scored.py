"""moe_route_scored against the formulas in 64 bits.

The ids have to be equal.  Tolerance of a weight: an fp32 exponential is within 2 ulp and its
argument, a difference, within half an ulp of itself; with the sum of up to 512 terms (16 and
then 5 levels), the quotients and the factor that is (48 + |l - max|) * 2^-23 relative.
"""
import itertools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def formula(l, k, score="softmax", bias=None, groups=1, groups_kept=1, group_top=2, renorm=True, scale=1.0):
    """(ids, w) of one token's logits, in 64 bits: a stable sort."""
    l = l.astype(np.float64)
    on = l > -np.inf
    with np.errstate(all="ignore"):
        if score == "softmax":
            top = l[on].max() if on.any() else 0.0
            e = np.where(on, np.exp(l - top), 0.0)
            s = e / e.sum()
        else:
            s = np.where(on, 1.0 / (1.0 + np.exp(-l)), 0.0)
        c = s if bias is None else s + bias.astype(np.float64)
    if bias is None and groups == 1 or bias is None and group_top == 1:
        c = l.copy()   # (grows with the score, and never ties where the score does not)
    c = np.where(on & ~np.isnan(c), c, -np.inf)
    if groups > 1:
        g = c.reshape(groups, -1)
        gs = -np.sort(-g, axis=1)[:, :group_top].sum(1)
        kept = np.argsort(-gs, kind="stable")[:groups_kept]
        c = np.where(np.isin(np.arange(groups), kept)[:, None], g, -np.inf).reshape(-1)
    ids = [e for e in np.argsort(-c, kind="stable") if c[e] > -np.inf][:k]
    w = s[ids]
    if renorm and ids:
        # the ratio of the exact scores: log s relative to its largest
        logs = l[ids] if score == "softmax" else l[ids] - np.logaddexp(0.0, l[ids])
        w = np.exp(logs - logs.max())
        w = w / w.sum()
    pad = k - len(ids)
    return np.array(list(ids) + [-1] * pad), np.concatenate([w * scale, np.zeros(pad)])


def check(q, logits, k, live=None, tol_of=None, **kw):
    """The call against the formula, token by token; returns (ids, w)."""
    ids, w = q.moe_route_scored(logits, k, live=live, **kw)
    q.qmm_check_status()
    T = logits.shape[0]
    l = logits.float().cpu().numpy()
    l = np.where(np.isnan(l), -np.inf, l)
    n = T if live is None else min(max(int(live), 0), T)
    args = dict(kw, bias=None if kw.get("bias") is None else kw["bias"].cpu().numpy())
    gi, gw = ids.cpu().numpy(), w.double().cpu().numpy()
    assert gi.shape == gw.shape == (T, k)
    for t in range(n):   # (a row of -inf: its differences are not used)
        ri, rw = formula(l[t], k, **args)
        assert np.array_equal(gi[t], ri), (t, gi[t], ri)
        on = ri >= 0
        top = l[t].max()
        tol = (48 + np.where(on, np.abs(top - np.where(on, l[t][ri], 0.0)) if on.any() else 0.0, 0.0)) * 2.0 ** -23 * np.abs(rw) + 2.0 ** -140
        assert np.all(np.abs(gw[t] - rw) <= tol), (t, gw[t], rw)
    assert np.all(gi[n:] == -1) and np.all(gw[n:] == 0)
    return ids, w


ES = [1, 2, 7, 31, 32, 33, 60, 64, 100, 128, 160, 256, 300, 511, 512]


@pytest.mark.parametrize("score,use_bias,renorm,dt", list(itertools.product(["softmax", "sigmoid"], [False, True], [False, True], [F32, BF16])))
def test_top_k(q, score, use_bias, renorm, dt):
    for i, E in enumerate(ES):
        g = torch.Generator().manual_seed(E)
        T, k = [1, 3, 33, 130, 700][i % 5], min(E, [1, 8, 16, 2, 5][(i // 2) % 5])
        logits = (2 * torch.randn(T, E, generator=g)).to(dt).cuda()
        bias = (0.2 * torch.randn(E, generator=g)).cuda() if use_bias else None
        check(q, logits, k, score=score, bias=bias, renorm=renorm, scale=[1.0, 2.5][i % 2])


@pytest.mark.parametrize("E,groups,kept,k", [(8, 2, 1, 4), (8, 4, 2, 3), (256, 8, 4, 8), (160, 5, 3, 6), (512, 32, 5, 16), (96, 32, 32, 7), (60, 3, 2, 16),
                                             (64, 16, 1, 4), (12, 6, 6, 12), (256, 2, 1, 1)])
@pytest.mark.parametrize("score,use_bias,top", list(itertools.product(["softmax", "sigmoid"], [False, True], [1, 2])))
def test_groups(q, E, groups, kept, k, score, use_bias, top):
    g = torch.Generator().manual_seed(E + groups)
    logits = (1.5 * torch.randn(137, E, generator=g)).cuda()
    bias = (0.2 * torch.randn(E, generator=g)).cuda() if use_bias else None
    check(q, logits, k, score=score, bias=bias, groups=groups, groups_kept=kept, group_top=top, scale=2.5)


@pytest.mark.parametrize("E,groups,kept", [(64, 1, 1), (256, 1, 1), (256, 8, 4), (500, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_32_bits_tell(q, E, groups, kept, score):
    """A bias that brings every expert's sum to the same number but for its own rounding."""
    for seed in range(6):
        g = torch.Generator().manual_seed(seed)
        l = 2 * torch.randn(1, E, generator=g)
        s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        bias = (0.5 - s)[0].float()
        check(q, l.cuda(), min(8, E // groups * kept), score=score, bias=bias.cuda(), groups=groups, groups_kept=kept)


@pytest.mark.parametrize("top,use_bias", [(1, True), (2, False), (2, True)])
@pytest.mark.parametrize("E,groups,kept", [(64, 8, 3), (256, 8, 4), (512, 16, 5), (90, 6, 1)])
def test_groups_closer_than_32_bits_tell(q, E, groups, kept, top, use_bias):
    """Every group's score is the same but for the rounding of its one or two largest logits; the rest are far below."""
    g = torch.Generator().manual_seed(E + top)
    T, size = 40, E // groups
    l = -6 + 0.1 * torch.randn(T, groups, size, generator=g, dtype=torch.float64)
    at = torch.rand(T, groups, size, generator=g).argsort(2)[:, :, :2]
    d = 0.2 * torch.rand(T, groups, generator=g, dtype=torch.float64) if top == 2 else 1e-8 * torch.rand(T, groups, generator=g, dtype=torch.float64)
    l.scatter_(2, at, torch.logit(torch.stack([0.7 + d, 0.6 - d], 2)))
    bias = (torch.full((E,), 0.125) if use_bias else torch.zeros(E)).cuda() if use_bias or top == 1 else None
    check(q, l.reshape(T, E).float().cuda(), min(2 * kept, 8), score="sigmoid", bias=bias, groups=groups, groups_kept=kept, group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("use_bias", [False, True])
def test_ties_go_to_the_lower_index(q, score, use_bias):
    for E, groups, kept in ((40, 1, 1), (256, 8, 4), (512, 1, 1)):
        g = torch.Generator().manual_seed(E)
        logits = torch.randint(-2, 3, (50, E), generator=g).float()
        logits[0] = 0.0
        logits[1] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)
        bias = (torch.randint(0, 2, (E,), generator=g) * 0.25).cuda() if use_bias else None
        check(q, logits.cuda(), 8, score=score, bias=bias, groups=groups, groups_kept=kept)


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_experts_that_are_off(q, score, renorm):
    E, k = 48, 6
    g = torch.Generator().manual_seed(5)
    logits = 2 * torch.randn(40, E, generator=g)
    logits[0] = -float("inf")                              # nothing left
    logits[1, 1:] = -float("inf")                          # one left
    logits[2, torch.arange(E) % 10 != 3] = float("nan")    # five left, NaN in the rest
    logits[3, ::2] = float("nan")
    logits[4] = torch.finfo(F32).min                       # a mask of the type's lowest value, everywhere
    logits[5, 4:] = torch.finfo(F32).min
    logits[6, :40] = torch.finfo(torch.bfloat16).min
    logits[7] = -200 - torch.arange(E).float()             # scores that underflow: renormalised they are ratios all the same
    logits[8] = 200 + torch.arange(E).float() / 2
    logits[9:, torch.randperm(E, generator=g)[:20]] = -float("inf")
    bias = 0.1 * torch.randn(E, generator=g)
    bias[7], bias[8] = float("nan"), -float("inf")
    one = dict(score=score, renorm=renorm)
    finite = [t for t in range(40) if renorm or t not in (7, 8) or score == "softmax"]
    check(q, logits[finite].cuda(), k, **one)
    rows = [t for t in range(40) if t not in (4, 5, 6, 7, 8)]   # (with a bias far scores are equal in 64 bits)
    check(q, logits[rows].cuda(), k, bias=bias.cuda(), **one)
    check(q, logits[rows].cuda(), k, bias=bias.cuda(), groups=4, groups_kept=2, **one)
    ids, w = q.moe_route_scored(logits.cuda(), k, bias=bias.cuda(), groups=4, groups_kept=3, **one)
    i = ids.cpu()
    assert bool(((i >= -1) & (i < E)).all()) and not bool(((i == 7) | (i == 8)).any())
    assert bool(torch.isfinite(w).all())


def test_infinite_logits(q):
    logits = torch.randn(3, 64)
    logits[0, 5] = logits[1, 9] = logits[1, 3] = float("inf")
    ids, w = q.moe_route_scored(logits.cuda(), 4, score="sigmoid")
    assert ids[0, 0] == 5 and ids[1, :2].tolist() == [3, 9] and bool(torch.isfinite(w).all())
    ids, w = q.moe_route_scored(logits.cuda(), 4, score="softmax")
    assert ids[0, 0] == 5 and bool(w[:2].isnan().any(1).all()) and bool(torch.isfinite(w[2]).all())
    ids, w = q.moe_route_scored(logits.cuda(), 4, score="softmax", bias=torch.zeros(64, device="cuda"))
    assert ids[:2].eq(-1).all() and w[:2].eq(0).all() and ids[2].ge(0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kept,k", [(1, 2), (2, 6), (3, 16)])
def test_infinite_biases_beside_groups_that_tie(q, score, kept, k):
    g = torch.Generator().manual_seed(k)
    logits = torch.randn(40, 64, generator=g)
    logits[:, 16:32] = logits[:, :16]   # (groups 0 and 1 tie)
    for off in [(33, 40), (33, 40, 50), (33, 40, 50, 51)]:
        bias = torch.full((64,), 0.25)
        bias[list(off)] = float("inf")
        check(q, logits.cuda(), k, score=score, bias=bias.cuda(), groups=4, groups_kept=kept, group_top=2)
        check(q, logits.cuda(), k, score=score, bias=bias.cuda(), groups=4, groups_kept=kept, group_top=1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kept,k", [(1, 2), (2, 6)])
def test_sums_of_a_group_beyond_32_bits(q, score, sign, kept, k):
    logits = torch.randn(40, 64, generator=torch.Generator().manual_seed(k))
    bias = sign * torch.tensor([2.0e38, 2.5e38, 3.0e38, 2.2e38]).repeat_interleave(16)
    check(q, logits.cuda(), k, score=score, bias=bias.cuda(), groups=4, groups_kept=kept, group_top=2)
    bias[:48] = sign * 1.7014118e38   # (their sums are the largest number, or round to it or past it)
    bias[16:32] = sign * 1.7014117e38
    check(q, logits.cuda(), k, score=score, bias=bias.cuda(), groups=4, groups_kept=kept, group_top=2)


@pytest.mark.parametrize("E,groups", [(32, 32), (64, 32), (24, 24), (33, 11)])
@pytest.mark.parametrize("at", [100.0, -3000.0])
def test_large_biases_of_single_experts(q, E, groups, at):
    """Groups decided by one expert, whose sums differ by what a large bias rounds off."""
    g = torch.Generator().manual_seed(E)
    for _ in range(4):
        logits = 2 * torch.randn(1, E, generator=g)
        bias = (at - torch.sigmoid(logits.double()))[0].float()
        logits = logits + 1e-6 * torch.randn(60, E, generator=g)
        if groups < E:
            logits[:, ::E // groups] = float("-inf")   # (a group with fewer)
        check(q, logits.cuda(), 4, score="sigmoid", bias=bias.cuda(), groups=groups, groups_kept=4, group_top=1)


@pytest.mark.parametrize("n", [-3, 0, 1, 77, 199, 200, 1000])
def test_live_tokens(q, n):
    logits = torch.randn(200, 64, generator=torch.Generator().manual_seed(1)).cuda()
    if 0 <= n < 200:
        logits[n:] = float("nan")
    check(q, logits, 4, live=torch.tensor([n], dtype=torch.int32, device="cuda"), score="sigmoid")


def test_pitches_slices_and_outputs(q):
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(50, 300, generator=g).cuda()
    for part in (wide[:, :100], wide[:, 4:104], wide[3:, 7:107], wide[::2, 8:108]):
        ids, w = check(q, part, 3, score="sigmoid")
        ref = q.moe_route_scored(part.contiguous(), 3, score="sigmoid")
        assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])
    out_i = torch.full((60, 3), 9, dtype=torch.int32, device="cuda")
    out_w = torch.full((60, 3), 9.0, device="cuda")
    got = q.moe_route_scored(wide[:, :100], 3, score="sigmoid", ids=out_i[5:55], w=out_w[5:55])   # (60 bytes in: copied)
    ref = q.moe_route_scored(wide[:, :100].contiguous(), 3, score="sigmoid")
    assert got[0].data_ptr() == out_i[5:].data_ptr() and torch.equal(out_i[5:55], ref[0]) and torch.equal(out_w[5:55], ref[1])
    rest = list(range(5)) + list(range(55, 60))
    assert out_i[rest].eq(9).all() and out_w[rest].eq(9).all()
    empty = q.moe_route_scored(wide[:0, :100], 3)
    assert empty[0].shape == (0, 3)


def test_a_graph_and_another_stream(q):
    g = torch.Generator().manual_seed(3)
    a, b = (torch.randn(37, 256, generator=g).cuda() for _ in range(2))
    bias = (0.1 * torch.randn(256, generator=g)).cuda()
    call = lambda x, **kw: q.moe_route_scored(x, 8, score="sigmoid", bias=bias, groups=8, groups_kept=4, **kw)  # noqa: E731
    want = [call(a), call(b)]
    x, live = a.clone(), torch.tensor([37], dtype=torch.int32, device="cuda")
    ids, w = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(x, ids=ids, w=w, live=live)
    s.synchronize()
    assert torch.equal(ids, want[0][0]) and torch.equal(w, want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, ids=ids, w=w, live=live)
    x.copy_(b)
    live.fill_(20)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids[:20], want[1][0][:20]) and torch.equal(w[:20], want[1][1][:20])
    assert ids[20:].eq(-1).all() and w[20:].eq(0).all()


def test_refusals(q):
    x = torch.randn(4, 16).cuda()
    with pytest.raises(ValueError):
        q.moe_route_scored(x, 2, score="tanh")
    with pytest.raises(q.QmmError):
        q.moe_route_scored(x, 17)
    with pytest.raises(q.QmmError):
        q.moe_route_scored(x, 2, groups=3)
    with pytest.raises(TypeError):
        q.moe_route_scored(x.half(), 2)
    with pytest.raises(TypeError):
        q.moe_route_scored(x, 2, bias=torch.zeros(16, device="cuda", dtype=BF16))
    with pytest.raises(ValueError):
        q.moe_route_scored(x, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        q.moe_route_scored(x, 2, live=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        q.moe_route_scored(x.t(), 2)
