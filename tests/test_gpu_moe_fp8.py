"""moe_expert_stage_fp8 against the formulas in 64 bits, step by step from its workspace: the grouping
has to be equal; H within the tolerance of test_gpu_fp8a8's SwiGLU; Y from the H that was stored.

Tolerance of Y: that of each expert's down product (test_gpu_fp8a8) times its weight, and the sum of
k + 1 terms in fp32, each addition within 2^-24 of the sum of magnitudes; bf16 output half a bf16 step,
and each expert's row then perhaps held as fp16 in units that bring the largest of 64 columns to
2^14 .. 2^15.  fp16 has 11 significant bits: the step in [2^e, 2^(e+1)) is 2^(e-10), half of it at most
2^-11 of the value; below 2^-14 the step is 2^-24, half of it 2^-25 of a unit, a unit at most 2^-14 of
the largest: 2^-39 of that.
"""
import numpy as np
import pytest
import torch
from test_gpu_fp8a8 import check_swiglu, formula, half_bf16_step

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def experts(seed, D, F, E):
    """E4M3 codes over their whole range and scales that differ by block."""
    g = torch.Generator().manual_seed(seed)
    kb, fb = -(-D // 128), F // 128
    Wgu = (torch.randn(E, 2 * F, D, generator=g) * 60).clamp(-448, 448).to(F8)
    Wd = (torch.randn(E, D, F, generator=g) * 60).clamp(-448, 448).to(F8)
    Sgu = (1 + torch.rand(E, 2 * fb, kb, generator=g)) * 2.0 ** -9 / D ** 0.5
    Sd = (1 + torch.rand(E, kb, fb, generator=g)) * 2.0 ** -6 / F ** 0.5
    return [t.cuda() for t in (Wgu, Sgu, Wd, Sd)]


def tokens(seed, T, D):
    g = torch.Generator().manual_seed(seed)
    Xq = (torch.randn(T, D, generator=g) * 100).clamp(-448, 448).to(F8).cuda()
    return Xq, (torch.exp(torch.randn(T, -(-D // 128), generator=g)) * 2.0 ** -7).cuda()


def choice(seed, T, E, k, how):
    """(ids, w) [T, k]."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(T, k, generator=g)
    if how == "twice":      # the same expert more than once in a token
        ids = torch.randint(0, max(1, min(E, 3)), (T, k), generator=g)
    elif how == "one":      # every pair to one expert
        ids = torch.full((T, k), E - 1)
    elif how == "none":
        ids = torch.full((T, k), -1)
    else:
        ids = torch.rand(T, E, generator=g).argsort(1)[:, :k] if k <= E else torch.randint(0, E, (T, k), generator=g)
        if how == "skewed":
            ids = torch.where(torch.rand(T, k, generator=g) < 0.7, torch.zeros_like(ids), ids)
        if how == "holes":  # pairs without an expert, and ids out of range, with NaN weights
            off = torch.rand(T, k, generator=g) < 0.4
            ids = torch.where(off, torch.tensor([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 5, (T, k), generator=g)], ids)
            w[off] = float("nan")
            ids[T // 2] = -1
    return ids.to(torch.int32).cuda(), w.cuda()


def check(q, seed, T, D, F, E, k, how="even", dt=F32, res=None, weights=None, plan=None):
    Wgu, Sgu, Wd, Sd = weights or experts(seed, D, F, E)
    Xq, Xs = tokens(seed + 1, T, D)
    ids, w = choice(seed + 2, T, E, k, how)
    R = None if res is None else (2 * torch.randn(T, D, generator=torch.Generator().manual_seed(seed))).to(res).cuda()
    P, kb = T * k, -(-D // 128)
    ws = torch.empty(q.moe_expert_stage_fp8_workspace_size(T, D, F, E, k) + 256, dtype=torch.uint8, device="cuda")
    ws.fill_(0x7F)   # (NaN codes and large scales in what nothing writes)
    if plan is None:
        Y = q.moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd, R=R, out_dtype=dt, ws=ws[:-256])
    else:
        Y = q.qmm_dbg_moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd, plan, R=R, out_dtype=dt, ws=ws[:-256])
    q.qmm_check_status()
    assert ws[-256:].eq(0x7F).all()
    lay = q.moe_expert_stage_fp8_workspace_layout(T, D, F, E, k)
    view = lambda n, t, s: q.workspace_view(ws, lay, n, t, s)  # noqa: E731
    # grouping: stable by expert
    flat = ids.cpu().numpy().reshape(-1)
    on = (flat >= 0) & (flat < E)
    order = [p for p in np.argsort(np.where(on, flat, E), kind="stable") if on[p]]
    counts = np.bincount(flat[on], minlength=E)
    row = np.full(P, -1)
    row[order] = np.arange(len(order))
    off = view("offsets", torch.int32, (E + 1,)).cpu().numpy()
    assert np.array_equal(view("counts", torch.int32, (E,)).cpu().numpy(), counts)
    assert np.array_equal(off, np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(view("row", torch.int32, (P,)).cpu().numpy(), row)
    src = view("src", torch.int32, (P,)).cpu().numpy()[:len(order)]
    assert np.array_equal(src, np.array(order, dtype=int) // k)
    # H, and Y from the stored H
    Hq, Hs = view("Hq", F8, (P, F)), view("Hs", F32, (P, F // 128))
    y, tol = np.zeros((T, D)), np.zeros((T, D))
    if R is not None:
        y += R.double().cpu().numpy()
    size = np.abs(y)
    wf = w.double().cpu().numpy().reshape(-1)
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        t = torch.from_numpy(src[a:b].astype(np.int64)).cuda()
        check_swiglu(Hq[a:b], Hs[a:b], *formula(Xq[t], Xs[t], Wgu[e], Sgu[e]))
        v, d = formula(Hq[a:b], Hs[a:b], Wd[e], Sd[e])
        p = np.array(order[a:b])
        np.add.at(y, p // k, wf[p][:, None] * v)
        np.add.at(size, p // k, np.abs(wf[p][:, None] * v))
        if dt == BF16:
            d = d + 2.0 ** -11 * (np.abs(v) + d) + 2.0 ** -39 * np.abs(v).max(1, keepdims=True)
        np.add.at(tol, p // k, np.abs(wf[p])[:, None] * d)
    tol += (k + 1) * 2.0 ** -24 * (size + tol)
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(y) + tol)
    assert Y.dtype == dt and Y.shape == (T, D)
    assert np.all(np.abs(Y.double().cpu().numpy() - y) <= tol)
    return Y


HOWS = ["even", "skewed", "holes", "twice", "one"]
SHAPES = [(1, 256, 128, 8, 2), (1, 2048, 768, 16, 8), (2, 16, 128, 3, 1), (3, 144, 256, 5, 5), (7, 400, 384, 1, 1), (16, 128, 128, 2, 2),
          (17, 272, 128, 4, 3), (33, 1000 // 16 * 16, 256, 6, 4), (64, 512, 128, 12, 6), (100, 2000, 256, 4, 4), (129, 640, 512, 3, 2),
          (200, 256, 1024, 5, 2), (300, 384, 256, 2, 1), (513, 128, 128, 7, 3), (700, 272, 256, 2, 2), (1030, 256, 128, 4, 2), (260, 144, 128, 2, 1), (513, 1024, 768, 3, 1),
          (1500, 272, 384, 2, 1)]
MANY = (1, 128, 1, 1)


@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_stage(q, i, how):
    check(q, 10 * i, *SHAPES[i], how=how, dt=[F32, BF16][i % 2], res=[None, F32, BF16][(i + len(how)) % 3])


@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_tiles_of_128_rows(q, i, how):
    """Every shape by the kernel for many rows an expert."""
    check(q, 10 * i + 1, *SHAPES[i], how=how, dt=[BF16, F32][i % 2], res=[None, F32, BF16][(i + len(how)) % 3], plan=MANY)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,D,F,E,k", [(64, 2048, 768, 64, 4), (700, 400, 384, 96, 3), (300, 1008, 1024, 48, 4), (2500, 272, 256, 130, 2), (500, 2320, 128, 200, 4),
                                       (40, 128, 1280, 100, 4), (3000, 640, 640, 3, 2)])
def test_more_tiles_than_ctas(q, T, D, F, E, k, dt):
    """Several tiles a persistent CTA, of one to twenty K blocks, odd and even."""
    check(q, T, T, D, F, E, k, dt=dt, res=BF16, plan=MANY)
    check(q, T, T, D, F, E, k, how="holes", dt=dt, plan=MANY)


@pytest.mark.parametrize("tn", [16, 32, 64, 128])
@pytest.mark.parametrize("cs", [(1, 1), (2, 2), (3, 1), (1, 2), (8, 2)])
def test_tiles_of_few_rows(q, tn, cs):
    for n, (shape, how) in enumerate([((3, 1040, 256, 5, 4), "even"), ((200, 1040, 256, 3, 2), "skewed"), ((90, 1024, 256, 40, 6), "holes"), ((40, 1040, 256, 2, 3), "twice")]):
        check(q, tn + n, *shape, how=how, dt=[F32, BF16][n % 2], res=[BF16, None][n % 2], plan=(0, tn, *cs))


def test_the_rule_reaches_both_kernels(q):
    plans = {q.qmm_dbg_moe_fp8_plan(T, 2048, 768, 128, 8)[0] for T in (1, 8, 301, 5268)}
    assert plans == {0, 1}
    check(q, 77, 301, 512, 768, 128, 8, dt=BF16)


@pytest.mark.parametrize("T,k,E", [(2048, 1, 512), (300, 16, 512), (1025, 2, 2), (2049, 3, 40), (5000, 2, 8)])
def test_grouping_over_several_chunks(q, T, k, E):
    check(q, T, T, 128, 128, E, k)
    check(q, T, T, 128, 128, E, k, how="holes")


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,D,k", [(1216, 1040, 2), (1217, 1040, 2), (1216, 2064, 6), (1217, 2064, 6), (1300, 1024, 16)])
def test_rows_summed_in_one_block_or_several(q, T, D, k, dt):
    """Both ways to give a token's columns to blocks, on both sides of the rule and with a part of a block left."""
    check(q, T, T, D, 128, 4, k, how="holes", dt=dt, res=BF16, plan=(0, 64, 1, 1))
    check(q, T, T, D, 128, 4, k, how="holes", dt=dt, plan=MANY)


def test_more_experts_than_pairs_and_more_choices_than_experts(q):
    check(q, 1, 3, 256, 128, 512, 2)
    check(q, 2, 40, 256, 128, 2, 16)


@pytest.mark.parametrize("T", [1, 50])
def test_tokens_without_experts(q, T):
    R = torch.randn(T, 256).cuda()
    Wgu, Sgu, Wd, Sd = experts(0, 256, 128, 4)
    Xq, Xs = tokens(0, T, 256)
    ids, w = choice(0, T, 4, 3, "none")
    assert torch.equal(q.moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd, R=R, out_dtype=F32), R)
    assert q.moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd).eq(0).all()
    for plan in (MANY, (0, 16, 1, 1), (0, 128, 2, 1)):
        assert torch.equal(q.qmm_dbg_moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd, plan, R=R, out_dtype=F32), R)
    assert q.moe_expert_stage_fp8(Xq[:0], Xs[:0], ids[:0], w[:0], Wgu, Sgu, Wd, Sd).shape == (0, 256)
    q.qmm_check_status()


def test_nan_rows_stay_in_their_token(q):
    T, D, F, E, k = 40, 256, 128, 4, 2
    Wgu, Sgu, Wd, Sd = experts(3, D, F, E)
    Xq, Xs = tokens(3, T, D)
    ids, w = choice(3, T, E, k, "even")
    want = q.moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd)
    bad = Xq.clone()
    bad.view(torch.uint8)[[0, 7, 39], 5] = 0x7F
    got = q.moe_expert_stage_fp8(bad, Xs, ids, w, Wgu, Sgu, Wd, Sd)
    rest = [t for t in range(T) if t not in (0, 7, 39)]
    assert got[[0, 7, 39]].isnan().all() and torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("plan", [MANY, (0, 16, 1, 1), (0, 128, 2, 1)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_what_is_not_finite_stays_in_its_token(q, plan, dt):
    """NaN codes, scales that are infinite, NaN or near the largest number: the other tokens' bits are as without them."""
    T, D, F, E, k = 301, 272, 256, 3, 2
    Wgu, Sgu, Wd, Sd = experts(4, D, F, E)
    Xq, Xs = tokens(4, T, D)
    ids, w = choice(4, T, E, k, "even")
    want = q.qmm_dbg_moe_expert_stage_fp8(Xq, Xs, ids, w, Wgu, Sgu, Wd, Sd, plan, out_dtype=dt)
    assert want.isfinite().all()
    code, scale, weight = Xq.clone(), Xs.clone(), w.clone()
    code.view(torch.uint8)[[0, 300], 5] = 0x7F
    scale[7, 0], scale[31, 1], scale[32, 2], weight[140, 1] = float("nan"), float("inf"), 3e38, float("nan")
    got = q.qmm_dbg_moe_expert_stage_fp8(code, scale, ids, weight, Wgu, Sgu, Wd, Sd, plan, out_dtype=dt)
    rest = [t for t in range(T) if t not in (0, 7, 31, 32, 140, 300)]
    assert got[[0, 7, 140, 300]].isnan().all() and torch.equal(got[rest], want[rest])
    q.qmm_check_status()


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_residual_in_place_slices_and_repeats(q, T, dt):
    D, F, E, k = 272, 128, 4, 2
    Wgu, Sgu, Wd, Sd = experts(5, D, F, E)
    Xq, Xs = tokens(5, T + 2, D)
    ids, w = choice(5, T + 2, E, k, "even")
    R = torch.randn(T + 2, D + 20).to(dt).cuda()
    part = slice(1, T + 1)
    args = [t[part].clone() for t in (Xq, Xs, ids, w)]
    want = q.moe_expert_stage_fp8(*args, Wgu, Sgu, Wd, Sd, R=R[part, :D].clone(), out_dtype=dt)
    for _ in range(3):   # the same bits every call
        assert torch.equal(q.moe_expert_stage_fp8(*args, Wgu, Sgu, Wd, Sd, R=R[part, :D].clone(), out_dtype=dt), want)
    for r in (R[part, :D], R[part, 3:3 + D]):
        ref = want if r.data_ptr() == R[part].data_ptr() else q.moe_expert_stage_fp8(*args, Wgu, Sgu, Wd, Sd, R=r.clone(), out_dtype=dt)
        got = q.moe_expert_stage_fp8(Xq[part], Xs[part], ids[part], w[part], Wgu, Sgu, Wd, Sd, R=r, out_dtype=dt)
        assert torch.equal(got, ref)
    out = torch.full((T + 2, D), 9.0, dtype=dt, device="cuda")
    out[part] = R[part, :D]
    q.moe_expert_stage_fp8(*args, Wgu, Sgu, Wd, Sd, R=out[part], out_dtype=dt, Y=out[part])
    assert torch.equal(out[part], want) and out[0].eq(9).all() and out[-1].eq(9).all()


def test_graphs_and_streams(q):
    """Two captured graphs, each with a workspace of its own, replayed side by side; inputs change between replays."""
    T, D, F, E, k = 24, 512, 256, 8, 3
    Wgu, Sgu, Wd, Sd = experts(6, D, F, E)
    sets = [(*tokens(s, T, D), *choice(s, T, E, k, "even")) for s in range(4)]
    want = [q.moe_expert_stage_fp8(*s, Wgu, Sgu, Wd, Sd) for s in sets]
    graphs = []
    for _ in range(2):
        ins = [t.clone() for t in sets[0]]
        ws = torch.empty(q.moe_expert_stage_fp8_workspace_size(T, D, F, E, k), dtype=torch.uint8, device="cuda")
        Y = torch.empty_like(want[0])
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            q.moe_expert_stage_fp8(*ins, Wgu, Sgu, Wd, Sd, Y=Y, ws=ws)
        graphs.append((ins, Y, stream, graph, ws))   # (a graph uses its workspace as long as it is replayed)
    for i, j in ((0, 1), (2, 3), (3, 0)):
        for (ins, Y, *_), s in zip(graphs, (i, j)):
            for a, b in zip(ins, sets[s]):
                a.copy_(b)
        torch.cuda.synchronize()
        for _, _, stream, graph, _ in graphs:
            with torch.cuda.stream(stream):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for (ins, Y, *_), s in zip(graphs, (i, j)):
            assert torch.equal(Y, want[s])
    q.qmm_check_status()


def test_a_layer(q):
    """Norm, router, experts and a shared expert with its residual, as a model runs them, against the same in 64 bits on the
    codes that the calls hand on."""
    T, D, F, E, k = 70, 512, 256, 16, 4
    Wgu, Sgu, Wd, Sd = experts(8, D, F, E)
    shared = [t[0] for t in experts(9, D, F, 1)]
    g = torch.Generator().manual_seed(8)
    x, r = torch.randn(T, D, generator=g).to(BF16).cuda(), torch.randn(T, D, generator=g).to(BF16).cuda()
    G = torch.ones(D, device="cuda")
    Wr = (torch.randn(E, D, generator=g) / D ** 0.5).cuda()
    bias = (0.05 * torch.randn(E, generator=g)).cuda()
    n = q.qmm_add_rmsnorm_fp8(x, G, R=r, Rout=r, bf16_out=True)
    ids, w = q.moe_route_scored(n["Y"].float() @ Wr.t(), k, score="sigmoid", bias=bias, groups=4, groups_kept=2, scale=2.5)
    y = q.moe_expert_stage_fp8(n["Q"], n["S"], ids, w, Wgu, Sgu, Wd, Sd, R=r, out_dtype=F32)
    Hq, Hs = q.qmm_fp8a8_swiglu_blk128(n["Q"], n["S"], shared[0], shared[1])
    out = q.qmm_fp8a8_epilogue_blk128(Hq, Hs, shared[2], shared[3], R=y, out_dtype=F32, Y=y)
    q.qmm_check_status()
    assert out.data_ptr() == y.data_ptr()
    X = n["Q"].double() * n["S"].double().repeat_interleave(128, 1)
    deq = lambda c, s: c.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
    ref = r.double()
    for c, s, c2, s2, wt in [(*shared, torch.ones(T, device="cuda"))] + \
            [(Wgu[e], Sgu[e], Wd[e], Sd[e], torch.where(ids == e, w, 0.0).sum(1)) for e in range(E)]:
        gt, u = (X @ deq(c, s).t()).chunk(2, 1)
        ref = ref + wt.double()[:, None] * ((torch.nn.functional.silu(gt) * u) @ deq(c2, s2).t())
    # H's rounding: each code within 2^-4 of its value, F of them a sum; in the mean 2^-5 and random
    err = (out.double() - ref).norm() / (ref - r.double()).norm()
    assert err <= 2.0 ** -4, err


def test_refusals(q):
    Wgu, Sgu, Wd, Sd = experts(0, 256, 128, 4)
    Xq, Xs = tokens(0, 5, 256)
    ids, w = choice(0, 5, 4, 2, "even")
    good = dict(Xq=Xq, Xs=Xs, ids=ids, w=w, Wgu=Wgu, Sgu=Sgu, Wd=Wd, Sd=Sd)
    for name, bad, error in [("ids", ids.long(), TypeError), ("w", w.to(BF16), TypeError), ("w", w[:4], ValueError), ("Xs", Xs[:, :1], ValueError),
                             ("Wd", Wd[:3], ValueError), ("Sgu", Sgu[:, :1].contiguous(), ValueError), ("Sd", Sd.transpose(1, 2), ValueError),
                             ("R", torch.zeros(5, 255, device="cuda"), ValueError), ("ws", torch.empty(64, dtype=torch.uint8, device="cuda"), q.QmmError),
                             ("out_dtype", torch.float16, TypeError)]:
        with pytest.raises(error):
            q.moe_expert_stage_fp8(**{**good, name: bad})
    for name, bad in [("ids", ids[:, 0].contiguous()), ("ids", ids[0, 0]), ("Wgu", Wgu[0]), ("Wgu", Wgu[0, 0]), ("Wgu", Wgu[:, :255].contiguous()),
                      ("Wd", Wd[0]), ("Xs", Xs[:, 0].contiguous())]:
        with pytest.raises(ValueError):
            q.moe_expert_stage_fp8(**{**good, name: bad})
    for plan in ((1, 64, 1, 1), (0, 48, 1, 1), (0, 16, 3, 1), (0, 16, 1, 2), (0, 16, 0, 1), (0, 16, 1, 9)):   # (2 K blocks, 1)
        with pytest.raises(q.QmmError):
            q.qmm_dbg_moe_expert_stage_fp8(**good, plan=plan)
    x = torch.zeros(5, 256, device="cuda")
    with pytest.raises(q.QmmError):   # in place, of another type
        q.moe_expert_stage_fp8(**good, R=x, Y=x.view(-1)[:640].view(BF16).view(5, 256))
