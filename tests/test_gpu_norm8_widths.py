"""Every kernel form of the 8-bit norms, by width: a warp a row with one, two or four vectors of
8 values a lane (up to 256, 512 and 1024 values), a CTA a row with one or two (fp32 or mixed
rows), two or four (all bf16).

Tolerance, from the present order of additions: a thread adds at most 16 pairs of squares one after
the other, then the two halves, then 5 or 10 steps of a tree: at most 27 additions of positive terms, each
within 2^-24, halved by the square root; the mean, eps, the square root, the reciprocal and two
products add at most 6 roundings: y is within 20 * 2^-24 of the formula's, a scale (a product with the
rounded 1/448 or 1/127: two roundings) within REL = 24 * 2^-24.  A quotient adds the scale's error, its reciprocal
(1 ulp) and a product: below 2 REL.
"""
import pytest
import test_gpu_norm8 as t
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


@pytest.fixture(autouse=True)
def tolerance(monkeypatch):
    monkeypatch.setattr(t, "REL", 24 * 2.0 ** -24)


def inputs(T, D, xt, rt, gt):
    X = t.rows(T + D, T, D, xt)
    R = t.rows(T + D + 1, T, D, rt, 3.0) if rt else None
    return X, R, (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(D))).to(gt).cuda()


@pytest.mark.parametrize("xt,rt,gt", t.TYPES)
@pytest.mark.parametrize("D", [256, 272, 384, 496, 512, 528, 768, 1008, 1024, 1040, 8208])
def test_fp8(q, D, xt, rt, gt):
    for T in (1, 13):
        X, R, G = inputs(T, D, xt, rt, gt)
        t.check_fp8(q.qmm_add_rmsnorm_fp8(X, G, R=R, bf16_out=True), *t.formula(X, G, R, 1e-6))


@pytest.mark.parametrize("xt,rt,gt", t.TYPES)
@pytest.mark.parametrize("D", [256, 288, 512, 544, 992, 1024, 1056, 8224])
def test_q8_1(q, D, xt, rt, gt):
    for T in (1, 13):
        X, R, G = inputs(T, D, xt, rt, gt)
        t.check_q81(q.qmm_add_rmsnorm_q8_1(X, G, R=R, bf16_out=True), *t.formula(X, G, R, 1e-6))


@pytest.mark.parametrize("D", [256, 512, 1024, 2048, 16384])
def test_nothing_beside_the_rows(q, D):
    """Row slices in and out: what lies between and behind the rows stays."""
    T = 9
    for xt, rt in ((BF16, BF16), (F32, F32), (F32, BF16)):
        X, R, G = inputs(T, D, xt, rt, F32)
        wide = {k: torch.full((T + 1, D + 64), 7.0, dtype=v.dtype, device="cuda") for k, v in (("X", X), ("R", R), ("Rout", R))}
        wide["X"][:T, :D], wide["R"][:T, :D] = X, R
        Q = torch.full((T + 1, D), 7, dtype=torch.int8, device="cuda")
        S = torch.full((T + 1, D // 128), 7.0, device="cuda")
        out = q.qmm_add_rmsnorm_fp8(wide["X"][:T, :D], G, R=wide["R"][:T, :D], Rout=wide["Rout"][:T, :D], Q=Q[:T], S=S[:T])
        t.check_fp8(dict(out, Q=out["Q"].view(torch.float8_e4m3fn)), *t.formula(X, G, R, 1e-6))
        for w in wide.values():
            assert bool((w[:T, D:] == 7).all()) and bool((w[T] == 7).all())
        assert bool((Q[T] == 7).all()) and bool((S[T] == 7).all())
        assert torch.equal(wide["X"][:T, :D], X) and torch.equal(wide["R"][:T, :D], R)


def test_q8_1_nan_and_infinity_show_in_the_scales(q):
    """int8 has no NaN: a block that a NaN or an infinity reaches has a NaN d and s."""
    X = t.rows(5, 6, 384, BF16).contiguous()
    G = torch.ones(384, device="cuda")
    clean = q.qmm_add_rmsnorm_q8_1(X, G)
    Z = X.clone()
    Z[1, 200] = float("nan")
    Z[4, 7] = float("inf")
    out = q.qmm_add_rmsnorm_q8_1(Z, G, bf16_out=True)
    d, s = (out[k].view(torch.float16) for k in ("Yd", "Ys"))
    assert torch.isnan(d[1]).all() and torch.isnan(s[1]).all() and torch.isnan(out["Y"][1]).all()
    # inf / inf in its own block; v / inf = 0 in the others
    assert torch.isnan(d[4, 0]) and torch.isnan(s[4, 0]) and not d[4, 1:].any() and not out["Yq"][4, 32:].any()
    for r in (0, 2, 3, 5):
        assert all(torch.equal(out[k][r], clean[k][r]) for k in ("Yq", "Yd", "Ys"))
