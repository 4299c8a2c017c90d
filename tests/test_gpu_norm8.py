"""qmm_add_rmsnorm_fp8 / qmm_add_rmsnorm_q8_1 against the formulas in 64 bits.

Tolerances, from the arithmetic: the sum of squares is at most 64 terms per
thread in sequence plus 13 adds of a tree, each within 2^-24, halved by the square
root; the mean, square root, division, two products and the scale's division add
fewer than 10 roundings: every y and scale is within REL = 64 * 2^-24 of the
formula.  A code is the nearest to within half a step of its format at the
quotient, plus 2 REL of the quotient (y and the scale); a bf16 row within half a bf16
step plus REL.  The stored sum is one
fp32 addition and one rounding: equal bits.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
REL = 64 * 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def rows(seed, T, D, dtype, scale=1.0, pitch=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, pitch or D, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) * scale
    x[:, :: max(1, D // 5)] *= 15.0
    return x.to(dtype).cuda()[:, :D]


def formula(X, G, R, eps):
    v = X.float()
    stored = None
    if R is not None:
        stored = (v + R.float()).to(R.dtype)
        v = stored
    v = v.double().cpu()
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * G.double().cpu()
    return stored, y.numpy()


def groups(y, n):
    T, D = y.shape
    full = np.zeros((T, -(-D // n) * n))
    full[:, :D] = y
    return full.reshape(T, -1, n)


def e4m3_step(t):
    return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(t), 1e-30))), -6) - 3)


def half_bf16_step(t):
    """bf16 has 8 significant bits: half a step in [2^e, 2^(e+1)) is 2^(e - 8)."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 1e-38))) - 8)


def check_fp8(out, stored, y):
    T, D = y.shape
    if stored is not None:
        assert torch.equal(out["R"], stored)
    s = out["S"].double().cpu().numpy()
    full = groups(y, 128)
    ref = np.abs(full).max(-1) / 448
    assert s.shape == ref.shape
    assert np.all(np.abs(s - ref) <= REL * ref)
    code = groups(out["Q"].float().cpu().numpy().astype(np.float64), 128)
    t = full / np.where(ref == 0, 1, ref)[..., None]
    assert np.all(np.abs(code - t) <= 0.5 * e4m3_step(t) + 2 * REL * np.abs(t))
    if out["Y"] is not None:
        d = np.abs(out["Y"].double().cpu().numpy() - y)
        assert np.all(d <= half_bf16_step(np.abs(y) * (1 + REL)) + REL * np.abs(y))


def check_q81(out, stored, y):
    if stored is not None:
        assert torch.equal(out["R"], stored)
    full = groups(y, 32)
    ref = np.abs(full).max(-1) / 127
    d = out["Yd"].view(torch.float16).double().cpu().numpy()
    s = out["Ys"].view(torch.float16).double().cpu().numpy()
    code = groups(out["Yq"].cpu().numpy().astype(np.float64), 32)
    t = full / np.where(ref == 0, 1, ref)[..., None]
    assert np.all(np.abs(code - t) <= 0.5 + 2 * REL * np.abs(t))
    assert np.all(np.abs(d - ref) <= (2.0 ** -11 + REL) * ref * 1.01 + 2.0 ** -25)
    want = ref * code.sum(-1)
    assert np.all(np.abs(s - want) <= (2.0 ** -11 + 2 * REL) * np.abs(want) * 1.01 + 2.0 ** -25)


TYPES = [(BF16, None, BF16), (BF16, BF16, BF16), (F32, BF16, BF16), (BF16, F32, F32), (F32, F32, F32), (F32, None, BF16)]


@pytest.mark.parametrize("xt,rt,gt", TYPES)
@pytest.mark.parametrize("T,D", [(1, 16), (3, 128), (5, 144), (2, 2000), (37, 2048), (4, 2064), (19, 5120), (2, 8192), (3, 16384)])
def test_fp8(q, T, D, xt, rt, gt):
    X = rows(T + D, T, D, xt)
    R = rows(T + D + 1, T, D, rt, 3.0) if rt else None
    G = (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(D))).to(gt).cuda()
    out = q.qmm_add_rmsnorm_fp8(X.contiguous(), G, R=R, bf16_out=D % 3 == 2)
    check_fp8(out, *formula(X, G, R, 1e-6))


@pytest.mark.parametrize("xt,rt,gt", TYPES)
@pytest.mark.parametrize("T,D", [(1, 32), (7, 160), (300, 2048), (5, 2592), (11, 5120), (2, 16384)])
def test_q8_1(q, T, D, xt, rt, gt):
    X = rows(T + D, T, D, xt)
    R = rows(T + D + 1, T, D, rt, 3.0) if rt else None
    G = (1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(D))).to(gt).cuda()
    out = q.qmm_add_rmsnorm_q8_1(X, G, R=R, eps=1e-5, bf16_out=True)
    check_q81(out, *formula(X, G, R, 1e-5))


def test_row_slices_and_the_sum_in_place(q):
    T, D = 23, 640
    X = rows(1, T, D, BF16, pitch=1000)
    R = rows(2, T, D, F32, pitch=648)
    G = torch.ones(D, device="cuda")
    stored, y = formula(X, G, R, 1e-6)
    around = R._base.clone() if R._base is not None else None
    out = q.qmm_add_rmsnorm_fp8(X, G, R=R, Rout=R)
    assert out["R"].data_ptr() == R.data_ptr()
    check_fp8(out, stored, y)
    if around is not None:   # nothing beside the rows is written
        assert torch.equal(R._base[:, D:], around[:, D:])
    # the sum into x's own buffer
    X2, R2 = rows(3, T, D, BF16), rows(4, T, D, BF16)
    stored, y = formula(X2, G, R2, 1e-6)
    check_fp8(q.qmm_add_rmsnorm_fp8(X2, G, R=R2, Rout=X2), stored, y)


def test_rows_of_zeros_and_tiny_rows(q):
    X = torch.zeros(4, 256, device="cuda")
    X[1] = 1e-30                       # below eps: y and the scales are tiny
    X[2, :128] = 0                     # a group of zeros beside one that is not
    X[2, 128:] = torch.linspace(-1, 1, 128)
    X[3] = 1e30                        # the square is infinite: 1 / inf = 0, y = 0
    G = torch.ones(256, device="cuda")
    out = q.qmm_add_rmsnorm_fp8(X, G)
    code, s = out["Q"].float().cpu(), out["S"].cpu()
    assert torch.equal(code[0], torch.zeros(256)) and torch.equal(s[0], torch.zeros(2))
    assert torch.equal(code[1], torch.full((256,), 448.0))
    assert abs(float(s[1, 0]) / (1e-27 / 448) - 1) < 1e-5
    assert s[2, 0] == 0 and torch.equal(code[2, :128], torch.zeros(128)) and float(code[2, 255]) == 448
    assert torch.equal(code[3], torch.zeros(256)) and torch.equal(s[3], torch.zeros(2))
    # denormal scales: every quotient is still in range
    out = q.qmm_add_rmsnorm_fp8(X[1:2], torch.full((256,), 1e-14, device="cuda"))
    assert 0 < float(out["S"][0, 0]) < 2.0 ** -126
    assert torch.all((out["Q"].float() - 448).abs() <= 32)
    out = q.qmm_add_rmsnorm_q8_1(X, G)
    assert not out["Yq"][0].any() and not out["Yd"][0].any() and not out["Ys"][0].any()


def test_nan_and_infinity_stay_in_their_row(q):
    X = rows(5, 6, 384, BF16).contiguous()
    clean = q.qmm_add_rmsnorm_fp8(X, torch.ones(384, device="cuda"))
    Z = X.clone()
    Z[1, 200] = float("nan")
    Z[4, 7] = float("inf")
    out = q.qmm_add_rmsnorm_fp8(Z, torch.ones(384, device="cuda"))
    code = out["Q"].float()
    assert torch.isnan(code[1]).all() and torch.isnan(out["S"][1]).all()
    # inf / inf at the infinity, and its whole group; v / inf = 0 elsewhere
    assert torch.isnan(code[4, :128]).all() and not code[4, 128:].any()
    for r in (0, 2, 3, 5):
        assert torch.equal(out["Q"][r].view(torch.uint8), clean["Q"][r].view(torch.uint8))
        assert torch.equal(out["S"][r], clean["S"][r])


def test_no_rows(q):
    G = torch.ones(128, device="cuda")
    out = q.qmm_add_rmsnorm_fp8(torch.empty(0, 128, device="cuda"), G)
    assert out["Q"].shape == (0, 128) and out["S"].shape == (0, 1)
    out = q.qmm_add_rmsnorm_q8_1(torch.empty(0, 128, device="cuda"), G, R=torch.empty(0, 128, device="cuda"))
    assert out["Yd"].shape == (0, 4)


def test_offsets_past_32_bits(q):
    """Rows whose element offsets pass 2^32: the last rows equal the same rows alone."""
    T, D = 270000, 16384               # 4.4e9 elements
    X = torch.empty((T, D), dtype=BF16, device="cuda")
    X[:4] = rows(6, 4, D, BF16)
    X[-4:] = rows(7, 4, D, BF16)
    X[4:-4] = 1
    G = torch.ones(D, device="cuda")
    Q = torch.empty((T, D), dtype=torch.uint8, device="cuda")
    out = q.qmm_add_rmsnorm_fp8(X, G, Q=Q)
    for part in (slice(0, 4), slice(T - 4, T)):
        alone = q.qmm_add_rmsnorm_fp8(X[part].contiguous(), G)
        assert torch.equal(out["Q"][part], alone["Q"].view(torch.uint8))
        assert torch.equal(out["S"][part], alone["S"])


def test_own_stream_and_graph(q):
    X, R, G = rows(8, 9, 2048, BF16).contiguous(), rows(9, 9, 2048, BF16).contiguous(), torch.ones(2048, device="cuda")
    ref = q.qmm_add_rmsnorm_fp8(X, G, R=R)
    bufs = {k: torch.zeros_like(ref[k]) for k in ("Q", "S", "R")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = q.qmm_add_rmsnorm_fp8(X, G, R=R)
        graph = torch.cuda.CUDAGraph()
    s.synchronize()
    assert torch.equal(out["Q"].view(torch.uint8), ref["Q"].view(torch.uint8))
    with torch.cuda.graph(graph):
        q.qmm_add_rmsnorm_fp8(X, G, R=R, Rout=bufs["R"], Q=bufs["Q"], S=bufs["S"])
    X.copy_(rows(10, 9, 2048, BF16))
    graph.replay()
    check_fp8(dict(bufs, Y=None), *formula(X, G, R, 1e-6))


def test_refusals(q):
    X, G = torch.ones(4, 256, device="cuda"), torch.ones(256, device="cuda")
    with pytest.raises(q.QmmError, match="D % 16"):
        q.qmm_add_rmsnorm_fp8(X[:, :200].contiguous(), G[:200].contiguous())
    with pytest.raises(q.QmmError, match="D % 32"):
        q.qmm_add_rmsnorm_q8_1(X[:, :240].contiguous(), G[:240].contiguous())
    with pytest.raises(q.QmmError, match="16384"):
        q.qmm_add_rmsnorm_fp8(torch.ones(1, 16400, device="cuda"), torch.ones(16400, device="cuda"))
    with pytest.raises(q.QmmError, match="eps"):
        q.qmm_add_rmsnorm_fp8(X, G, eps=-1.0)
    with pytest.raises(q.QmmError, match="eps"):
        q.qmm_add_rmsnorm_fp8(X, G, eps=float("nan"))
    with pytest.raises(q.QmmError, match="aligned"):
        q.qmm_add_rmsnorm_fp8(torch.ones(4, 264, device="cuda")[:, 1:257], G)
    with pytest.raises(q.QmmError, match="pitches"):
        q.qmm_add_rmsnorm_fp8(torch.ones(4, 260, device="cuda")[:, :256], G)
    with pytest.raises(TypeError):
        q.qmm_add_rmsnorm_fp8(X.half(), G)
    with pytest.raises(TypeError):
        q.qmm_add_rmsnorm_fp8(X.cpu(), G)
    with pytest.raises(TypeError):
        q.qmm_add_rmsnorm_fp8(X, G, R=X, Rout=X.to(BF16))
    with pytest.raises(ValueError):
        q.qmm_add_rmsnorm_fp8(X, G, Rout=X)
    with pytest.raises(ValueError):
        q.qmm_add_rmsnorm_fp8(X, G, R=X[:3])
    with pytest.raises(ValueError):
        q.qmm_add_rmsnorm_fp8(X.t(), G)
    with pytest.raises(ValueError):
        q.qmm_add_rmsnorm_fp8(X, G, S=torch.empty(4, 3, device="cuda"))
