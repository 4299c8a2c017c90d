"""qmm_fp8a8_blk128 / qmm_fp8a8_swiglu_blk128 against the formulas in 64 bits.

Tolerance of a product, from the arithmetic: products of E4M3 codes are exact in
fp32; a block's 128 products are added in fp32 (each addition within 2^-23 of the
block's sum of magnitudes, truncation included), scaled (2 roundings) and added over
the KB blocks: |y - formula| <= (128 + KB + 4) * 2^-23 * A, with A the same sum over
magnitudes.  bf16 output adds half a bf16 step.  SwiGLU: |silu'| <= 1.1, so h is
within 1.1 |u| dg + |silu| du, plus 32 * 2^-24 relative for the exponential, the
division and the product (a few ulp each, an exponent error growing with |g|).  A
scale is within the largest such error of its group; a code is the nearest to within
half a step at the quotient, plus those errors over the scale.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def operands(seed, M, K, N):
    """Codes over the whole range of E4M3 and scales that differ by block."""
    g = torch.Generator().manual_seed(seed)
    kb = -(-K // 128)
    Xq = (torch.randn(M, K, generator=g) * 100).clamp(-448, 448).to(F8)
    W = (torch.randn(N, K, generator=g) * 60).clamp(-448, 448).to(F8)
    Xs = torch.exp(torch.randn(M, kb, generator=g)) * 2.0 ** -7
    S = (1 + torch.rand(-(-N // 128), kb, generator=g)) * 2.0 ** -9 / K ** 0.5
    return [t.cuda() for t in (Xq, Xs, W, S)]


def formula(Xq, Xs, W, S):
    """(y, tolerance) in 64 bits."""
    K, N = Xq.shape[1], W.shape[0]
    kb = -(-K // 128)
    x = Xq.float().double() * Xs.double().repeat_interleave(128, 1)[:, :K]
    w = W.float().double() * S.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y, A = x @ w.t(), x.abs() @ w.abs().t()
    return y.cpu().numpy(), (128 + kb + 4) * 2.0 ** -23 * A.cpu().numpy()


def e4m3_step(t):
    return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(t), 1e-30))), -6) - 3)


def half_bf16_step(t):
    """bf16 has 8 significant bits: half a step in [2^e, 2^(e+1)) is 2^(e - 8)."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(t), 1e-38))) - 8)


def check_swiglu(Hq, Hs, y, tol):
    F = y.shape[1] // 2
    g, u, dg, du = y[:, :F], y[:, F:], tol[:, :F], tol[:, F:]
    silu = g / (1 + np.exp(-g))
    h = silu * u
    dh = 1.1 * (np.abs(u) + du) * dg + np.abs(silu) * du + 32 * 2.0 ** -24 * np.abs(h)
    h, dh = h.reshape(len(y), -1, 128), dh.reshape(len(y), -1, 128)
    s = Hs.double().cpu().numpy()
    ref = np.abs(h).max(-1) / 448
    ds = dh.max(-1) / 448 + 4 * 2.0 ** -24 * ref
    assert np.all(np.abs(s - ref) <= ds)
    code = Hq.view(F8).float().cpu().numpy().astype(np.float64).reshape(h.shape)
    t = h / ref[..., None]
    dt = (dh + np.abs(t) * ds[..., None]) / ref[..., None] * 1.01 + 4 * 2.0 ** -24 * np.abs(t)
    assert np.all(np.abs(code - t) <= 0.5 * e4m3_step(np.abs(t) + dt) + dt)


MS = [1, 2, 7, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513]
KS = [16, 48, 128, 144, 272, 1024, 2000, 2048, 4096, 400]
NS = [1, 8, 64, 72, 127, 128, 129, 200, 256, 384, 1000, 1352, 36]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("i", range(32))
def test_product(q, i, dt):
    M, K, N = MS[i % len(MS)], KS[(3 * i + i // 10) % len(KS)], NS[(5 * i) % len(NS)]
    ops = operands(i, M, K, N)
    y, tol = formula(*ops)
    Y = q.qmm_fp8a8_blk128(*ops, out_dtype=dt)
    q.qmm_check_status()
    assert Y.dtype == dt and Y.shape == (M, N)
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(y) + tol)
    assert np.all(np.abs(Y.double().cpu().numpy() - y) <= tol)


@pytest.mark.parametrize("M,K,N", [(1, 5120, 5120), (1000, 2560, 512), (2048, 512, 5120), (4100, 128, 640), (700, 5120, 1536)])
def test_product_of_the_workloads_sizes(q, M, K, N):
    ops = operands(M, M, K, N)
    y, tol = formula(*ops)
    Y = q.qmm_fp8a8_blk128(*ops, out_dtype=F32)
    q.qmm_check_status()
    assert np.all(np.abs(Y.double().cpu().numpy() - y) <= tol)


@pytest.mark.parametrize("M,K,F", [(1, 16, 128), (1, 5120, 1024), (2, 2048, 768), (7, 144, 256), (16, 2000, 384), (17, 128, 128),
                                   (33, 1024, 768), (64, 272, 128), (65, 512, 640), (128, 256, 256), (129, 2048, 768), (200, 48, 256),
                                   (256, 1024, 128), (257, 384, 512), (300, 2560, 1024), (1030, 640, 1280), (2048, 256, 2048)])
def test_swiglu(q, M, K, F):
    ops = operands(M + K, M, K, 2 * F)
    y, tol = formula(*ops)
    Hq, Hs = q.qmm_fp8a8_swiglu_blk128(*ops)
    q.qmm_check_status()
    check_swiglu(Hq, Hs, y, tol)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_columns_past_the_last_whole_wave(q, dt):
    """One wave of full tiles and a remainder that goes in a launch of its own (4 x 20 tiles of
    256 x 256 or 256 x (128 + 128) for 76 pairs of SMs), with a ragged end on both sides."""
    M, K = 1021, 5120
    ops = operands(5, M, K, 4999)
    y, tol = formula(*ops)
    big = torch.full((M + 1, 4999), 7.0, dtype=dt, device="cuda")
    q.qmm_fp8a8_blk128(*ops, out_dtype=dt, Y=big[:M])
    q.qmm_check_status()
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(y) + tol)
    assert np.all(np.abs(big[:M].double().cpu().numpy() - y) <= tol) and bool((big[M] == 7).all())
    if dt == F32:
        ops = operands(6, M, K, 2 * 2560)
        y, tol = formula(*ops)
        Hq, Hs = q.qmm_fp8a8_swiglu_blk128(*ops)
        q.qmm_check_status()
        check_swiglu(Hq, Hs, y, tol)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("M,K,N", [(257, 128, 1), (257, 256, 4097), (600, 128, 66), (700, 128, 777), (1000, 384, 2047),
                                   (1000, 384, 2049), (1000, 384, 2050), (2047, 144, 5117), (4000, 128, 3331)])
def test_rows_of_any_pitch(q, M, K, N, dt):
    """Row pitches that are no multiple of 16 bytes, down to a single element, in tiles of many tokens."""
    ops = operands(M + N, M, K, N)
    y, tol = formula(*ops)
    big = torch.full((M + 2, N), 7.0, dtype=dt, device="cuda")
    q.qmm_fp8a8_blk128(*ops, out_dtype=dt, Y=big[:M])
    q.qmm_check_status()
    if dt == BF16:
        tol = tol + half_bf16_step(np.abs(y) + tol)
    assert np.all(np.abs(big[:M].double().cpu().numpy() - y) <= tol) and bool((big[M:] == 7).all())


@pytest.mark.parametrize("M,N", [(1, 128), (24, 200), (130, 512), (600, 384)])
def test_integers_are_exact(q, M, N):
    """Small integer codes and power-of-two scales: every partial sum is exact."""
    g = torch.Generator().manual_seed(M)
    K = 768
    Xq = torch.randint(-8, 9, (M, K), generator=g).float()
    W = torch.randint(-8, 9, (N, K), generator=g).float()
    Xs = 2.0 ** torch.randint(-2, 3, (M, K // 128), generator=g).float()
    S = 2.0 ** torch.randint(-2, 3, (-(-N // 128), K // 128), generator=g).float()
    ops = [Xq.to(F8).cuda(), Xs.cuda(), W.to(F8).cuda(), S.cuda()]
    y, _ = formula(*ops)
    Y = q.qmm_fp8a8_blk128(*ops, out_dtype=F32)
    assert np.array_equal(Y.double().cpu().numpy(), y)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nan_and_zero_scales_stay_in_their_row(q, M):
    K, N = 512, 384
    Xq, Xs, W, S = operands(M, M, K, N)
    clean = q.qmm_fp8a8_blk128(Xq, Xs, W, S, out_dtype=F32)
    hq, hs = q.qmm_fp8a8_swiglu_blk128(Xq, Xs, *operands(1, 1, K, 512)[2:])
    Z, Zs = Xq.clone(), Xs.clone()
    Z.view(torch.uint8)[1, 300] = 0x7F      # a NaN code
    Zs[2] = 0                               # a token of zeros
    bad = q.qmm_fp8a8_blk128(Z, Zs, W, S, out_dtype=F32)
    bq, bs = q.qmm_fp8a8_swiglu_blk128(Z, Zs, *operands(1, 1, K, 512)[2:])
    assert torch.isnan(bad[1]).all() and not bad[2].any()
    assert torch.isnan(bq.float()[1]).all() and torch.isnan(bs[1]).all()
    assert not bq.float()[2].any() and not bs[2].any()
    keep = [r for r in range(M) if r not in (1, 2)]
    assert torch.equal(bad[keep], clean[keep])
    assert torch.equal(bq.view(torch.uint8)[keep], hq.view(torch.uint8)[keep]) and torch.equal(bs[keep], hs[keep])


@pytest.mark.parametrize("M", [1, 30, 129, 1000])
def test_the_same_every_call_and_nothing_else_written(q, M):
    K, N = 1040, 520
    ops = operands(M, M, K, N)
    big = torch.full((M + 2, N), 7.0, device="cuda")
    Y = big[1:-1]
    ref = q.qmm_fp8a8_blk128(*ops, out_dtype=F32)
    for _ in range(3):
        q.qmm_fp8a8_blk128(*ops, out_dtype=F32, Y=Y)
        assert torch.equal(Y, ref)
    assert (big[0] == 7).all() and (big[-1] == 7).all()


def test_offsets_past_32_bits(q):
    """Outputs and codes whose offsets pass 2^32 elements."""
    M, K, N = 140000, 16, 32768
    Xq, Xs, W, S = operands(3, 64, K, N)
    X = Xq.view(torch.uint8).repeat(M // 64 + 1, 1)[:M].contiguous()
    Y = q.qmm_fp8a8_blk128(X, Xs.repeat(M // 64 + 1, 1)[:M].contiguous(), W, S)
    q.qmm_check_status()
    alone = q.qmm_fp8a8_blk128(Xq, Xs, W, S)
    assert torch.equal(Y[:64], alone)
    n = M % 64
    assert torch.equal(Y[M - n:], alone[:n]) and torch.equal(Y[M - n - 64:M - n], alone)


def test_no_tokens(q):
    _, _, W, S = operands(0, 1, 256, 256)
    X, Xs = torch.empty((0, 256), dtype=F8, device="cuda"), torch.empty((0, 2), device="cuda")
    assert q.qmm_fp8a8_blk128(X, Xs, W, S).shape == (0, 256)
    assert q.qmm_fp8a8_swiglu_blk128(X, Xs, W, S)[0].shape == (0, 128)


@pytest.mark.parametrize("M", [1, 200])
def test_own_stream_and_graph(q, M):
    ops = operands(M, M, 640, 512)
    ref = q.qmm_fp8a8_blk128(*ops)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = q.qmm_fp8a8_blk128(*ops)
        graph = torch.cuda.CUDAGraph()
    s.synchronize()
    assert torch.equal(out, ref)
    Y = torch.zeros_like(ref)
    Hq, Hs = torch.zeros((M, 256), dtype=F8, device="cuda"), torch.zeros((M, 2), device="cuda")
    with torch.cuda.graph(graph):
        q.qmm_fp8a8_blk128(*ops, Y=Y)
        q.qmm_fp8a8_swiglu_blk128(*ops, Hq=Hq, Hs=Hs)
    new = operands(M + 1, M, 640, 512)
    for a, b in zip(ops, new):
        a.copy_(b)
    graph.replay()
    assert torch.equal(Y, q.qmm_fp8a8_blk128(*new))
    check_swiglu(Hq, Hs, *formula(*new))


def test_refusals(q):
    Xq, Xs, W, S = operands(0, 4, 256, 256)
    with pytest.raises(q.QmmError, match="K % 16"):
        q.qmm_fp8a8_blk128(Xq[:, :200].contiguous(), Xs, W[:, :200].contiguous(), S)
    with pytest.raises(q.QmmError, match="F % 128"):
        q.qmm_fp8a8_swiglu_blk128(Xq, Xs, W[:192].contiguous(), S[:1].contiguous())
    with pytest.raises(q.QmmError, match="aligned"):
        q.qmm_fp8a8_blk128(torch.zeros(4 * 256 + 1, dtype=torch.uint8, device="cuda")[1:].view(4, 256), Xs, W, S)
    with pytest.raises(ValueError):
        q.qmm_fp8a8_blk128(Xq[:, ::2], Xs, W, S)
    with pytest.raises(ValueError):
        q.qmm_fp8a8_blk128(Xq, Xs[:, :1].contiguous(), W, S)
    with pytest.raises(ValueError):
        q.qmm_fp8a8_blk128(Xq, Xs, W, S[:1].contiguous())
    with pytest.raises(TypeError):
        q.qmm_fp8a8_blk128(Xq.float(), Xs, W, S)
    with pytest.raises(TypeError):
        q.qmm_fp8a8_blk128(Xq, Xs.double(), W, S)
    with pytest.raises(TypeError):
        q.qmm_fp8a8_blk128(Xq, Xs, W, S, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        q.qmm_fp8a8_blk128(Xq, Xs, W, S, out_dtype=F32, Y=torch.empty((4, 256), dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        q.qmm_fp8a8_blk128(Xq.cpu(), Xs, W, S)
    with pytest.raises(ValueError):
        q.qmm_fp8a8_swiglu_blk128(Xq, Xs, W, S, Hq=torch.empty((4, 256), dtype=F8, device="cuda"))
