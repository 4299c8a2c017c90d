"""qmm_fp8a8_epilogue_blk128 with an output and a residual whose offsets pass 32 bits: tolerances of
test_gpu_fp8a8_epilogue, on the GPU."""
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
    yield q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("plan", [None, (0, 0, 128, 1)])
@pytest.mark.parametrize("N,res,dt", [(33000, F32, BF16), (33001, BF16, F32)])
def test_more_than_2_to_31_outputs(q, N, res, dt, plan):
    M, K = 66000, 144
    g = torch.Generator("cuda").manual_seed(N)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    X, W = (rand(M, K) * 100).clamp(-448, 448).to(F8), (rand(N, K) * 60).clamp(-448, 448).to(F8)
    Xs, S = torch.exp(rand(M, 2)) * 2.0 ** -7, (1 + rand(-(-N // 128), 2).abs()) * 2.0 ** -13
    b, R = rand(N), torch.empty(M, N + 8, dtype=res, device="cuda").normal_(generator=g)[:, :N]
    kw = dict(bias=b, act="silu", R=R, out_dtype=dt)
    Y = q.qmm_fp8a8_epilogue_blk128(X, Xs, W, S, **kw) if plan is None else \
        q.qmm_dbg_fp8a8_epilogue_blk128(X, Xs, W, S, (plan, (0, 0, 0, 0), N), **kw)
    q.qmm_check_status()
    w = W.double() * S.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    for m in [*range(0, M, 16000), M - 300]:   # 300 rows of every 16000, and the last
        rows = slice(m, m + 300)
        x = X[rows].double() * Xs[rows].double().repeat_interleave(128, 1)[:, :K]
        v, tol = x @ w.t() + b.double(), (128 + 2 + 4) * 2.0 ** -23 * (x.abs() @ w.abs().t())
        tol += 2.0 ** -24 * (v.abs() + tol)
        tol = 1.13 * tol + 32 * 2.0 ** -24 * v.abs()
        y = torch.nn.functional.silu(v) + R[rows].double()
        tol += 2.0 ** -24 * (y.abs() + tol)
        if dt == BF16:
            tol += 2.0 ** -8 * (y.abs() + tol)
        assert ((Y[rows].double() - y).abs() <= tol).all(), m
