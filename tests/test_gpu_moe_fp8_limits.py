"""The FP8 mixture-of-experts operators at the ends of fp32's range."""
import pytest
import torch
from test_gpu_moe_fp8 import MANY

pytestmark = pytest.mark.gpu
F32, F8 = torch.float32, torch.float8_e4m3fn
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


@pytest.mark.parametrize("scale", [INF, -INF, float("nan"), 3e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_places_without_an_expert_have_weight_zero_whatever_the_scale(q, scale, score, renorm):
    logits = torch.full((40, 64), -INF, device="cuda")
    logits[:, 3], logits[::2, 50] = 1.0, 0.5
    ids, w = q.moe_route_scored(logits, 4, score=score, renorm=renorm, scale=scale)
    q.qmm_check_status()
    assert ids[0].tolist() == [3, 50, -1, -1] and ids[1].tolist() == [3, -1, -1, -1]
    assert w[ids < 0].eq(0).all() and not w[ids >= 0].eq(0).any()


@pytest.mark.parametrize("plan", [MANY, (0, 16, 1, 1), (0, 64, 1, 1), (0, 128, 1, 1)])
def test_an_intermediate_row_up_to_the_largest_number(q, plan):
    """g = 1.5 and u = 2.6e38: h = silu(g) u = 3.19e38 is finite, where g u is not.  g and u are within 2^-20 (a few
    roundings), silu and the products within 2^-18: s = h / 448, the largest code 448."""
    T, D, F = 20, 128, 128
    X = torch.zeros(T, D, device="cuda").to(F8)
    X[:, 0] = 1.0
    W = torch.zeros(1, 2 * F, D, device="cuda").to(F8)
    W[:, :, 0] = 1.0
    Sgu = torch.tensor([1.5, 2.6e38], device="cuda").view(1, 2, 1)
    Wd = torch.ones(1, D, F, device="cuda").to(F8)
    Sd = torch.full((1, 1, 1), 2.0 ** -20, device="cuda")
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    ws = torch.empty(q.moe_expert_stage_fp8_workspace_size(T, D, F, 1, 1), dtype=torch.uint8, device="cuda")
    q.qmm_dbg_moe_expert_stage_fp8(X, torch.ones(T, 1, device="cuda"), ids, w, W, Sgu, Wd, Sd, plan, out_dtype=F32, ws=ws)
    q.qmm_check_status()
    lay = q.moe_expert_stage_fp8_workspace_layout(T, D, F, 1, 1)
    h = 1.5 / (1 + torch.exp(torch.tensor(-1.5, dtype=torch.float64))) * float(Sgu[0, 1, 0])
    s = q.workspace_view(ws, lay, "Hs", F32, (T, 1)).double().cpu()
    assert ((s - h / 448).abs() <= 2.0 ** -17 * h / 448).all()
    assert q.workspace_view(ws, lay, "Hq", F8, (T, F)).float().eq(448).all()
