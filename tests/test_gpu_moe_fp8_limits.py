"""The FP8 mixture-of-experts operators at the ends of fp32's range."""
import pytest
import torch

pytestmark = pytest.mark.gpu
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
