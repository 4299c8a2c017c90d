"""moe_expert_stage_fp8 with the pairs and widths of prompts, by the rule's own choice, against the formulas in 64 bits
(check of test_gpu_moe_fp8, its tolerances)."""
import pytest
import torch
from test_gpu_moe_fp8 import check, experts

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


# Chunks of 2048 pairs: up to eight are counted by every CTA for itself, more by a launch of their own.
PAIRS = [(2048, 8), (16384, 1), (16385, 1), (3277, 5), (1025, 16), (5268, 8)]


@pytest.mark.parametrize("how", ["even", "skewed", "holes"])
@pytest.mark.parametrize("E", [128, 512, 77])
@pytest.mark.parametrize("T,k", PAIRS)
def test_grouping_of_many_pairs(q, T, k, E, how):
    check(q, T + E, T, 128, 128, E, k, how=how, dt=BF16)


@pytest.mark.parametrize("how", ["even", "skewed"])
def test_grouping_of_the_longest_prompt(q, how):
    check(q, 5, 21504, 128, 128, 256, 8, how=how, dt=BF16)


@pytest.fixture(scope="module")
def wide():
    return experts(11, 2048, 768, 128)


@pytest.mark.parametrize("T,how,dt,res", [(301, "even", BF16, BF16), (1100, "skewed", F32, BF16), (2048, "even", BF16, None),
                                          (2049, "holes", BF16, F32)])
def test_a_prompt_at_model_width(q, wide, T, how, dt, res):
    check(q, T, T, 2048, 768, 128, 8, how=how, dt=dt, res=res, weights=wide)


def test_a_prompt_of_another_width(q):
    check(q, 3, 900, 2560, 1024, 24, 8, how="skewed", dt=BF16, res=BF16)
