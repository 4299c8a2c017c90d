"""What precision the experts' rows have when moe_expert_stage_fp8 adds them, where R cancels the sum.

The rows are read back from the workspace of a call with an fp32 output; R is minus that call's result, so
that little is left.  Against R + sum_j w y in 64 bits from these rows: k + 1 additions in fp32, each
within 2^-24 of the sum of magnitudes, and bf16 output half a bf16 step of what is left.  Only with a bf16
output and the kernel for many rows an expert each row is rounded to 11 bits in a unit that brings the largest of 64
columns to 2^14 .. 2^15: half a step is at most 2^-11 of the value, or below 2^-14 units 2^-25 of one, 2^-39 of the
largest.
"""
import pytest
import torch
from test_gpu_moe_fp8 import MANY, choice, experts, tokens

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


@pytest.mark.parametrize("plan", [MANY, (0, 16, 1, 1), (0, 32, 2, 1), (0, 64, 1, 2), (0, 128, 2, 2)])
@pytest.mark.parametrize("T,D,F,E,k,how", [(1, 272, 256, 4, 2, "even"), (9, 1008, 256, 4, 1, "even"), (301, 272, 256, 3, 2, "holes"), (700, 1040, 256, 5, 8, "twice")])
def test_rows_where_the_sum_cancels(q, T, D, F, E, k, how, plan):
    weights = experts(T, D, F, E)
    args = (*tokens(T + 1, T, D), *choice(T + 2, T, E, k, how), *weights)
    w = args[3].double()
    ws = torch.empty(q.moe_expert_stage_fp8_workspace_size(T, D, F, E, k), dtype=torch.uint8, device="cuda")
    R = -q.qmm_dbg_moe_expert_stage_fp8(*args, plan, out_dtype=F32, ws=ws)
    lay = q.moe_expert_stage_fp8_workspace_layout(T, D, F, E, k)
    y = q.workspace_view(ws, lay, "y", F32, (T * k, D)).double()
    row = q.workspace_view(ws, lay, "row", torch.int32, (T * k,)).long()
    on = (row >= 0).view(T, k, 1)
    terms = torch.where(on, w[:, :, None] * y[row.clamp(min=0)].view(T, k, D), 0.0)
    want, size = R.double() + terms.sum(1), R.double().abs() + terms.abs().sum(1)
    exact = (k + 1) * 2.0 ** -24 * size
    top = torch.nn.functional.pad(terms.abs(), (0, -D % 64)).view(T, k, -1, 64).amax(-1).repeat_interleave(64, -1)[:, :, :D]
    eleven = torch.maximum(2.0 ** -11 * terms.abs(), 2.0 ** -39 * top).sum(1) * (1 + 2.0 ** -10)
    for dt in (F32, BF16):
        Y = q.qmm_dbg_moe_expert_stage_fp8(*args, plan, R=R, out_dtype=dt, ws=ws)
        tol = exact + (eleven if dt == BF16 and plan == MANY else 0.0)
        if dt == BF16:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        assert ((Y.double() - want).abs() <= tol).all()
    q.qmm_check_status()
