"""moe_expert_stage_fp8 and moe_route_scored at the largest sizes that their shape checks let pass: pairs, widths, and
weights whose offsets pass 32 bits."""
import pytest
import torch
from test_gpu_moe_fp8 import MANY, check, choice, experts, tokens

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


@pytest.mark.parametrize("plan", [None, MANY, (0, 128, 1, 1)])
@pytest.mark.parametrize("how", ["even", "holes"])
def test_the_most_pairs(q, how, plan):
    """2^22 pairs.  Tokens repeat a few patterns, and a row's sums do not depend on its place, so that the rows come from a
    small call of the same kernels; k + 1 additions in fp32 are left, each within 2^-24 of the sum of magnitudes."""
    T, k, E, D, F, n = 1 << 18, 16, 512, 16, 128, 5
    weights = experts(1, D, F, E)
    Xq, Xs = tokens(2, n, D)
    plan = plan or q.qmm_dbg_moe_fp8_plan(T, D, F, E, k)
    each = torch.arange(n * E, device="cuda")
    rows = q.qmm_dbg_moe_expert_stage_fp8(Xq.view(torch.uint8)[each // E].view(F8), Xs[each // E], (each % E).int()[:, None], torch.ones(n * E, 1, device="cuda"), *weights, plan, out_dtype=F32)
    rows = rows.double().view(n, E, D)
    ids, w = choice(3, T, E, k, how)
    of = torch.arange(T, device="cuda") % n
    Y = q.qmm_dbg_moe_expert_stage_fp8(Xq.view(torch.uint8)[of].view(F8), Xs[of], ids, w, *weights, plan, out_dtype=F32)
    q.qmm_check_status()
    on = (ids >= 0) & (ids < E)
    terms = torch.where(on[:, :, None], w.double()[:, :, None] * rows[of[:, None], torch.where(on, ids, 0).long()], 0.0)
    assert ((Y.double() - terms.sum(1)).abs() <= (k + 1) * 2.0 ** -24 * terms.abs().sum(1)).all()


@pytest.mark.parametrize("D,F,plan", [(D, F, plan) for D, F, cs in ((1 << 20, 128, (8, 1)), (16, 1 << 20, (1, 8)))
                                      for plan in (None, MANY, (0, 16, *cs), (0, 128, 1, 1))])
def test_the_widest_rows(q, D, F, plan):
    check(q, 4, 3, D, F, 2, 2, dt=F32, res=BF16, plan=plan)


@pytest.mark.parametrize("plan", [MANY, (0, 16, 1, 4), (0, 64, 1, 1)])
def test_weights_whose_offsets_pass_32_bits(q, plan):
    """17 GB of gate and up codes in 2^30 rows, 8.6 GB of down codes."""
    D, F, E = 16, 1 << 20, 512
    g = torch.Generator("cuda").manual_seed(0)
    Wgu, Wd = (torch.empty(s, dtype=F8, device="cuda") for s in ((E, 2 * F, D), (E, D, F)))
    for e in range(E):
        for W in (Wgu, Wd):
            W[e] = (torch.randn(W.shape[1:], generator=g, device="cuda") * 60).clamp(-448, 448).to(F8)
    Sgu = (1 + torch.rand(E, 2 * F // 128, 1, generator=g, device="cuda")) * 2.0 ** -11
    Sd = (1 + torch.rand(E, 1, F // 128, generator=g, device="cuda")) * 2.0 ** -16
    check(q, 6, 5, D, F, E, 2, dt=F32, res=F32, weights=(Wgu, Sgu, Wd, Sd), plan=plan)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_of_many_tokens(q, score):
    """2^22 tokens of 8 experts (equal logits to the lower index)."""
    l = torch.randn(1 << 22, 8, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    ids, w = q.moe_route_scored(l, 3, score=score)
    q.qmm_check_status()
    top = torch.sort(l.double(), dim=1, descending=True, stable=True).indices[:, :3]
    assert torch.equal(ids.long(), top)
    s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
    s = s.gather(1, top)
    s = s / s.sum(1, keepdim=True)
    far = (l.max() - l.min()).item()
    assert ((w.double() - s).abs() <= (48 + far) * 2.0 ** -23 * s).all()
