"""A layer of norm, router, experts and shared expert captured into one graph and replayed with other inputs and other live
counts: the bits of the same calls outside a graph, and rows of padding that keep residual and shared expert alone."""
import pytest
import torch
from test_gpu_moe_fp8 import experts

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


@pytest.mark.parametrize("T", [1, 4, 48, 700])
def test_a_layer_in_a_graph(q, T):
    D, F, E, k = 512, 256, 32, 4
    routed, shared = experts(1, D, F, E), [t[0] for t in experts(2, D, F, 1)]
    bias, gain = 0.05 * torch.randn(E, device="cuda"), torch.ones(D, device="cuda")

    def inputs(seed, live):
        g = torch.Generator().manual_seed(seed)
        return [torch.randn(T, D, generator=g).to(BF16).cuda(), torch.randn(T, D, generator=g).to(BF16).cuda(),
                (2 * torch.randn(T, E, generator=g)).cuda(), torch.tensor([live], dtype=torch.int32, device="cuda")]

    def layer(x, r, logits, live, ws, experts_too=True):
        n = q.qmm_add_rmsnorm_fp8(x, gain, R=r, Rout=r)
        ids, w = q.moe_route_scored(logits, k, score="sigmoid", bias=bias, groups=4, groups_kept=2, scale=2.5, live=live)
        if experts_too:
            q.moe_expert_stage_fp8(n["Q"], n["S"], ids, w, *routed, R=r, Y=r, ws=ws)
        H = q.qmm_fp8a8_swiglu_blk128(n["Q"], n["S"], *shared[:2])
        return q.qmm_fp8a8_epilogue_blk128(*H, *shared[2:], R=r, Y=r)

    ws = [torch.empty(q.moe_expert_stage_fp8_workspace_size(T, D, F, E, k), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cases = [(1, T), (2, T // 2), (3, 0), (4, T + 5), (1, T)]
    want = [layer(*inputs(*c), ws[0]) for c in cases]
    alone = [layer(*inputs(*c), ws[0], experts_too=False) for c in cases]
    held = inputs(9, T)
    layer(*[t.clone() for t in held], ws[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(*held, ws[1])
    for case, w, a in zip(cases, want, alone):
        for t, new in zip(held, inputs(*case)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        live = min(case[1], T)
        assert torch.equal(w[live:], a[live:]) and (live == 0 or not torch.equal(w[:live], a[:live]))
    q.qmm_check_status()
