"""The router by scores, the FP8 expert stage and the product with an epilogue refuse tensors that are not on
the current device (no GPU: tensors without storage, on devices that need not be there)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_quantized_weight_route_gb300 as q

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
F32, BF16, F8, U8, I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32

CALLS = {
    "route": (q.moe_route_scored, dict(logits=((4, 8), F32), bias=((8,), F32), live=((1,), I32), ids=((4, 2), I32), w=((4, 2), F32)), dict(k=2)),
    "product": (q.qmm_fp8a8_epilogue_blk128, dict(Xq=((4, 256), F8), Xs=((4, 2), F32), W=((256, 256), F8), S=((2, 2), F32), bias=((256,), BF16),
                                                  R=((4, 256), F32), Y=((4, 256), BF16)), dict(act="silu")),
    "stage": (q.moe_expert_stage_fp8, dict(Xq=((4, 256), F8), Xs=((4, 2), F32), ids=((4, 2), I32), w=((4, 2), F32), Wgu=((3, 256, 256), F8),
                                           Sgu=((3, 2, 2), F32), Wd=((3, 256, 128), F8), Sd=((3, 2, 1), F32), R=((4, 256), BF16),
                                           Y=((4, 256), BF16), ws=((1 << 20,), U8)), {}),
}
CASES = [(call, name) for call, (_, spec, _) in CALLS.items() for name in spec]


@pytest.fixture(autouse=True)
def two_devices(monkeypatch):
    """cuda:0 current, cuda:1 beside it, and no way into the library."""
    monkeypatch.setattr(q, "_current_device", lambda: 0, raising=False)

    def no_call():
        raise AssertionError("the call went through to the library")
    monkeypatch.setattr(q, "lib", no_call)
    with FakeTensorMode():
        yield


@pytest.mark.parametrize("call,name", CASES)
@pytest.mark.parametrize("where", ["cuda:1", "cpu"])
def test_a_tensor_elsewhere_is_refused(call, name, where):
    f, spec, fixed = CALLS[call]
    args = {n: torch.empty(s, dtype=d, device=where if n == name else "cuda:0") for n, (s, d) in spec.items()}
    with pytest.raises((ValueError, TypeError), match=rf"\b{name} "):
        f(**args, **fixed)
