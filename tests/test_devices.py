"""Tensors that are not on the current device are refused by every call (no GPU: tensors
without storage, on devices that need not be there).

The library launches on the current device, with the tilings and the error word of that
device: with operands elsewhere it would hand one GPU the addresses of another.
"""
import os
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import block_quantized_weight_route_gb300 as q

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
F32, BF16, F8, U8, I8, I16, I32 = (torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int8,
                                   torch.int16, torch.int32)


@pytest.fixture(autouse=True)
def two_devices(monkeypatch):
    """cuda:0 current, cuda:1 beside it, and no way into the library."""
    monkeypatch.setattr(q, "_current_device", lambda: 0, raising=False)

    def no_call():
        raise AssertionError("the call went through to the library")
    monkeypatch.setattr(q, "lib", no_call)
    with FakeTensorMode():
        yield


# call: (function, {argument: (shape, type)}, fixed arguments)
CALLS = {
    "norm fp8": (q.qmm_add_rmsnorm_fp8, dict(X=((4, 256), BF16), G=((256,), BF16), R=((4, 256), BF16), Rout=((4, 256), BF16),
                                             Q=((4, 256), F8), S=((4, 2), F32), Y=((4, 256), BF16)), {}),
    "norm q8_1": (q.qmm_add_rmsnorm_q8_1, dict(X=((4, 256), F32), G=((256,), F32), R=((4, 256), F32),
                                               Rout=((4, 256), F32), Y=((4, 256), BF16)), {}),
    "fp8 x fp8": (q.qmm_fp8a8_blk128, dict(Xq=((4, 256), F8), Xs=((4, 2), F32), W=((256, 256), F8), S=((2, 2), F32),
                                           Y=((4, 256), BF16)), {}),
    "fp8 swiglu": (q.qmm_fp8a8_swiglu_blk128, dict(Xq=((4, 256), F8), Xs=((4, 2), F32), Wgu=((256, 256), F8),
                                                   Sgu=((2, 2), F32), Hq=((4, 128), F8), Hs=((4, 1), F32)), {}),
    "w4a16": (q.qmm_w4a16, dict(X=((4, 64), BF16), Wc=((64, 32), U8), Ws=((64, 4), U8), Y=((4, 64), F32), ws=((256,), U8)),
              dict(scale2=1.0)),
    "fp8": (q.qmm_fp8_blk128, dict(X=((4, 128), BF16), W=((128, 128), U8), S=((1, 1), F32), Y=((4, 128), BF16),
                                   ws=((256,), U8)), {}),
    "q8": (q.qmm_q8_0_q8_1, dict(Xq=((4, 64), I8), Xd=((4, 2), I16), Wq=((32, 64), I8), Wd=((32, 2), I16), ws=((256,), U8)), {}),
    "route": (q.moe_route_permute, dict(logits=((4, 8), F32), ws=((256,), U8)), dict(k=2)),
    "stage": (q.moe_expert_stage_w4_iq4, dict(X=((4, 128), BF16), logits=((4, 2), F32), Wgu_c=((2, 256, 64), U8),
                                              Wgu_s=((2, 256, 8), U8), gu_scale2=((2,), F32), Wd_idx=((2, 128, 64), U8),
                                              Wd_s=((2, 128, 4), I16), ws=((256,), U8), Y=((4, 128), F32)), dict(k=1)),
    "down": (q.qmm_dbg_down_iq4, dict(Hq=((4, 128), I8), Hd=((4, 4), I16), offsets=((3,), I32), Wd_idx=((2, 128, 64), U8),
                                      Wd_s=((2, 128, 4), I16), ws=((256,), U8)), {}),
    "combine": (q.qmm_dbg_combine, dict(Yslot=((4, 128), F32), row=((2, 2), I32), w=((2, 2), F32)), {}),
}


def tensors(spec, elsewhere):
    return {k: torch.empty(shape, dtype=dt, device="cuda:1" if k in elsewhere else "cuda:0") for k, (shape, dt) in spec.items()}


@pytest.mark.parametrize("name,arg", [(n, a) for n, c in CALLS.items() for a in c[1]])
def test_one_tensor_elsewhere(name, arg):
    f, spec, fixed = CALLS[name]
    with pytest.raises(ValueError, match="current device is cuda:0"):
        f(**tensors(spec, {arg}), **fixed)


@pytest.mark.parametrize("name", CALLS)
def test_all_tensors_on_another_device(name):
    f, spec, fixed = CALLS[name]
    with pytest.raises(ValueError, match="current device is cuda:0"):
        f(**tensors(spec, set(spec)), **fixed)


@pytest.mark.parametrize("name", ["norm fp8", "norm q8_1", "fp8 x fp8", "fp8 swiglu"])
def test_tensors_on_the_host(name):
    f, spec, fixed = CALLS[name]
    for arg in spec:
        ts = tensors(spec, set())
        ts[arg] = torch.empty(spec[arg][0], dtype=spec[arg][1])
        with pytest.raises(TypeError, match="CUDA tensor"):
            f(**ts, **fixed)


def test_a_stream_of_another_device(monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        q._stream(torch.device("cuda", 1))


def test_import_with_a_torch_without_cuda():
    """The package is imported (to build, to ask for sizes) where torch has no CUDA."""
    program = ("import torch\n"
               "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
               "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
               "import block_quantized_weight_route_gb300 as q\n"
               "try: q.qmm_fp8a8_blk128(torch.zeros(1, 16), None, None, None)\n"
               "except TypeError as e: assert 'CUDA tensor' in str(e)\n"
               "else: raise AssertionError\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
