"""First calls of the FP8 x FP8 products from several threads at once, in a process of their own."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import sys, threading
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import block_quantized_weight_route_gb300 as q
from test_gpu_fp8a8 import operands
SHAPES = [(1, 640, 512), (40, 640, 512), (100, 1024, 640), (700, 512, 1024)]
data = [operands(i, *s) for i, s in enumerate(SHAPES)]
torch.cuda.synchronize()
N = 8
got, errors, start = [[None] * len(SHAPES) for _ in range(N)], [], threading.Barrier(N)
def work(t):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for i in range(len(SHAPES)):
                j = (i + t) % len(SHAPES)
                Xq, Xs, W, S = data[j]
                Y = q.qmm_fp8a8_blk128(Xq, Xs, W, S, out_dtype=torch.float32)
                Hq, Hs = q.qmm_fp8a8_swiglu_blk128(Xq, Xs, W[:W.shape[0] // 256 * 256], S[:W.shape[0] // 256 * 2])
                got[t][j] = (Y, Hq.view(torch.uint8), Hs)
            torch.cuda.current_stream().synchronize()
    except Exception as e:
        errors.append(repr(e))
ts = [threading.Thread(target=work, args=(t,)) for t in range(N)]
[t.start() for t in ts]
[t.join() for t in ts]
assert not errors, errors
q.qmm_check_status()
for j in range(len(SHAPES)):
    for t in range(1, N):
        assert all(torch.equal(a, b) for a, b in zip(got[0][j], got[t][j])), (j, t)
print("threads ok")
"""


def test_first_calls_from_threads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", PROGRAM, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "threads ok" in r.stdout, (r.stdout[-2000:], r.stderr[-2000:])
