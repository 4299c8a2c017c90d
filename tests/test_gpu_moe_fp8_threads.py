"""First calls of the FP8 expert stage, the router and the product with an epilogue from several threads at once,
each on a stream and with workspaces of its own, in a process of their own."""
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
from test_gpu_moe_fp8 import choice, experts, tokens
SHAPES = [(1, 256, 128, 8, 2), (40, 256, 128, 4, 2), (300, 256, 256, 2, 1), (700, 384, 128, 3, 2)]
stage = [(*tokens(i, s[0], s[1]), *choice(i, s[0], s[3], s[4], "even"), *experts(i, s[1], s[2], s[3])) for i, s in enumerate(SHAPES)]
product = [operands(i, s[0], s[1], 512) for i, s in enumerate(SHAPES)]
logits = [torch.randn(s[0], 64, device="cuda") for s in SHAPES]
bias = torch.randn(64, device="cuda")
torch.cuda.synchronize()
N = 8
got, errors, start = [[None] * len(SHAPES) for _ in range(N)], [], threading.Barrier(N)
def work(t):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for i in range(len(SHAPES)):
                j = (i + t) % len(SHAPES)
                got[t][j] = (q.moe_expert_stage_fp8(*stage[j]), q.qmm_fp8a8_epilogue_blk128(*product[j], act="silu"),
                             *q.moe_route_scored(logits[j], 4, score="sigmoid", bias=bias, groups=4, groups_kept=2))
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
