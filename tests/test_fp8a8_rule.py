"""The rule that picks an FP8 x FP8 product's tiling (no GPU: its source compiled for the host, with
the numbers of clusters that a GB300 holds at once, as cudaOccupancyMaxActiveClusters gives
them there, in place of the question)."""
import ctypes
import os
import subprocess

import pytest

from block_quantized_weight_route_gb300 import build as qbuild

HARNESS = r"""
#include "gemm_fp8a8.cu"
static int g_broken;   // 1 + the index of a tile that cannot be asked about
namespace qmm {
cudaError_t fp8a8_narrow_at_once(bool gated, int tn, int cs, int dev, int* clusters) {
    static const int fit[9] = {0, 152, 76, 46, 36, 28, 23, 15, 15};
    if (g_broken && tn == 8 << g_broken) return cudaErrorInvalidConfiguration;
    *clusters = fit[cs] * (tn * (gated ? 2 : 1) <= 32 ? 2 : 1);
    return cudaSuccess;
}
}
extern "C" int plan(int M, int K, int N, int gated, int broken, int* f) {
    g_broken = broken;
    qmm::Fp8a8Plans r{};
    const cudaError_t e = qmm::fp8a8_plan(M, K, N, gated != 0, 152, 0, &r);
    const int v[9] = {r.first.pair, r.first.bn, r.first.tn, r.first.cs, r.second.pair, r.second.bn, r.second.tn, r.second.cs, r.split};
    for (int i = 0; i < 9; ++i) f[i] = v[i];
    return (int)e;
}
extern "C" int fits(int M, int K, int N, int gated, const int* f) {
    const qmm::Fp8a8Plans r{{f[0] != 0, f[1], f[2], f[3]}, {f[4] != 0, f[5], f[6], f[7]}, f[8]};
    return qmm::fp8a8_plans_fit(r, M, K, N, gated != 0);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    src, lib = d / "rule.cpp", d / "rule.so"
    src.write_text(HARNESS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(lib))


def plan(rule, M, K, N, gated=False, broken=0):
    f = (ctypes.c_int * 9)()
    return rule.plan(M, K, N, int(gated), broken, f), (tuple(f[:4]), tuple(f[4:8]), f[8])


def test_a_tiling_that_cannot_be_asked_about_is_an_error(rule):
    for gated in (False, True):
        assert plan(rule, 5, 640, 384, gated)[0] == 0
        for broken in (1, 2, 3, 4):
            assert plan(rule, 6 + broken, 640, 384, gated, broken)[0] != 0


@pytest.mark.parametrize("gated", [False, True])
def test_every_plan_can_be_run(rule, gated):
    """What the rule takes is what the launches can do: a K block for each CTA of a cluster, the
    second launch's columns from a weight block on."""
    for M in (1, 2, 17, 64, 65, 128, 129, 300, 513, 1021, 2048, 5268, 21504, 300000):
        for K in (16, 128, 400, 640, 2000, 5120, 17408):
            for N in (128, 640, 768, 1408, 2560, 5120, 17408, 151936):
                for n in (N,) if gated else (N, N - 1, N + 36):
                    e, pl = plan(rule, M, K, n, gated)
                    f = (ctypes.c_int * 9)(*pl[0], *pl[1], pl[2])
                    assert e == 0 and rule.fits(M, K, n, int(gated), f), (M, K, n, pl)


@pytest.mark.parametrize("M,K,N,gated,want", [
    (1, 5120, 5120, False, (0, 0, 16, 6)),
    (300, 5120, 5120, False, (0, 0, 128, 1)),
    (2048, 5120, 5120, False, (1, 256, 0, 0)),
    (5268, 17408, 5120, False, (1, 256, 0, 0)),
    (1, 5120, 17408, True, (0, 0, 16, 2)),
    (2048, 5120, 17408, True, (1, 256, 0, 0)),
])
def test_the_workloads_sizes(rule, M, K, N, gated, want):
    e, pl = plan(rule, M, K, N, gated)
    assert e == 0 and pl[0] == want
    assert pl[2] == (4864 if (M, N) == (2048, 5120) else N)


@pytest.mark.parametrize("M", [1, 2, 5, 16])
@pytest.mark.parametrize("K", [16, 128, 256, 400, 640, 1024, 5120])
@pytest.mark.parametrize("N", [1, 128, 768, 2048, 5120, 17408])
def test_up_to_16_tokens_take_the_narrow_kernel(rule, M, K, N):
    """Faster there than the kernel of 256 tokens a tile, by up to 28% with small K."""
    e, pl = plan(rule, M, K, N)
    assert e == 0 and pl[0][0] == 0 and pl[0][2] == 16 and pl[2] == N, pl
