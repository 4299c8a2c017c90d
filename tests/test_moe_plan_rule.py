"""The rule that picks the FP8 expert stage's kernel and tiling (no GPU: its source compiled for the host,
as in test_fp8a8_rule)."""
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
extern "C" int plan(int T, int D, int F, int E, int k, int broken, int* f) {
    g_broken = broken;
    qmm::MoePlan r{};
    const cudaError_t e = qmm::moe_plan(T, D, F, E, k, 152, 0, &r);
    const int v[4] = {r.many, r.tn, r.cs_gate_up, r.cs_down};
    for (int i = 0; i < 4; ++i) f[i] = v[i];
    return (int)e;
}
extern "C" int fits(int T, int D, int F, int E, int k, const int* f) {
    return qmm::moe_plan_fits(qmm::MoePlan{f[0] != 0, f[1], f[2], f[3]}, T, D, F, E, k);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("moe_rule")
    src, lib = d / "rule.cpp", d / "rule.so"
    src.write_text(HARNESS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(lib))


def plan(rule, T, D, F, E, k, broken=0):
    f = (ctypes.c_int * 4)()
    return rule.plan(T, D, F, E, k, broken, f), tuple(f)


def test_every_plan_can_be_run(rule):
    """A K block for each CTA of a cluster, and no more tiles than the grid's third dimension has room for."""
    for T in (1, 2, 5, 32, 33, 301, 5268, 21504, 262144):
        for D in (16, 128, 400, 2048, 2560, 1 << 20):
            for F in (128, 768, 1024, 1 << 20):
                for E in (1, 8, 60, 128, 512):
                    for k in (1, 2, 8, 16):
                        if T * k > 1 << 22 or E * max(2 * F, D) > 2 ** 31 - 512:
                            continue
                        e, pl = plan(rule, T, D, F, E, k)
                        assert e == 0 and rule.fits(T, D, F, E, k, (ctypes.c_int * 4)(*pl)), (T, D, F, E, k, pl)


def test_a_tiling_that_cannot_be_asked_about_is_an_error(rule):
    for broken in (1, 2, 3, 4):
        assert plan(rule, 40 + broken, 640, 384, 6, 2, broken)[0] != 0


@pytest.mark.parametrize("T,D,F,E,k,many", [(1, 2048, 768, 128, 8, 0), (8, 2048, 768, 128, 8, 0), (64, 2048, 768, 64, 8, 0),
                                            (64, 2048, 768, 16, 8, 0), (301, 2048, 768, 128, 8, 1), (512, 2048, 768, 128, 8, 1),
                                            (200, 2048, 2048, 8, 8, 1), (5268, 2048, 768, 128, 8, 1), (21504, 2560, 1024, 256, 8, 1)])
def test_the_faster_kernel_of_the_measured_shapes(rule, T, D, F, E, k, many):
    """Where the two kernels were measured against each other and differ by more than a few percent, the faster one."""
    assert plan(rule, T, D, F, E, k)[1][0] == many


def test_the_answer_does_not_hang_on_the_one_before(rule):
    """(The last shapes' plans are kept.)"""
    shapes = [(T, D, 768, E, k) for T in (1, 7, 301, 5268) for D in (2048, 2064) for E in (8, 128) for k in (2, 8)]
    first = [plan(rule, *s) for s in shapes]
    assert [plan(rule, *s) for s in reversed(shapes)] == first[::-1]


def test_the_combine_goes_by_the_devices_sms(tmp_path):
    src, lib = tmp_path / "combine.cpp", tmp_path / "combine.so"
    src.write_text('#include "qmm_internal.h"\nextern "C" int splits(int T, int sms) { return qmm::moe_combine_splits(T, sms); }\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(qbuild.nvcc())), "include")
    r = subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", qbuild.CSRC, "-I", cuda, str(src), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rule = ctypes.CDLL(str(lib))
    for sms in (1, 76, 152):
        assert [rule.splits(T, sms) for T in (1, 8 * sms, 8 * sms + 1)] == [1, 1, 0]
