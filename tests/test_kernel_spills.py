"""Registers spilled by the FP8 x FP8 kernels, as the compiler reports them (no GPU needed): a spill in a K loop costs 20
to 40% of a product's time, and no result shows it."""
import re
import subprocess

import pytest

from block_quantized_weight_route_gb300 import build as qbuild

SPILL = re.compile(r"Compiling entry function '(\w+)'.*?(\d+) bytes spill stores, (\d+) bytes spill loads", re.S)


def spills(tmp_path, source):
    """{kernel: (bytes stored, bytes loaded)} of a source file compiled with the library's flags."""
    r = subprocess.run([qbuild.nvcc(), *qbuild.ARCH, *qbuild.NVCC_FLAGS, "-Xptxas", "-v", "-cubin", f"{qbuild.CSRC}/{source}", "-o",
                        str(tmp_path / "x.cubin")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return {name: (int(a), int(b)) for name, a, b in SPILL.findall(r.stderr)}


def test_pair_kernels_without_an_epilogue(tmp_path):
    forms = {}
    for name, spilled in spills(tmp_path, "fp8a8_pair.cu").items():
        bn, gated, bf16, ragged, epilogue = map(int, re.search(r"PairCfgILi(\d+)ELb(\d)ELb(\d)ELb(\d)ELb(\d)E", name).groups())
        if not epilogue:
            forms[bn, gated, bf16, ragged] = spilled
    assert set(forms) == {(bn, 0, bf16, ragged) for bn in (128, 192, 256) for bf16 in (0, 1) for ragged in (0, 1)} | {(256, 1, 1, 0)}
    assert not {f: s for f, s in forms.items() if s != (0, 0)}


@pytest.mark.parametrize("source", ["fp8a8_narrow.cu", "fp8a8_experts.cu"])
def test_kernels_for_few_tokens_and_for_experts(tmp_path, source):
    found = spills(tmp_path, source)
    assert found and not {f: s for f, s in found.items() if s != (0, 0)}
