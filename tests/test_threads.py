"""The library may be called from several threads (ctypes lets go of the interpreter's lock for
the call): what its launchers keep between calls is not plain memory (no GPU needed)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_weight_route_gb300",
                    "csrc")


def test_no_plain_static_variables_in_the_launchers():
    """A variable that lives from call to call is atomic (PerDevice), a thread's own, or constant."""
    bad = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not os.path.isfile(path):
            continue
        for n, line in enumerate(open(path), 1):
            code = line.split("//")[0]
            m = re.match(r"\s+static\s+(?!constexpr|const\b|thread_local|PerDevice|assert)([\w:<>]+)\s+\w+\s*(\[|=|;)", code)
            if m:
                bad.append(f"{os.path.basename(path)}:{n}: {code.strip()}")
    assert not bad, bad


HARNESS = r"""
#include "device_cache.h"
#include <thread>
#include <vector>
static qmm::PerDevice cache;
static int ask(int dev) {
    int v = cache.get(dev);
    if (v == 0) cache.set(dev, v = 100 + dev);
    return v;
}
int main() {
    std::vector<std::thread> ts;
    int bad[8] = {};
    for (int t = 0; t < 8; ++t)
        ts.emplace_back([t, &bad] {
            for (int i = 0; i < 1000; ++i) bad[t] += ask(i % qmm::kMaxDevices) != 100 + i % qmm::kMaxDevices;
        });
    for (auto& t : ts) t.join();
    int sum = 0;
    for (int b : bad) sum += b;
    return sum != 0;
}
"""


def test_the_cache_under_the_thread_sanitizer(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "h.cpp", tmp_path / "h"
    src.write_text(HARNESS)
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-pthread", "-I", CSRC, str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    if r.returncode and "tsan" in r.stderr:
        pytest.skip("no thread sanitizer")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    if "unexpected memory mapping" in r.stderr:
        pytest.skip("the thread sanitizer does not run on this kernel")
    assert r.returncode == 0 and "data race" not in r.stderr, r.stderr[-2000:]
