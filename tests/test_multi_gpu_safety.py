"""What code that may run on several GPUs at once does not do (no GPU needed).

bench.py runs the library on every rank of a multi-GPU job, so no kernel of it may
copy to several CTAs at once: a multicast copy is for code that only ever has one GPU.
"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_weight_route_gb300",
                    "csrc")


def instructions():
    """(file, text) of every inline PTX statement's string, its pieces joined."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if not os.path.isfile(path):
            continue
        with open(path) as f:
            src = f.read()
        for m in re.finditer(r"\basm\b[^(]*\((\s*(?:\"(?:[^\"\\]|\\.)*\"\s*)+)", src):
            yield os.path.basename(path), "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))


def test_the_scan_sees_the_copies():
    assert sum("cp.async.bulk.tensor" in t for _, t in instructions()) >= 2


def test_no_multicast_copy():
    bad = [(f, t) for f, t in instructions() if "cp.async.bulk" in t and "multicast" in t]
    assert not bad, bad
