"""The three 8-bit operators chained as a user chains them (examples/dense_ffn_fp8.py).

Each block rounds its activations to E4M3 twice (relative half step at most 2^-4, rms
about 2^-5.2 for values spread over a binade); a product of many terms averages the
roundings of its inputs, so one block's output is off by about 2^-5.2 sqrt(2) = 4% rms
against fp32 activations; two blocks, whose inputs are already off, by about 6%.  The
second block's input is also the residual stream, which is exact, so the whole stays
below 12%.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_ffn_fp8.py")
    spec = importlib.util.spec_from_file_location("dense_ffn_fp8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,width,ffn", [(300, 512, 1024), (5, 640, 384), (1, 2048, 768)])
def test_blocks_against_fp32_activations(tokens, width, ffn):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    err = load().main(["--layers", "2", "--width", str(width), "--ffn", str(ffn), "--tokens", str(tokens)])
    assert err <= 0.12


def test_a_token_alone_and_in_a_prompt():
    """A token's norm and codes do not depend on the other tokens; its products may be
    split over K another way, which moves the bf16 output by a rounding at most here and there."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m = load()
    f = m.DenseFFN(1024, 768, 3)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(200, 1024, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(200, 1024, generator=g, device="cuda").to(torch.bfloat16)
    y, rr = f(x, r.clone())
    for t in (0, 77, 199):
        y1, r1 = f(x[t:t + 1], r[t:t + 1].clone())
        assert torch.equal(r1, rr[t:t + 1])
        d = (y1.float() - y[t:t + 1].float()).norm() / y1.float().norm()
        assert d <= 2.0 ** -8
