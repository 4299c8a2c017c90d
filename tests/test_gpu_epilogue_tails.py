"""The activations of qmm_fp8a8_epilogue_blk128 against the formulas in 64 bits, relative to the result: small negative
results have their bits too.

The product is 0, so that v is the bias.  In units of 2^-24 relative to the result (half a step of fp32 is one):
  z's rounding: silu none; gelu_tanh two constants, three products and a sum, 6 |z|; gelu's -x^2/2 one product, x^2/2
  __expf: within 2 + 1.173 |argument| units of 2^-23, so 4 + 2.35 |argument|
  the rest of silu and gelu_tanh: sum, shared reciprocal (product 1, approximate reciprocal 2, product 1), two products: 7
  the rest of gelu: 1 / (1 + p x) 5, by whose relative error q changes at most 2.6 times as much, 13; the polynomial's
  fit 4 and its evaluation 6; two products and the difference: 3
silu: 11 + 2.35 |v| <= 16 + 3 |v|; gelu_tanh: 11 + 8.35 |z| <= 16 + 9 |z|; gelu: 30 + 3.35 v^2 / 2 <= 32 + 2 v^2.
Results and exponentials below the smallest normal number may be 0: |v| 2^-125.  bf16: half a bf16 step more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_quantized_weight_route_gb300 as q
    q.build_library()
    return q


def reference(v, act):
    """(the activation of v in 64 bits, its bound in units of 2^-24 of the result)."""
    if act == "gelu":
        return v * 0.5 * torch.special.erfc(-v * 0.5 ** 0.5), 32 + 2 * v * v
    z = v if act == "silu" else 2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    return v / (1 + torch.exp(-z)), (16 + 3 * v.abs()) if act == "silu" else 16 + 9 * z.abs()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("N", [6144, 6143])
@pytest.mark.parametrize("M", [3, 300])
@pytest.mark.parametrize("low,high", [(-12.0, 0.0), (0.0, 12.0), (-0.01, 0.01)])
def test_dense_arguments(q, act, dt, N, M, low, high):
    X = torch.zeros(M, 128, device="cuda").to(F8)
    W = torch.zeros(N, 128, device="cuda").to(F8)
    b = torch.linspace(low, high, N, device="cuda")
    Y = q.qmm_fp8a8_epilogue_blk128(X, torch.ones(M, 1, device="cuda"), W, torch.ones(-(-N // 128), 1, device="cuda"), bias=b, act=act, out_dtype=dt)
    q.qmm_check_status()
    v = b.double()
    want, units = reference(v, act)
    tol = units * 2.0 ** -24 * want.abs() + v.abs() * 2.0 ** -125
    if dt == BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -134
    off = (Y.double() - want).abs()
    assert (off <= tol).all(), (v[(off - tol).amax(0).argmax()].item(), ((off - tol) / want.abs().clamp(min=1e-300)).max().item())
