"""What follows the sums of the matrix product is fp32 arithmetic to its last steps, and shows with an fp32 output."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def k2():
    from dense_gqa_decoder_gb300 import k2 as mod
    return mod


@pytest.mark.parametrize("k", [16, 640])
@pytest.mark.parametrize("t", [1, 3, 40, 130, 1000])
def test_swiglu_is_off_by_four_steps(k2, t, k):
    """Gates and factors that arrive exactly.  e^-g is off by a step of 2^-23 (CUDA's bound of expf) and so is the reciprocal
    (PTX's bound of rcp.approx), the sum and the two products by half a step each: 3.5, and what products of those add is far
    below the other half.  Down to -87 everything is a normal number."""
    gen = torch.Generator().manual_seed(k)
    n = 512
    gates = torch.cat([torch.linspace(-87, 87, n - 64), torch.randn(64, generator=gen)]).bfloat16()
    factors = (1 + torch.rand(n, generator=gen)).bfloat16()
    w = torch.zeros(2 * n, k, dtype=torch.bfloat16)
    w[0::2, 0], w[1::2, k - 1] = gates, factors
    x = torch.zeros(t, k, dtype=torch.bfloat16)
    x[:, 0] = x[:, k - 1] = 1
    out = torch.zeros(t, n, device="cuda")
    k2.linear(w.cuda(), x.cuda(), out, activation="swiglu")
    g = gates.double()
    want = (g / (1 + torch.exp(-g)) * factors.double())[None]
    assert ((out.double().cpu() - want).abs() <= want.abs() * 4 * 2.0 ** -23).all()
