"""Activations and the gradient through them keep their digits in 32 bits where they
are small."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("cols", [1024, 1023])
@pytest.mark.parametrize("scale", [0.1, 1.0, 8.0, 30.0])
def test_value_relative_error_in_32_bits(cuda_device, act, cols, scale):
    """An exponential within 2 units in the last place whose argument's roundings are
    carried along, a sum, a reciprocal of 1 unit and a product: 2^-21 of the value;
    values below 2^-110 may be cut to 0."""
    g = torch.Generator(device="cuda").manual_seed(1)
    p8 = L.pack8(torch.randn(257, cols, device="cuda", generator=g) * scale)
    want = R.act(R.values(p8.q.view(torch.uint8), p8.scale), act)
    got = L.unpack8(p8, dtype=torch.float32, activation=act).double()
    over = (got - want).abs() / (want.abs() * 2.0 ** -21 + 2.0 ** -110)
    assert float(over.max()) <= 1, float(over.max())


def exact_slope(z, act):
    """Slope in 64 bits without a difference of near numbers: p + z a' p (1 - p) with
    1 - p = logistic(-u)."""
    if act == "silu":
        u, du = z, torch.ones_like(z)
    else:
        c = 2 * (2 / torch.pi) ** 0.5
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
    p, n = torch.sigmoid(u), torch.sigmoid(-u)
    return p, z * du * p * n


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("cols", [1024, 1023])
@pytest.mark.parametrize("scale", [0.1, 1.0, 8.0, 30.0])
def test_slope_relative_error_in_32_bits(cuda_device, act, cols, scale):
    """p has an error of 2^-21 of itself at most: an exponential within 2 units in
    the last place, whose argument's roundings are carried along (2^-22), a sum and a
    reciprocal of 1.5 units (2^-22.4).  The second term has two such factors, a
    polynomial of three roundings and two products: 2^-19.5 of itself.  The product
    with dy is rounded once more, and results below 2^-110 may be cut to 0."""
    g = torch.Generator(device="cuda").manual_seed(1)
    p8 = L.pack8(torch.randn(257, cols, device="cuda", generator=g) * scale)
    z = R.values(p8.q.view(torch.uint8), p8.scale)
    dy = torch.randn(257, cols, device="cuda", generator=g)
    a, b = exact_slope(z, act)
    got = L.activation_grad(dy, p8, act).double()
    d = dy.double()
    tol = d.abs() * (a * 2.0 ** -21 + b.abs() * 2.0 ** -19.5 + (a + b).abs() * 2.0 ** -23) + 2.0 ** -110
    over = (got - d * (a + b)).abs() / tol
    assert float(over.max()) <= 1, float(over.max())
