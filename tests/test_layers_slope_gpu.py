"""Activations in 32 bits keep their digits where they are small."""
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
