"""A few rows through the linear layer: which of the operands decides how the
weight is read."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
@pytest.mark.parametrize("k,n", [(1024, 4096), (1000, 520), (4104, 129), (8, 5)])
def test_input_rows_of_any_alignment(cuda_device, rows, k, n):
    """x is read value by value, so where its rows start changes nothing: the same
    bits from a slice at an odd place of a wider buffer."""
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn(rows, k, device="cuda", generator=g).bfloat16()
    w = (torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16()
    wide = torch.zeros(rows, k + 5, device="cuda", dtype=torch.bfloat16)
    wide[:, 3:3 + k] = x
    y, z8 = L.linear(x, w, activation="silu", keep_pre=True)
    y2, z82 = L.linear(wide[:, 3:3 + k], w, activation="silu", keep_pre=True)
    assert torch.equal(y, y2)
    assert torch.equal(z8.q.view(torch.uint8), z82.q.view(torch.uint8)) and torch.equal(z8.scale, z82.scale)
    z = x.double() @ w.double().t()
    a = R.act(z, "silu")
    tol = a.abs() * (R.U_BF16 + R.ACT_REL) + 1.2 * (x.double().abs() @ w.double().abs().t()) * (k + 2) * 2.0 ** -23
    assert bool(((y.double() - a).abs() <= tol).all())
    dy = torch.randn(rows, n, device="cuda", generator=g).bfloat16()
    wide = torch.zeros(rows, n + 5, device="cuda", dtype=torch.bfloat16)
    wide[:, 3:3 + n] = dy
    assert torch.equal(L.linear_backward_input(dy, w), L.linear_backward_input(wide[:, 3:3 + n], w))
