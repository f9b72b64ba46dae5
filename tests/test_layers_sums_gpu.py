"""Bias gradients on both sides of the rule that puts their sums beside the
unpacking of the input or in a launch of their own (at most 12288 rows, or rows of
3 k + 2 n >= 3200 bytes: beside)."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,k,n", [(12288, 64, 64), (12289, 64, 64), (12289, 40, 1000), (20000, 33, 1544),
                                      (20000, 64, 1504), (20000, 1024, 64), (20000, 1024, 63), (40000, 256, 200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_bias_gradient(cuda_device, rows, k, n, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + k + n)
    dy = torch.randn(rows, n, device="cuda", generator=g).bfloat16()
    p = L.pack8(torch.randn(rows, k, device="cuda", generator=g).bfloat16())
    db = torch.empty(n, dtype=dtype, device="cuda")
    dw = L.linear_backward_weight(dy, p, dbias=db, grad_dtype=dtype)
    d = dy.double()
    # 32-bit sums, one rounding of 2^-24 a term at most, and the result's own
    tol = d.sum(0).abs() * R.u_of(dtype) + d.abs().sum(0) * rows * 2.0 ** -24
    assert bool(((db.double() - d.sum(0)).abs() <= tol).all())
    assert torch.equal(dw, L.linear_backward_weight(dy, p, grad_dtype=dtype))
