"""What a kept norm keeps of device memory."""
import io

import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tensors,numel", [(1, 5), (13, 20000), (90, 300), (110, 300), (388, 300), (800, 70), (30, 3000000)])
def test_norms_kept(cuda_device, tensors, numel):
    g = torch.Generator(device="cuda").manual_seed(tensors)
    t = [torch.randn(numel, device="cuda", generator=g) for _ in range(tensors)]
    kept = [L.grad_norm(t), L.clip_grad_norm(t, 1e30), L.clip_grad_norm(t, 1e30, out=[torch.empty_like(v) for v in t])]
    more = [L.grad_norm(t[i % min(3, tensors):]) for i in range(6)]  # whose workspaces take the place of the first ones'
    want, tol = R.norm(t)
    for n in kept:
        assert n.shape == () and n.untyped_storage().nbytes() <= 1024
        assert abs(float(n) - want) <= tol * want
    for i, n in enumerate(more):
        want, tol = R.norm(t[i % min(3, tensors):])
        assert abs(float(n) - want) <= tol * want
    f = io.BytesIO()
    torch.save(kept[0], f)
    assert f.tell() < 4096
