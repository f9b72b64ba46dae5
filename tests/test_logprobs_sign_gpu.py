"""No log probability is above 0 and no entropy below, whatever place or height a row's
largest logits have, although sums start from a base that may lie below the largest."""
import math

import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu
KINDS = ["high", "alone", "over a floor", "two", "two and the lowest value", "over a slope", "late"]


@pytest.mark.parametrize("vocab", [1, 2, 40, 1000, 2049, 5000, 32000, 50301])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_signs(cuda_device, vocab, kind, dtype):
    rows = 1024
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, device="cuda", generator=g)
    at = torch.randint(0, vocab, (rows, 1), device="cuda", generator=g)
    other = torch.randint(0, vocab, (rows, 1), device="cuda", generator=g)
    # up to ln 1024 + 1: on both sides of what makes a thread raise its base
    h = torch.rand(rows, 1, device="cuda", generator=g) * 7.93
    if kind == "high":
        x.scatter_(1, at, x.amax(1, keepdim=True) + h)
    elif kind == "alone":
        x = torch.full_like(x, -math.inf).scatter_(1, at, h)
    elif kind == "over a floor":
        x = torch.full_like(x, -60.0).scatter_(1, at, h * 3)
    elif kind == "two":
        x = torch.full_like(x, -math.inf).scatter_(1, other, 0.0).scatter_(1, at, h)
    elif kind == "two and the lowest value":
        x = torch.full_like(x, torch.finfo(dtype).min).scatter_(1, other, -20.0).scatter_(1, at, -20.0 + h)
    elif kind == "over a slope":
        x = x.mul_(0.01).sort(1).values.sub_(25.0).scatter_(1, at, -25.0 + 3 * h)
    else:
        x[:, -1:] = x.amax(1, keepdim=True) + h
    x = x.to(dtype)
    r = L.token_logprobs(x, at[:, 0], entropy=True, top=min(3, vocab))
    assert float(r.entropy.min()) >= 0 and float(r.top_logprob.max()) <= 0 and float(r.logprob.max()) <= 0
    r = L.token_logprobs(x, at[:, 0], entropy=True)
    assert float(r.entropy.min()) >= 0 and float(r.logprob.max()) <= 0
    loss, _ = L.token_loss(x, at[:, 0], 1.0)
    assert float(loss.min()) >= 0
