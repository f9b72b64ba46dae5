"""The layer operators together, as the training example uses them: gradients of
a stack against 64-bit autograd, and a run that learns."""
import importlib.util
import math
import os

import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("train_blocks", os.path.join(ROOT, "examples", "train_blocks.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def exact_forward(model, p, x):
    s = x
    for i in range(model.n_blocks):
        y = s * (s.square().mean(-1, keepdim=True) + example.EPS).rsqrt() * p[f"norm{i}"]
        z = y @ p[f"w1_{i}"].t() + p[f"b1_{i}"]
        a = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        s = s + a @ p[f"w2_{i}"].t() + p[f"b2_{i}"]
    y = s * (s.square().mean(-1, keepdim=True) + example.EPS).rsqrt() * p["norm"]
    return y @ p["head"].t() + p["head_b"]


@pytest.mark.parametrize("tokens,hidden,ffn,out", [(256, 128, 512, 48), (77, 75, 203, 19), (1, 64, 256, 8)])
def test_gradients_of_a_stack(cuda_device, tokens, hidden, ffn, out):
    """Odd layer sizes put the parameters and gradients on odd addresses of the
    flat vectors.  An 8-bit value is off by 2^-4 of itself at most and evenly
    spread, 3.6% in the square mean, and so is what is linear in it; bfloat16
    steps between the layers add 2^-8 each, six a block.  Together under 8% of a
    gradient's norm."""
    model = example.Blocks(2, hidden, ffn, out)
    flat = model.init("cuda", 3).bfloat16()
    p = model.views(flat)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
    dout = torch.randn(tokens, out, device="cuda", generator=g).bfloat16()
    y, kept = model.forward(p, x)
    grad = torch.full((flat.numel(),), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx = model.backward(p, dout, kept, model.views(grad))
    exact = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = x.double().requires_grad_()
    want = exact_forward(model, exact, x64)
    want.backward(dout.double())
    want = want.detach()
    assert float((y.double() - want).norm() / want.norm()) < 0.03
    assert float((dx.double() - x64.grad).norm() / x64.grad.norm()) < 0.08
    for name, v in model.views(grad).items():
        e = exact[name].grad
        assert bool(torch.isfinite(v.float()).all()), name
        assert float((v.double() - e).norm()) <= 0.08 * float(e.norm()) + 1e-12, name
    assert L.status() == 0


def test_example_learns(cuda_device):
    losses = example.train(workers=2, steps=25, hidden=128, blocks=2, tokens=256, out=32)
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-3:]) < 0.6 * sum(losses[:3]), losses
