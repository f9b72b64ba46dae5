"""The layer operators beside torch's autograd: no graph is lost without a word."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rand(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(BF)


def calls():
    x, w, b, dy, p = rand(1, 16, 64), rand(2, 48, 64), rand(3, 48), rand(4, 16, 48), None
    p = L.pack8(x)
    wn, rstd = torch.ones(64, device="cuda"), torch.ones(16, device="cuda")
    return [
        (L.pack8, (x,), 1), (L.activation_grad, (x, p, "gelu"), 1), (L.add_rmsnorm, (x, wn, x), 3),
        (L.add_rmsnorm_backward, (x, x, wn, rstd, x), 5), (L.linear, (x, w, b, dy), 4),
        (L.linear_backward_input, (dy, w), 2), (L.linear_backward_weight, (dy, x), 2),
    ]


def test_tensors_that_require_grad(cuda_device):
    """Each tensor argument of each operator, one at a time."""
    for f, args, tensors in calls():
        for i in range(tensors):
            if not torch.is_tensor(args[i]):
                continue
            given = list(args)
            given[i] = args[i].clone().requires_grad_()
            with pytest.raises(ValueError, match="requires grad"):
                f(*given)
            with torch.no_grad():
                f(*given)
        f(*args)


def test_outputs_that_require_grad(cuda_device):
    x, w, dy = rand(1, 16, 64), rand(2, 48, 64), rand(4, 16, 48)
    leaf = torch.zeros(48, 64, device="cuda", dtype=BF, requires_grad=True)
    with pytest.raises(ValueError, match="requires grad"):
        L.linear_backward_weight(dy, x, dweight=leaf)
    with torch.no_grad():
        L.linear_backward_weight(dy, x, dweight=leaf)
    assert torch.equal(leaf, L.linear_backward_weight(dy, x))
    del w


def test_in_an_autograd_function(cuda_device):
    """As a user records them: the operators' gradients under torch's graph."""
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return L.linear(x, w)

        @staticmethod
        def backward(ctx, dy):
            x, w = ctx.saved_tensors
            return L.linear_backward_input(dy, w), L.linear_backward_weight(dy, x)

    x, w = rand(1, 16, 64).requires_grad_(), rand(2, 48, 64).requires_grad_()
    Linear.apply(x, w).float().square().sum().backward()
    y = x.detach().double() @ w.detach().double().t()
    for got, want in ((x.grad, 2 * y @ w.detach().double()), (w.grad, 2 * y.t() @ x.detach().double())):
        assert float((got.double() - want).norm() / want.norm()) < 0.02  # three roundings to bfloat16


def test_outputs_written_in_place_are_seen(cuda_device):
    """autograd refuses a backward pass through a saved value that a call overwrote."""
    x, w, dy, res = rand(1, 16, 64), rand(2, 48, 64), rand(4, 16, 48), rand(5, 16, 48)
    rstd, wn = torch.ones(16, device="cuda"), torch.ones(64, device="cuda")
    dw, db, g, own = torch.empty_like(w), torch.empty(48, device="cuda", dtype=BF), torch.empty(64, device="cuda"), x.clone()
    p = L.pack8(x)
    for call, tensors in [(lambda: L.linear(x, w, residual=res, out=res), [res]),
                          (lambda: L.linear_backward_input(dy, w, out=own), [own]),
                          (lambda: L.linear_backward_weight(dy, x, dweight=dw, dbias=db), [dw, db]),
                          (lambda: L.add_rmsnorm_backward(own, x, wn, rstd, dweight=g, out=own), [own, g]),
                          (lambda: L.activation_grad(own, p, "gelu", out=own), [own]),
                          (lambda: L.unpack8(p, out=own), [own])]:
        before = [t._version for t in tensors]
        call()
        assert all(t._version > v for t, v in zip(tensors, before))
    a = rand(6, 16, 48).requires_grad_()
    saved = res.clone()
    y = (a * saved).sum()
    L.linear(x, w, out=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        t = torch.empty(16, 48, device="cuda", dtype=BF)
        L.linear(x, w, out=t)
