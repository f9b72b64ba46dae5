"""Gradients of logits whose log-sum-exp has few digits left for what ln S adds (rows
far from 0, targets with nearly all of the probability) against the softmax itself,
not against the rounded log-sum-exp."""
import math

import pytest
import torch

from sparse_communication_sharded_gb300 import ScapeError
from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R
from tests.test_logprobs_gpu import KINDS, logits_of, near, targets_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def far_rows(seed, rows, vocab, offset):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, vocab, device="cuda", generator=g) * 2.0 + offset
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    x[torch.arange(rows, device="cuda"), t] += 12.0 * torch.rand(rows, device="cuda", generator=g)
    t[::5] = -1
    return x, t


def elsewhere(x):
    """Rows for a gradient at other places modulo 16 bytes than x's."""
    return torch.empty(x.shape[0], x.shape[1] + 5, dtype=x.dtype, device="cuda")[:, 1:1 + x.shape[1]]


@pytest.mark.parametrize("offset", [0.0, 300.0, -300.0, 3000.0, -3000.0, 50000.0])
@pytest.mark.parametrize("rows,vocab", [(64, 1000), (9, 5003), (40, 2)])
def test_loss_of_far_rows(cuda_device, rows, vocab, offset):
    """The same bounds wherever the gradient's rows lie."""
    x, t = far_rows(rows, rows, vocab, offset)
    w = torch.rand(rows, device="cuda") + 0.1
    want, tol = R.Rows(x, t).gradient(-w, F32)
    for out in (None, elsewhere(x)):
        near(L.token_loss(x, t, w, out=out)[1], want, tol, "here" if out is None else "elsewhere")


def test_loss_of_wide_far_rows(cuda_device):
    """A row that no blocks hold."""
    x, t = far_rows(3, 2, 700001, 3000.0)
    t[0] = 699999
    w = torch.ones(2, device="cuda")
    near(L.token_loss(x, t, w)[1], *R.Rows(x, t).gradient(-w, F32))


# Two logits a, a - b: S = 1 + e^-b is rounded once (2^-24), its logarithm and the two
# numbers of the log-sum-exp relative to themselves; the exponentials are off by 2^-22
# of themselves, the logarithm, the sum and expm1 by a few 2^-24 of theirs.
def two(a, b):
    x = torch.tensor([[a, a - b]], device="cuda")
    p = 1.0 / (1.0 + math.exp(b))  # the other's
    return x, p, R.E + 2.0 ** -20 * p


@pytest.mark.parametrize("a", [0.5, 20.0, 300.0, -300.0, 3000.0, -3000.0])
@pytest.mark.parametrize("b", [5.0, 10.0, 15.0])
def test_loss_of_a_sure_target(cuda_device, a, b):
    x, p, tol = two(a, b)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    for out in (None, elsewhere(x)):
        dx = L.token_loss(x, t, 1.0, out=out)[1].double()
        assert abs(float(dx[0, 0]) + p) <= tol and abs(float(dx[0, 1]) - p) <= tol


def with_rest(x, t, dlp, dent=None, out=None):
    r = L.token_logprobs(x, t, entropy=dent is not None, lse_rest=True)
    return r, L.token_logprobs_backward(x, t, r.lse, dlp, entropy=r.entropy, dentropy=dent, out=out, lse_rest=r.lse_rest)


def bounds(x, t, dlp, dtype, r=None, dent=None):
    """The oracle's, whose own sums have no rounded log-sum-exp.  Beside the entropy, log
    p is off by what ln S is and by the roundings of its difference and of its rest."""
    o = R.Rows(x, t)
    if dent is None:
        return o.gradient(dlp, dtype)
    want, tol = o.gradient(dlp, dtype, r.entropy, dent)
    off = o.ds + 4 * R.E * (o.ln_s + R.B + r.entropy.double().abs())
    return want, tol + dent.double().abs()[:, None] * o.p * off[:, None]


@pytest.mark.parametrize("offset", [0.0, 300.0, -300.0, 3000.0, -3000.0, 50000.0])
@pytest.mark.parametrize("rows,vocab", [(64, 1000), (9, 5003), (40, 2), (2, 262147)])
def test_gradient_of_far_rows(cuda_device, rows, vocab, offset):
    x, t = far_rows(rows + 1, rows, vocab, offset)
    g = torch.Generator(device="cuda").manual_seed(rows)
    dlp, dent = (torch.randn(rows, device="cuda", generator=g) for _ in range(2))
    for out in (None, elsewhere(x)):
        r, dx = with_rest(x, t, dlp, out=out)
        near(dx, *bounds(x, t, dlp, F32), "log probability's")
        r, dx = with_rest(x, t, dlp, dent, out)
        near(dx, *bounds(x, t, dlp, F32, r, dent), "with the entropy's")
    own = x.clone()
    assert with_rest(own, t, dlp, dent, own)[1] is own
    near(own, *bounds(x, t, dlp, F32, r, dent), "in place")


@pytest.mark.parametrize("rows,vocab", [(1, 1), (5, 7), (4, 255), (7, 1000), (40, 8191), (300, 257)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_all_kinds_with_the_rest(cuda_device, rows, vocab, kind, dtype):
    x = logits_of(rows * vocab, rows, vocab, dtype, gap=3 if kind == "normal" else 0, kind=kind)
    t = targets_of(rows, rows, vocab)
    g = torch.Generator(device="cuda").manual_seed(rows)
    dlp, dent = (torch.randn(rows, device="cuda", generator=g) for _ in range(2))
    near(with_rest(x, t, dlp)[1], *bounds(x, t, dlp, dtype))
    r, dx = with_rest(x, t, dlp, dent)
    near(dx, *bounds(x, t, dlp, dtype, r, dent))


@pytest.mark.parametrize("a", [0.5, 20.0, 300.0, -300.0, 3000.0, -3000.0])
@pytest.mark.parametrize("b", [5.0, 10.0, 15.0])
def test_gradient_of_a_sure_target(cuda_device, a, b):
    x, p, tol = two(a, b)
    t = torch.zeros(1, dtype=torch.int64, device="cuda")
    _, dx = with_rest(x, t, torch.ones(1, device="cuda"))
    assert abs(float(dx[0, 0]) - p) <= tol and abs(float(dx[0, 1]) + p) <= tol


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_without_a_finite_sum(cuda_device, dtype):
    """Masked whole with the lowest value, nothing but -infinity, NaN, no target, a
    target out of range, side by side; five results and, if asked for, the rest."""
    x = torch.randn(6, 900, device="cuda").to(dtype)
    x[1], x[2], x[3, 5] = torch.finfo(dtype).min, -math.inf, math.nan
    t = torch.tensor([3, 4, 5, 6, -1, 900], device="cuda")
    dlp = torch.ones(6, device="cuda")
    r, dx = with_rest(x, t, dlp)
    assert L.token_logprobs(x, t).lse_rest is None
    full = L.token_logprobs(x, t, entropy=True, top=3, lse_rest=True)
    plain = L.token_logprobs(x, t, entropy=True, top=3)
    assert full.lse_rest.shape == (6,)
    assert all(torch.equal(a.nan_to_num(7.5), b.nan_to_num(7.5)) for a, b in zip(full, plain))
    assert len(r) == 5 and r.lse_rest.shape == (6,) and r.lse_rest.dtype == F32
    assert float(r.lse_rest[2]) == 0
    assert abs(float(r.lse_rest[1]) - math.log(900)) <= 8 * R.E * math.log(900)
    for i in (3, 5):
        assert bool(torch.isnan(dx[i]).all())
    assert not bool(dx[4].any())
    good = [0, 1, 2]
    near(dx[good], *R.Rows(x[good], t[good]).gradient(dlp[good], dtype))


def test_refusals_of_the_rest(cuda_device):
    x, t = torch.zeros(6, 50, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    f = torch.zeros(6, device="cuda")
    for bad in (f[:5], f.double(), f.cpu(), torch.zeros(12, device="cuda")[::2], 3.0):
        with pytest.raises(ValueError):
            L.token_logprobs_backward(x, t, f, f, lse_rest=bad)
    buf = torch.zeros(6, 50, device="cuda")
    with pytest.raises(ScapeError):
        L.token_logprobs_backward(x, t, f, f, out=buf, lse_rest=buf.view(-1)[:6])
