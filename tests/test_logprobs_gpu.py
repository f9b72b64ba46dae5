"""Log probabilities of tokens, entropy, alternatives, their gradient and the loss
against plain 64-bit formulas."""
import math

import pytest
import torch
import torch.nn.functional as F

from sparse_communication_sharded_gb300 import ScapeError
from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def logits_of(seed, rows, vocab, dtype, gap=0, kind="normal"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, vocab + gap, device="cuda", generator=g) * 3.0
    if kind == "peaked":
        x[:, seed % vocab] += 40.0
    elif kind == "masked":
        x[torch.rand(x.shape, device="cuda", generator=g) < 0.7] = -INF
    elif kind == "lowest":
        x[torch.rand(x.shape, device="cuda", generator=g) < 0.7] = torch.finfo(dtype).min
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "rising":
        x = x.sort(1).values
    elif kind == "large":
        x = x * 1e37
    elif kind == "empty":
        x[::2] = -INF
        x[1::2, :-1 - gap] = -INF
    return x.to(dtype)[:, :vocab]


def targets_of(seed, rows, vocab, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    t[::4] = torch.randint(-3, 0, (t[::4].numel(),), device="cuda", generator=g)
    return t.to(dtype)


def near(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    # past float32's range (2^128 less half a step of 2^104) a value rounds to infinity
    want = torch.where(want.abs() >= 2.0 ** 128 - 2.0 ** 103, want.sign() * INF, want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    d = torch.where(inf | torch.isnan(want), 0.0, (got - want).abs() - tol)
    assert bool((d <= 0).all()), f"{what}: over the tolerance by {float(d.max()):.3g}"


SIZES = [(1, 1), (3, 2), (5, 7), (2, 32), (9, 33), (4, 255), (300, 257), (7, 1000), (1, 32000), (40, 8191), (2, 50301),
         (200, 4100), (1, 262147), (2, 1000003)]
KINDS = ["normal", "peaked", "masked", "lowest", "equal", "rising", "large", "empty"]


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(cuda_device, rows, vocab, kind, dtype):
    x = logits_of(rows + vocab, rows, vocab, dtype, gap=3 if kind == "normal" else 0, kind=kind)
    t = targets_of(vocab, rows, vocab, torch.int32 if vocab % 2 else torch.int64)
    r = L.token_logprobs(x, t)
    assert r.entropy is None and r.top_logprob is None and r.top_token is None
    o = R.Rows(x, t)
    near(r.logprob, *o.logprob(), "logprob")
    near(r.lse, *o.lse_and_tol(), "lse")
    k = min(vocab, (1, 5, 20, 32)[vocab % 4])
    r = L.token_logprobs(x, t, entropy=True, top=k)
    near(r.logprob, *o.logprob(), "logprob")
    near(r.entropy, *o.entropy_and_tol(), "entropy")
    place, v, tol = o.top_k(k)
    assert r.top_token.dtype == torch.int64
    assert torch.equal(r.top_token, place)
    near(r.top_logprob, v, tol, "top")


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient(cuda_device, rows, vocab, kind, dtype):
    x = logits_of(rows * vocab, rows, vocab, dtype, gap=3 if kind == "normal" else 0, kind=kind)
    t = targets_of(rows, rows, vocab)
    g = torch.Generator(device="cuda").manual_seed(rows)
    dlp = torch.randn(rows, device="cuda", generator=g)
    dent = torch.randn(rows, device="cuda", generator=g)
    r = L.token_logprobs(x, t, entropy=True)
    o = R.Rows(x, t)
    near(L.token_logprobs_backward(x, t, r.lse, dlp), *o.gradient(dlp, dtype, own_lse=r.lse), "dlogits")
    got = L.token_logprobs_backward(x, t, r.lse, dlp, entropy=r.entropy, dentropy=dent)
    near(got, *o.gradient(dlp, dtype, r.entropy, dent, own_lse=r.lse), "with entropy")
    own = x.clone()
    assert L.token_logprobs_backward(own, t, r.lse, dlp, entropy=r.entropy, dentropy=dent, out=own) is own
    if x.is_contiguous():
        assert torch.equal(own, got)


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_loss(cuda_device, rows, vocab, kind, dtype):
    x = logits_of(rows * vocab + 1, rows, vocab, dtype, gap=3 if kind == "normal" else 0, kind=kind)
    t = targets_of(rows, rows, vocab, torch.int32)
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = torch.rand(rows, device="cuda", generator=g) + 0.1
    o = R.Rows(x, t)
    lp, tol = o.logprob()
    for weight in (w, 0.25):
        each = w if weight is w else torch.full_like(w, 0.25)
        loss, dx = L.token_loss(x, t, weight)
        near(loss, -each.double() * lp, each.double() * tol + (each * lp).abs().nan_to_num(posinf=0.0) * R.E, "loss")
        near(dx, *o.gradient(-each, dtype), "dlogits")
    own = x.clone()
    loss2, dx2 = L.token_loss(own, t, 0.25, out=own)
    assert dx2 is own
    if x.is_contiguous():
        assert torch.equal(own, dx) and torch.equal(loss2, loss)


@pytest.mark.parametrize("vocab", [64, 75, 4099])
@pytest.mark.parametrize("gap", [0, 3, 8])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_anywhere(cuda_device, vocab, gap, offset, dtype):
    """Logits and outputs that are slices of wider buffers, each at its own address;
    nothing beside the output is written, and no value depends on where it lies."""
    rows = 24
    x0 = logits_of(5, rows, vocab, dtype)
    t = targets_of(6, rows, vocab)
    w = torch.rand(rows, device="cuda") + 0.1
    buf = torch.full((rows, vocab + gap + offset), INF, dtype=dtype, device="cuda")
    x = buf[:, offset:offset + vocab]
    x.copy_(x0)
    a, b = (L.token_logprobs(v.view(4, 6, vocab) if v is x0 else v, t.view(4, 6) if v is x0 else t, entropy=True, top=3)
            for v in (x0, x))
    o = R.Rows(x0, t)
    near(b.logprob, *o.logprob())
    near(b.entropy, *o.entropy_and_tol())
    assert a.top_token.shape == (4, 6, 3) and torch.equal(a.top_token.view(rows, 3), b.top_token)
    for shift in (0, 1, 5):
        into = torch.full((rows, vocab + gap + 8), 7.0, dtype=dtype, device="cuda")
        y = into[:, shift:shift + vocab]
        near(L.token_loss(x, t, w, out=y)[1], *o.gradient(-w, dtype))
        near(L.token_logprobs_backward(x, t, b.lse, w, out=y), *o.gradient(w, dtype, own_lse=b.lse))
        y.fill_(7.0)
        assert bool((into == 7).all())
    assert torch.equal(x, x0)
    L.token_loss(x, t, w, out=x)
    near(x, *o.gradient(-w, dtype))
    assert bool((buf[:, :offset] == INF).all()) and bool((buf[:, offset + vocab:] == INF).all())


@pytest.mark.parametrize("vocab", [1, 8, 257, 500, 513, 1017, 1024, 1025, 2041, 2049])
@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_rows(cuda_device, vocab, gap, dtype):
    """More rows than a grid has warps, with all kinds of them side by side."""
    kinds = [logits_of(vocab + i, 719, vocab, dtype, gap, kind) for i, kind in enumerate(KINDS)]
    rows = 719 * len(kinds)
    buffer = torch.stack([F.pad(k, (0, gap), value=7.0) for k in kinds], 1).reshape(rows, vocab + gap)
    x = buffer[:, :vocab]
    t = targets_of(vocab, rows, vocab)
    g = torch.Generator(device="cuda").manual_seed(vocab)
    w = torch.rand(rows, device="cuda", generator=g) + 0.1
    dent = torch.randn(rows, device="cuda", generator=g)
    o = R.Rows(x, t)
    r, plain = L.token_logprobs(x, t, entropy=True), L.token_logprobs(x, t)
    near(r.logprob, *o.logprob(), "logprob")
    near(r.lse, *o.lse_and_tol(), "lse")
    near(r.entropy, *o.entropy_and_tol(), "entropy")
    near(plain.logprob, *o.logprob(), "logprob alone")
    near(plain.lse, *o.lse_and_tol(), "lse alone")
    near(L.token_logprobs_backward(x, t, r.lse, w), *o.gradient(w, dtype, own_lse=r.lse), "dlogits")
    got = L.token_logprobs_backward(x, t, r.lse, w, entropy=r.entropy, dentropy=dent)
    near(got, *o.gradient(w, dtype, r.entropy, dent, own_lse=r.lse), "with entropy")
    want, tol = o.logprob()
    to = torch.full_like(buffer, 7.0)[:, :vocab]
    for out in (to, x):
        loss, dx = L.token_loss(x, t, w, out=out)
        assert dx is out
        near(loss, -want * w, tol * w + want.abs() * w * 2.0 ** -23, "loss")
        near(dx, *o.gradient(-w, dtype), "gradient")
    assert bool((buffer[:, vocab:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [40, 1000, 70000])
def test_not_finite(cuda_device, dtype, vocab):
    """NaN and +infinity make their own row's results NaN; alternatives are distinct
    columns all the same; a row without a target has no gradient whatever it holds."""
    x = logits_of(1, 8, vocab, dtype)
    x[1, 7], x[3, vocab - 1], x[5] = math.nan, INF, math.nan
    t = torch.tensor([1, 2, 3, 4, -1, -1, 0, vocab], device="cuda")
    r = L.token_logprobs(x, t, entropy=True, top=20)
    bad = torch.tensor([False, True, False, True, False, True, False, False], device="cuda")
    assert torch.equal(torch.isnan(r.lse), bad) and torch.equal(torch.isnan(r.entropy), bad)
    assert torch.equal(torch.isnan(r.logprob), (bad & (t >= 0)) | (t >= vocab))
    assert float(r.logprob[4]) == 0 and float(r.logprob[5]) == 0
    for row in r.top_token.tolist():
        assert len(set(row)) == 20 and min(row) >= 0 and max(row) < vocab
    assert r.top_token[3, 0] == vocab - 1 and 7 not in r.top_token[1].tolist()
    good = [0, 2, 4, 6, 7]
    assert torch.equal(r.top_token[good], R.Rows(x[good], t[good]).top_k(20)[0])
    loss, dx = L.token_loss(x, t, 1.0)
    nan = (bad & (t >= 0)) | (t >= vocab)
    assert torch.equal(torch.isnan(loss), nan)
    assert torch.equal(torch.isnan(dx.float()).all(1), nan) and torch.equal(torch.isnan(dx.float()).any(1), nan)
    assert not bool(dx[4:6].any()) and not bool(loss[4:6].any())
    dx = L.token_logprobs_backward(x, t, r.lse, torch.ones(8, device="cuda"))
    assert torch.equal(torch.isnan(dx.float()).any(1), nan) and not bool(dx[4:6].any())


def test_equal_logits_come_by_column(cuda_device):
    """0 and -0 are equal; so are whole rows, and all of a masked row's rest."""
    x = torch.zeros(4, 5000, device="cuda")
    x[0, ::2] = -0.0
    x[1, 4000:] = 1.0
    x[2] = -INF
    x[2, [4999, 17]] = 2.0
    x[3] = torch.finfo(F32).min
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    top = L.token_logprobs(x, t, top=32).top_token
    first = list(range(32))
    assert top.tolist() == [first, list(range(4000, 4032)), [17, 4999] + list(range(17)) + list(range(18, 31)), first]


def test_gradient_by_differences(cuda_device):
    """Of the forward call, in float32 with steps of 2^-6: a difference of two is off by
    their tolerances over the step, and by the third derivative (at most 1, times the
    step squared over 6) of a function whose values are of size 10."""
    x = logits_of(2, 1, 40, F32)
    t = torch.tensor([11], device="cuda")
    r = L.token_logprobs(x, t, entropy=True)
    dlp, dent = torch.tensor([0.7], device="cuda"), torch.tensor([-0.4], device="cuda")
    dx = L.token_logprobs_backward(x, t, r.lse, dlp, entropy=r.entropy, dentropy=dent)
    h = 2.0 ** -6
    for j in range(0, 40, 3):
        f = []
        for s in (h, -h):
            y = x.clone()
            y[0, j] += s
            q = L.token_logprobs(y, t, entropy=True)
            f.append(0.7 * float(q.logprob) - 0.4 * float(q.entropy))
        # entropy's third derivative is below 10 for logits within 20 of another
        assert abs((f[0] - f[1]) / (2 * h) - float(dx[0, j])) < 2e-5 / h + 10 * h * h / 6


def test_empty_calls(cuda_device):
    x = torch.zeros(0, 9, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    r = L.token_logprobs(x, t, entropy=True, top=4)
    assert r.logprob.shape == (0,) and r.top_token.shape == (0, 4)
    loss, dx = L.token_loss(x, t, 1.0)
    assert loss.shape == (0,) and dx.shape == (0, 9)
    one = L.token_logprobs(torch.randn(9, device="cuda"), torch.tensor(3, device="cuda"), top=2)
    assert one.logprob.shape == () and one.top_token.shape == (2,)


def test_equal_calls_give_equal_bits(cuda_device):
    for rows, vocab in ((3, 50301), (700, 1000)):
        x = logits_of(3, rows, vocab, BF)
        t = targets_of(4, rows, vocab)
        a = L.token_logprobs(x, t, entropy=True, top=9)
        loss, dx = L.token_loss(x, t, 1.0)
        for _ in range(3):
            b = L.token_logprobs(x, t, entropy=True, top=9)
            assert all(torch.equal(u, v) for u, v in zip(a, b))
            l2, d2 = L.token_loss(x, t, 1.0)
            assert torch.equal(l2, loss) and torch.equal(d2, dx)


def test_refusals(cuda_device):
    x, t = logits_of(1, 6, 50, F32), torch.zeros(6, dtype=torch.int64, device="cuda")
    f = torch.zeros(6, device="cuda")
    for bad in (lambda: L.token_logprobs(x.half(), t), lambda: L.token_logprobs(x, t.float()),
                lambda: L.token_logprobs(x, t[:5]), lambda: L.token_logprobs(x, t.cpu()),
                lambda: L.token_logprobs(x, t, top=33), lambda: L.token_logprobs(x, t, top=-1),
                lambda: L.token_logprobs(x[:, :4], t, top=5), lambda: L.token_logprobs(x.t(), t),
                lambda: L.token_logprobs(x.cpu(), t), lambda: L.token_logprobs(x.clone().requires_grad_(), t),
                lambda: L.token_logprobs_backward(x, t, f[:5], f), lambda: L.token_logprobs_backward(x, t, f, f.double()),
                lambda: L.token_logprobs_backward(x, t, f, f, dentropy=f),
                lambda: L.token_logprobs_backward(x, t, f, f, out=torch.empty_like(x).bfloat16()),
                lambda: L.token_loss(x, t, f[:5]), lambda: L.token_loss(x, t, f, out=x[:, :49])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ScapeError):
        L.token_logprobs(x[:, :0], t)
    buf = torch.zeros(6, 90, device="cuda")
    with pytest.raises(ScapeError):
        L.token_loss(buf[:, :50], t, 1.0, out=buf[:, 10:60])
