"""Embedding lookup and its gradient against plain 64-bit formulas."""
import math

import pytest
import torch

from sparse_communication_sharded_gb300 import ScapeError
from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, dtype=BF, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape[:-1], shape[-1] + gap, device="cuda", generator=g).to(dtype)[..., :shape[-1]]


def tokens_of(seed, n, vocab, kind, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    if kind == "one":
        t[:] = vocab // 2
    elif kind == "few":
        t = t % min(3, vocab)
    elif kind == "padded":
        t[torch.rand(n, device="cuda", generator=g) < 0.4] = vocab - 1
        t[torch.rand(n, device="cuda", generator=g) < 0.2] = -100
    elif kind == "none":
        t[:] = -1
    elif kind == "sorted":
        t = t.sort().values
    elif kind == "outside":
        t[::3] = vocab
        t[1::5] = torch.iinfo(dtype).max
        t[2::7] = torch.iinfo(dtype).min
    return t.to(dtype)


def near(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    d = torch.nan_to_num((got - want).abs() - tol, nan=0.0)
    assert bool((d <= 0).all()), f"{what}: over the tolerance by {float(d.max()):.3g}"


@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (1, 32000, 2048), (5, 7, 33), (77, 300, 8), (1000, 50, 1283),
                                          (513, 1000, 64), (33, 9, 8200)])
@pytest.mark.parametrize("table", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("index", [torch.int64, torch.int32])
def test_lookup(cuda_device, n, vocab, cols, table, out, index):
    w = rand(n, vocab, cols, dtype=table)
    for kind in ("random", "padded", "outside"):
        t = tokens_of(n, n, vocab, kind, index)
        for scale in (1.0, math.sqrt(cols)):
            want, tol = R.embedding(t, w, float(torch.tensor(scale, dtype=F32)), out)
            near(L.embedding(t, w, scale=scale, dtype=out), want, tol, f"{kind} {scale}")


@pytest.mark.parametrize("cols", [64, 75])
@pytest.mark.parametrize("gap", [0, 3, 8, 16])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("table,out", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_lookup_anywhere(cuda_device, cols, gap, offset, table, out):
    """Tables that are slices of a wider buffer, outputs too, at any address; nothing
    beside the output is written."""
    w = rand(1, 40, cols + offset, dtype=table, gap=gap)[:, offset:]
    t = tokens_of(2, 91, 40, "padded").view(7, 13)
    buf = torch.full((7, 13, cols + gap + offset), 7.0, dtype=out, device="cuda")
    y = buf[..., offset:offset + cols]
    assert L.embedding(t, w, scale=0.5, out=y) is y
    want, tol = R.embedding(t, w, 0.5, out)
    near(y, want, tol)
    assert bool((buf[..., :offset] == 7).all()) and bool((buf[..., offset + cols:] == 7).all())


def test_lookup_shapes(cuda_device):
    w = rand(1, 10, 16)
    assert L.embedding(torch.tensor(3, device="cuda"), w).shape == (16,)
    assert torch.equal(L.embedding(torch.tensor(3, device="cuda"), w), w[3])
    assert L.embedding(torch.zeros(0, 4, dtype=torch.int64, device="cuda"), w).shape == (0, 4, 16)
    assert L.embedding(torch.zeros(2, 3, dtype=torch.int32, device="cuda"), w).dtype == BF
    assert L.embedding(torch.zeros(4, dtype=torch.int32, device="cuda"), rand(2, 3, 8)[:, :0]).shape == (4, 0)


@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (1, 1000, 64), (15, 3, 8), (16, 40, 33), (17, 400, 1280),
                                          (1000, 353, 72), (1025, 5000, 131), (4100, 64, 2056), (3000, 2000, 1283)])
@pytest.mark.parametrize("kind", ["random", "one", "few", "padded", "none", "sorted", "outside"])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_gradient(cuda_device, n, vocab, cols, kind, dtype, grad):
    dy = rand(n + cols, n, cols, dtype=dtype)
    t = tokens_of(n, n, vocab, kind, torch.int32 if cols % 2 else torch.int64)
    dw = torch.full((vocab, cols), math.nan, dtype=grad, device="cuda")
    assert L.embedding_backward(dy, t, dw, scale=1.5) is dw
    want, tol = R.embedding_backward(dy, t, torch.zeros_like(dw), 1.5, grad)
    near(dw, want, tol, kind)
    seen = torch.zeros(vocab + 1, dtype=torch.bool, device="cuda")
    seen[torch.where((t < 0) | (t >= vocab), vocab, t).long()] = True
    assert not bool(dw[~seen[:vocab]].any())
    again = torch.empty_like(dw)
    L.embedding_backward(dy, t, again, scale=1.5)
    assert torch.equal(again, dw)
    old = rand(5, vocab, cols, dtype=grad)
    more = old.clone()
    L.embedding_backward(dy, t, more, scale=-0.5, accumulate=True)
    want, tol = R.embedding_backward(dy, t, old, -0.5, grad)
    near(more, want, tol, f"{kind} added")
    assert torch.equal(more[~seen[:vocab]], old[~seen[:vocab]])


@pytest.mark.parametrize("cols", [64, 75, 1288])
@pytest.mark.parametrize("gap", [0, 3, 8])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("dtype,grad", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_gradient_anywhere(cuda_device, cols, gap, offset, dtype, grad):
    vocab, n = 45, 200
    dy = rand(3, n, cols + offset, dtype=dtype, gap=gap)[:, offset:]
    t = tokens_of(4, n, vocab, "padded")
    flat = torch.full((offset + vocab * (cols + gap) + 9,), 7.0, dtype=grad, device="cuda")
    dw = flat[offset:offset + vocab * (cols + gap)].view(vocab, cols + gap)[:, :cols]
    L.embedding_backward(dy, t, dw)
    want, tol = R.embedding_backward(dy, t, torch.zeros_like(dw), 1.0, grad)
    near(dw, want, tol)
    dw.fill_(7.0)
    assert bool((flat == 7).all())


@pytest.mark.parametrize("lengths", [(65, 64, 66, 80, 81, 96, 1), (512, 513, 528, 529, 577, 576, 16),
                                     (4097, 4095, 33, 4161, 4672), (32769, 17, 33344, 32704), (300001, 64, 65)])
@pytest.mark.parametrize("cols", [8, 13, 2056])
@pytest.mark.parametrize("before", [0, 7])
def test_gradient_of_common_tokens(cuda_device, lengths, cols, before):
    """Tokens with many positions side by side: whole values below 2^24 in all, so the sums
    are exact in any order and each position counts once."""
    lengths = ((before,) if before else ()) + lengths
    if cols > 100:
        lengths = tuple(n % 40000 for n in lengths)
    t = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).cuda()
    g = torch.Generator(device="cuda").manual_seed(cols)
    order = torch.randperm(t.numel(), device="cuda", generator=g)
    dy = torch.randint(-8, 9, (t.numel(), cols), device="cuda", generator=g)
    dy[:, 0] = 1  # counts
    want = torch.zeros(len(lengths), cols, dtype=torch.float64, device="cuda").index_add_(0, t, dy.double())
    for at in (torch.arange(t.numel(), device="cuda"), order):
        dw = L.embedding_backward(dy[at].bfloat16(), t[at], torch.empty(len(lengths), cols, device="cuda"))
        assert torch.equal(dw.double(), want)


def test_gradient_is_the_lookups(cuda_device):
    """By differences: the lookup is linear, so (y(w + h) - y(w - h)) . dy = 2 h . dw."""
    w, h = rand(1, 30, 24, dtype=F32), rand(2, 30, 24, dtype=F32)
    t = tokens_of(3, 100, 30, "padded")
    dy = rand(4, 100, 24, dtype=F32)
    dw = L.embedding_backward(dy, t, torch.empty_like(w), scale=3.0)
    up, down = L.embedding(t, w + h, scale=3.0), L.embedding(t, w - h, scale=3.0)
    left = ((up.double() - down.double()) * dy.double()).sum()
    right = 2 * (h.double() * dw.double()).sum()
    # each of 2400 products is off by two roundings of values of size 6, dw's by 100
    assert abs(float(left - right)) <= 1e-4 * float(dy.abs().sum())


def test_no_tokens_and_no_columns(cuda_device):
    dw = torch.full((5, 8), 7.0, device="cuda")
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    L.embedding_backward(torch.zeros(0, 8, device="cuda"), t, dw, accumulate=True)
    assert bool((dw == 7).all())
    L.embedding_backward(torch.zeros(0, 8, device="cuda"), t, dw)
    assert not bool(dw.any())
    L.embedding_backward(torch.zeros(3, 0, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"), dw[:, :0])


def test_infinities_stay_in_their_rows(cuda_device):
    t = torch.tensor([1, 2, 1, 3, 1], device="cuda")
    dy = torch.ones(5, 40, device="cuda")
    dy[0, 3], dy[2, 3], dy[3, 7], dy[1, 39] = math.inf, -math.inf, math.nan, math.inf
    dw = L.embedding_backward(dy, t, torch.empty(5, 40, device="cuda"))
    want = torch.zeros(5, 40, device="cuda").index_add_(0, t, dy)
    assert torch.equal(torch.nan_to_num(dw, nan=9e9), torch.nan_to_num(want, nan=9e9))


def test_refusals(cuda_device):
    w, t, dy = rand(1, 9, 16), torch.zeros(4, dtype=torch.int64, device="cuda"), rand(2, 4, 16)
    dw = torch.empty(9, 16, device="cuda")
    for bad in (lambda: L.embedding(t.float(), w), lambda: L.embedding(t.cpu(), w), lambda: L.embedding(t, w.half()),
                lambda: L.embedding(t, w[0]), lambda: L.embedding(t, w[:0]), lambda: L.embedding(t, w, dtype=torch.half),
                lambda: L.embedding(t, w, out=torch.empty(4, 15, device="cuda")),
                lambda: L.embedding(torch.zeros(8, dtype=torch.int64, device="cuda")[::2], w),
                lambda: L.embedding(t, w, scale="x"), lambda: L.embedding(t, w.t()),
                lambda: L.embedding_backward(dy, t[:3], dw), lambda: L.embedding_backward(dy, t, dw[:, :8]),
                lambda: L.embedding_backward(dy, t, dw[0]), lambda: L.embedding_backward(dy, t, dw.half()),
                lambda: L.embedding_backward(dy.t(), t, dw), lambda: L.embedding_backward(dy, t, dw.cpu()),
                lambda: L.embedding(t, w.clone().requires_grad_())):
        with pytest.raises(ValueError):
            bad()
    buf = rand(3, 20, 16)
    with pytest.raises(ScapeError):
        L.embedding(t, buf[:9], out=buf[8:12])
    with pytest.raises(ScapeError):
        L.embedding_backward(buf[:4], t, buf[3:12])
