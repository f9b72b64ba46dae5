"""What a program meets besides sizes: values that are not finite in large
products, several threads and streams at once, and more elements than 32 bits
count."""
import threading

import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R
from tests.test_layers_plan_gpu import FORWARD, INPUT_GRAD, PAIRS, REST, WEIGHT_GRAD, plan, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def test_values_that_are_not_finite_in_large_products(cuda_device):
    """They reach what the formula says and nothing else: the same bits elsewhere."""
    rows, k, n = 8200, 1256, 1272
    assert all(plan(p, rows, k, n)[0] in (PAIRS, REST) for p in (FORWARD, INPUT_GRAD))
    x, w, dy = rand(1, rows, k), rand(2, n, k, scale=0.05), rand(3, rows, n)
    y, z8 = L.linear(x, w, activation="silu", keep_pre=True)
    bad = x.clone()
    bad[300, 5], bad[2000, 0], bad[8199, k - 1] = INF, NAN, -INF
    hit = torch.zeros(rows, dtype=torch.bool, device="cuda")
    hit[[300, 2000, 8199]] = True
    y2, z82 = L.linear(bad, w, activation="silu", keep_pre=True)
    assert torch.equal(y2[~hit], y[~hit])
    assert torch.equal(z82.q.view(torch.uint8)[~hit], z8.q.view(torch.uint8)[~hit])
    assert torch.equal(z82.scale[~hit], z8.scale[~hit])
    want = R.act(bad[hit].double() @ w.double().t(), "silu")
    assert torch.equal(torch.isnan(y2[hit]), torch.isnan(want))
    assert torch.equal(torch.isinf(y2[hit]), torch.isinf(want))
    v = L.unpack8(z82)
    assert bool(torch.isnan(v[hit]).all())  # infinities become NaN in 8 bits

    bad = dy.clone()
    bad[300, 5], bad[2000, 0], bad[8199, n - 1] = INF, NAN, -INF
    dx, dx2 = L.linear_backward_input(dy, w), L.linear_backward_input(bad, w)
    assert torch.equal(dx2[~hit], dx[~hit]) and not bool(torch.isfinite(dx2[hit]).any())
    m, c = 2500, 1800  # a weight gradient by pairs
    assert plan(WEIGHT_GRAD, 72, c, m)[0] == PAIRS
    dy, a = rand(4, 72, m), rand(5, 72, c)
    bad = dy.clone()
    bad[3, 700], bad[70, m - 1] = INF, NAN
    db = torch.empty(m, dtype=F32, device="cuda")
    for x in (a, L.pack8(a)):
        g, g2 = L.linear_backward_weight(dy, x), L.linear_backward_weight(bad, x, grad_dtype=BF)
        hit = torch.zeros(m, dtype=torch.bool, device="cuda")
        hit[[700, m - 1]] = True
        assert torch.equal(g2[~hit], g[~hit]) and not bool(torch.isfinite(g2[hit]).any())
        L.linear_backward_weight(bad, x, grad_dtype=F32, dbias=db)
        assert torch.equal(~torch.isfinite(db), hit)
    assert L.status() == 0


def test_nan_checkpoint_values(cuda_device):
    """A NaN in a checkpoint is a NaN through every activation and its slope."""
    x = rand(1, 40, 96)
    x[7, 3], x[8, 95] = NAN, INF
    p = L.pack8(x)
    hit = torch.zeros(40, 96, dtype=torch.bool, device="cuda")
    hit[7, 3] = hit[8, 95] = True
    dy, w = rand(2, 40, 96), rand(3, 96, 96)
    for act in ("relu", "gelu", "silu"):
        for dtype in (BF, F32):
            assert torch.equal(torch.isnan(L.unpack8(p, dtype=dtype, activation=act)), hit)
            assert torch.equal(torch.isnan(L.activation_grad(dy.to(dtype), p, act)), hit)
        assert torch.equal(torch.isnan(L.linear_backward_input(dy, w, pre=p, activation=act)), hit)
        assert torch.equal(torch.isnan(L.linear_backward_input(dy[7:9], w, pre=L.Packed8(p.q[7:9], p.scale[7:9]),
                                                               activation=act)), hit[7:9])


def work(seed):
    """A step of every operator: forward, backward, odd sizes."""
    rows, k, n = 300 + seed, 263, 520
    x, w, dy = rand(seed, rows, k), rand(seed + 1, n, k, scale=0.05), rand(seed + 2, rows, n)
    wn, g = torch.ones(k, device="cuda"), torch.empty(k, device="cuda")
    o = L.add_rmsnorm(x.float(), wn, pack=True)
    y, z8 = L.linear(x, w, activation="gelu", keep_pre=True)
    db = torch.empty(n, dtype=BF, device="cuda")
    dz = L.activation_grad(dy, z8, "gelu")
    dw = L.linear_backward_weight(dz, L.pack8(x), dbias=db)
    dx = L.linear_backward_input(dz, w)
    dn = L.add_rmsnorm_backward(dx.float(), o.h, wn, o.rstd, dweight=g)
    return [o.y, o.rstd, y, dz, dw, db, dx, dn, g, L.unpack8(o.y8)]


def test_threads_and_streams_at_once(cuda_device):
    """Four threads, each on a stream of its own with its own data, give the bits
    that one gives alone."""
    want = [work(10 * i) for i in range(4)]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = work(10 * i)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert L.status() == 0


def test_more_than_32_bits_of_elements(cuda_device):
    """Every operator at rows whose elements are past the 2^31st (and 2^32nd) of their
    matrices, against the same rows on their own."""
    rows, cols = 1_060_000, 4104  # 4.35e9 elements, 8.7 GB in bfloat16
    assert rows * cols > 2 ** 32
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    part = rand(1, 4000, cols)
    for r in range(0, rows, 4000):
        x[r:r + 4000] = part
    at = torch.tensor([0, 523_264, 523_265, 1_046_529, 1_046_530, rows - 3], device="cuda")
    x[at] = rand(2, len(at), cols)
    few = x[at]
    p, q = L.pack8(x), L.pack8(few)
    assert torch.equal(p.q[at].view(torch.uint8), q.q.view(torch.uint8)) and torch.equal(p.scale[at], q.scale)
    y = L.unpack8(p, activation="silu")
    assert torch.equal(y[at], L.unpack8(q, activation="silu"))
    L.activation_grad(x, p, "gelu", out=y)
    assert torch.equal(y[at], L.activation_grad(few, q, "gelu"))
    w = torch.ones(cols, device="cuda")
    rstd = L.add_rmsnorm(few, w).rstd
    all_rstd = torch.ones(rows, device="cuda")
    all_rstd[at] = rstd
    L.add_rmsnorm_backward(x, x, w, all_rstd, out=y)
    assert torch.equal(y[at], L.add_rmsnorm_backward(few, few, w, rstd))
    del y
    o, f = L.add_rmsnorm(x, w, pack=True), L.add_rmsnorm(few, w, pack=True)
    assert torch.equal(o.y[at], f.y) and torch.equal(o.rstd[at], f.rstd)
    assert torch.equal(o.y8.q[at].view(torch.uint8), f.y8.q.view(torch.uint8))
    del o
    # products: the same rows in a smaller batch that takes the same tiles' arithmetic
    m = rand(3, 64, cols, scale=0.02)
    big = L.linear(x, m)
    want = few.double() @ m.double().t()
    tol = want.abs() * R.U_BF16 + (few.double().abs() @ m.double().abs().t()) * cols * 2.0 ** -23
    assert bool(((big[at].double() - want).abs() <= tol).all())
    dy = torch.zeros(rows, 64, dtype=BF, device="cuda")
    dy[at] = rand(4, len(at), 64)
    want = dy[at].double().t() @ L.unpack8(q, dtype=F32).double()
    g = L.linear_backward_weight(dy, p, grad_dtype=F32)
    tol = want.abs() * 2.0 ** -23 + (dy[at].double().abs().t() @ L.unpack8(q, dtype=F32).double().abs()) * 8 * 2.0 ** -23
    assert bool(((g.double() - want).abs() <= tol).all())
    dx = L.linear_backward_input(dy, m, pre=p, activation="relu")
    want = (dy[at].double() @ m.double()) * R.slope(L.unpack8(q, dtype=F32).double(), "relu")
    tol = want.abs() * R.U_BF16 + (dy[at].double().abs() @ m.double().abs()) * 66 * 2.0 ** -23
    assert bool(((dx[at].double() - want).abs() <= tol).all())
    assert L.status() == 0
