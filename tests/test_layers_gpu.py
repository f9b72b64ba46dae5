"""Training-layer operators on the GPU against plain 64-bit formulas.

Tolerances follow from the arithmetic: one rounding of the result to its type,
32-bit sums (a relative 2^-23 of the sum of magnitudes for every term, whatever
their order), the activations' documented function errors."""
import pytest
import torch

import sparse_communication_sharded_gb300 as pkg
from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = ["relu", "gelu", "silu"]


def rand(seed, *shape, dtype=BF, scale=1.0, gap=0):
    """Normal values; `gap` extra columns make it a slice of a wider buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape[:-1], shape[-1] + gap, device="cuda", generator=g) * scale
    return x.to(dtype)[..., :shape[-1]]


def off(n, dtype, by):
    """A vector of n elements that starts `by` elements into its allocation."""
    return torch.full((n + by + 8,), 7.0, dtype=dtype, device="cuda")[by:by + n]


def near(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    d = (got - want).abs() - tol
    assert bool((d <= 0).all()), f"{what}: over the tolerance by {float(d.max()):.3g}"


def vals(p):
    q = p.q.reshape(-1, p.q.shape[-1]).view(torch.uint8)
    return R.values(q, p.scale.reshape(q.shape[0], -1))


# ------------------------------------------------------------------ pack and unpack
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (7, 33), (5, 64), (128, 1280),
                                       (33, 1283), (2, 8200), (1000, 40), (65, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [0, 3, 16])
def test_pack_is_exact(cuda_device, rows, cols, dtype, gap):
    x = rand(rows * cols + gap, rows, cols, dtype=dtype, gap=gap)
    x = x * torch.exp2(torch.randint(-30, 30, (rows, 1), device="cuda").float()).to(dtype)
    x = torch.nn.functional.pad(x, (0, gap))[:, :cols] if gap else x
    p = L.pack8(x)
    v, code = R.pack8(x.double())
    assert torch.equal(p.scale, code)
    assert torch.equal(vals(p), v)
    assert torch.equal(L.unpack8(p, dtype=F32).double(), v)
    assert torch.equal(L.unpack8(p).double(), v)  # bfloat16 holds every value


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pack_edges(cuda_device, dtype):
    """Blocks of zeros, of one value at each power of two, at the limit between
    two scales, of subnormals, of the type's largest; infinities and NaN."""
    big = torch.finfo(dtype).max
    rows = [torch.zeros(40), torch.full((40,), big), torch.full((40,), -big)]
    for e in range(-149, 128, 7):
        rows.append(torch.full((40,), 2.0 ** e, dtype=torch.float64).float())
        rows.append(torch.full((40,), 1.75 * 2.0 ** e, dtype=torch.float64).float())
        rows.append(torch.cat([torch.full((39,), 0.3 * 2.0 ** e, dtype=torch.float64).float(),
                               torch.tensor([1.7578125 * 2.0 ** e], dtype=torch.float64).float()]))
    odd = torch.arange(40.0) - 20
    for bad in (float("inf"), float("-inf"), float("nan")):
        for at in (0, 5, 31, 32, 39):
            r = odd.clone()
            r[at] = bad
            rows.append(r)
    rows.append(torch.full((40,), float("nan")))
    x = torch.stack(rows).to("cuda").to(dtype)
    for t in (x, x.clone()[:, :39], torch.nn.functional.pad(x, (0, 1))[:, :40]):
        p = L.pack8(t)
        v, code = R.pack8(t.double())
        assert torch.equal(p.scale, code)
        assert torch.equal(torch.nan_to_num(vals(p), nan=1e300), torch.nan_to_num(v, nan=1e300))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (17, 1283), (64, 4096), (1, 8000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_unpack_through_activation_and_its_gradient(cuda_device, act, rows, cols, dtype):
    p = L.pack8(rand(rows, rows, cols, scale=3.0))
    z = vals(p)
    y = R.act(z, act)
    near(L.unpack8(p, dtype=dtype, activation=act), y,
         y.abs() * (R.u_of(dtype) + R.ACT_REL) + 1e-37, act)
    dy = rand(cols, rows, cols, dtype=dtype, gap=5)
    dz = dy.double() * R.slope(z, act)
    tol = dz.abs() * R.u_of(dtype) + dy.double().abs() * 3 * R.ACT_REL
    near(L.activation_grad(dy, p, act), dz, tol, act)
    own = dy.clone()
    assert L.activation_grad(own, p, act, out=own) is own
    near(own, dz, tol, act)


@pytest.mark.parametrize("act", ACTS)
def test_activation_extremes(cuda_device, act):
    """Far tails: no NaN out of 0 times an overflow."""
    z = torch.tensor([[0.0, -0.0, 1e-20, -1e-20, 88.0, -88.0, 100.0, -100.0, 1e4, -1e4, 1e19, -1e19,
                       1e30, -1e30, 3e38, -3e38]], device="cuda").t().contiguous()
    p = L.pack8(z)
    v = vals(p)
    y = L.unpack8(p, dtype=F32, activation=act)
    want = R.act(v, act)
    assert bool(torch.isfinite(y).all())
    near(y, want, want.abs() * 2.0 ** -17 + 1e-30, act)
    g = L.activation_grad(torch.ones_like(z), p, act)
    w = torch.where(v.abs() > 50, (v > 0).double(), R.slope(v.clamp(-50, 50), act))
    near(g, w, torch.full_like(w, 4 * R.ACT_REL), act)


@pytest.mark.parametrize("act", ACTS)
def test_activation_gradient_against_differences(cuda_device, act):
    z = rand(1, 64, 320, dtype=F32, scale=2.0)
    p = L.pack8(z)
    v = vals(p)
    v = torch.where(v.abs() < 1e-3, torch.full_like(v, 0.5), v) if act == "relu" else v
    d = 1e-4
    slope = (R.act(vals(p) + d, act) - R.act(vals(p) - d, act)) / (2 * d)
    got = L.activation_grad(torch.ones_like(z), p, act).double()
    keep = vals(p).abs() > 2 * d if act == "relu" else torch.ones_like(got, dtype=torch.bool)
    # the difference quotient is off by d^2/6 times a third derivative below 2
    assert bool(((got - slope).abs()[keep] <= 1e-8 + 4 * R.ACT_REL).all())


# ------------------------------------------------------------------ norm
SHAPES = [(1, 1), (1, 2048), (3, 32), (5, 257), (64, 256), (130, 1024), (129, 1025), (33, 1280),
          (777, 1283), (40, 2048), (9, 2049), (6, 5632), (4, 8192), (3, 8193), (2, 20000),
          (2500, 64)]


def norm_tols(y, h, rstd, cols, dtype):
    """rstd: a sum of squares of positive terms in 32 bits (cols roundings at
    most), the addition's rounding (2 of 2^-24 in each square), a root and a
    quotient; y adds three products."""
    r = (cols + 8) * 2.0 ** -24
    return y.abs() * (R.u_of(dtype) + r + 2.0 ** -21), rstd * r


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,gap", [(BF, F32, 0), (F32, F32, 0), (BF, BF, 3), (F32, BF, 8)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(cuda_device, rows, cols, dtype, wdtype, gap, residual):
    x = rand(1, rows, cols, dtype=dtype, gap=gap)
    res = rand(2, rows, cols, dtype=dtype, scale=2.0) if residual else None
    w = off(cols, wdtype, gap)
    w.copy_(1 + 0.1 * rand(3, cols, dtype=F32))
    o = L.add_rmsnorm(x, w, residual=res, eps=1e-5, pack=True)
    y, h, rstd = R.rms(x.double(), w.double(), 1e-5, None if res is None else res.double())
    ty, tr = norm_tols(y, h, rstd, cols, dtype)
    near(o.rstd, rstd, tr, "rstd")
    # h is rounded from the exact or once-rounded sum
    near(o.h, h, h.abs() * (R.u_of(dtype) + 2.0 ** -23) if residual else torch.zeros_like(h), "h")
    if residual:  # cancellation: the addition's rounding is relative to the sum itself
        ty = ty + y.abs() * 2.0 ** -23
    near(o.y, y, ty, "y")
    near(L.unpack8(o.y8, dtype=F32), y, R.pack_error(y) + y.abs() * ((cols + 16) * 2.0 ** -24), "y8")
    plain = L.add_rmsnorm(x, w, residual=res, eps=1e-5)
    assert plain.y8 is None and torch.equal(plain.y, o.y)


def test_norm_zero_rows_and_leading_dimensions(cuda_device):
    x = rand(5, 2, 3, 4, 96)
    x[1, 2] = 0
    w = torch.ones(96, device="cuda")
    o = L.add_rmsnorm(x, w, residual=torch.zeros_like(x), eps=1e-6, pack=True)
    assert o.y.shape == x.shape and o.rstd.shape == x.shape[:-1] and o.y8.scale.shape == (2, 3, 4, 3)
    assert torch.equal(o.y[1, 2], torch.zeros_like(o.y[1, 2]))
    near(o.rstd[1, 2], torch.full((4,), 1e3, dtype=torch.float64, device="cuda"), 1e-3)
    assert torch.equal(L.unpack8(o.y8)[1, 2], torch.zeros_like(x[1, 2]))
    # a row that is not finite stays alone
    x[0, 0, 0, 5] = float("inf")
    o2 = L.add_rmsnorm(x, w, eps=1e-6)
    assert torch.equal(o2.y[0, 1:], o.y[0, 1:]) and bool(torch.isnan(o2.y[0, 0, 0, 5]))


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,wdtype,gap", [(BF, F32, 0), (F32, F32, 0), (BF, BF, 3), (F32, BF, 8)])
@pytest.mark.parametrize("add", [False, True])
def test_norm_backward(cuda_device, rows, cols, dtype, wdtype, gap, add):
    h = rand(1, rows, cols, dtype=dtype, gap=gap)
    dy = rand(2, rows, cols, dtype=dtype, scale=1e-3, gap=gap)
    dh = rand(3, rows, cols, dtype=dtype, scale=1e-3) if add else None
    w = off(cols, wdtype, gap)
    w.copy_(1 + 0.1 * rand(4, cols, dtype=F32))
    rstd = torch.rsqrt(h.float().square().mean(-1) + 1e-5)
    dw = off(cols, F32 if wdtype == BF else dtype, gap)
    dx = L.add_rmsnorm_backward(dy, h, w, rstd, dh=dh, dweight=dw)
    args = (dy.double(), h.double(), w.double(), rstd.double())
    want, wdw = R.rms_backward(*args, None if dh is None else dh.double())
    n, d = args[1] * args[3][:, None], args[0] * args[2]
    mean = (d * n).abs().mean(1, keepdim=True) * (cols + 4) * 2.0 ** -23
    size = args[3][:, None] * (d.abs() + n.abs() * (d * n).mean(1, keepdim=True).abs())
    tol = want.abs() * R.u_of(dtype) + args[3][:, None] * n.abs() * mean + size * 2.0 ** -21
    if add:
        tol = tol + dh.double().abs() * 2.0 ** -22
    near(dx, want, tol, "dx")
    near(dw, wdw, wdw.abs() * R.u_of(dw.dtype) + (args[0] * n).abs().sum(0) * (rows + 4) * 2.0 ** -23, "dw")
    own = dy.clone()
    L.add_rmsnorm_backward(own, h, w, rstd, dh=dh, out=own)
    assert torch.equal(own, dx)


def test_norm_gradient_against_differences(cuda_device):
    """The gradient of sum(c * y(x)) along random directions, by central
    differences of the 64-bit forward formula."""
    rows, cols = 6, 320
    x, c = rand(1, rows, cols, dtype=F32), rand(2, rows, cols, dtype=F32)
    w = 1 + 0.1 * rand(3, cols, dtype=F32)
    o = L.add_rmsnorm(x, w, eps=1e-5)
    dw = torch.empty_like(w)
    dx = L.add_rmsnorm_backward(c, o.h, w, o.rstd, dweight=dw)
    f = lambda a, b: float((c.double() * R.rms(a, b, 1e-5)[0]).sum())  # noqa: E731
    for s in range(4):
        vx, vw = rand(10 + s, rows, cols, dtype=F32).double(), rand(20 + s, cols, dtype=F32).double()
        t = 1e-5
        num = (f(x.double() + t * vx, w.double()) - f(x.double() - t * vx, w.double())) / (2 * t)
        assert abs(num - float((dx.double() * vx).sum())) < 1e-4 * float((dx.double() * vx).norm())
        num = (f(x.double(), w.double() + t * vw) - f(x.double(), w.double() - t * vw)) / (2 * t)
        assert abs(num - float((dw.double() * vw).sum())) < 1e-4 * float((dw.double() * vw).norm())


# ------------------------------------------------------------------ linear
def product_error(a, b, k):
    """32-bit sums of k exact products."""
    return (a.double().abs() @ b.double().abs()) * (k + 2) * 2.0 ** -23


LINEAR = [(1, 1, 1), (1, 64, 64), (1, 1024, 4096), (2, 72, 136), (7, 33, 65), (16, 256, 264),
          (127, 129, 31), (128, 64, 256), (129, 1000, 257), (333, 1283, 719), (64, 6144, 128),
          (1000, 512, 1280), (2500, 192, 2304), (4099, 320, 1288)]


@pytest.mark.parametrize("rows,k,n", LINEAR)
@pytest.mark.parametrize("act,bias,residual,keep,gap", [
    (None, False, False, False, 0), ("gelu", True, False, True, 0), ("silu", True, True, False, 3),
    ("relu", False, True, True, 8), (None, True, False, True, 1)])
def test_linear_forward(cuda_device, rows, k, n, act, bias, residual, keep, gap):
    x = rand(1, rows, k, gap=gap)
    w = rand(2, n, k, scale=k ** -0.5, gap=gap)
    b = None
    if bias:
        b = off(n, BF, gap)
        b.copy_(rand(3, n))
    res = rand(4, rows, n, gap=gap) if residual else None
    got = L.linear(x, w, bias=b, residual=res, activation=act, keep_pre=keep)
    y, z8 = got if keep else (got, None)
    z = x.double() @ w.double().t()
    ez = product_error(x, w.t(), k)
    if bias:
        z = z + b.double()
        ez = ez + z.abs() * 2.0 ** -24
    a = R.act(z, act)
    want = a + res.double() if residual else a
    # slopes are at most 1.2
    tol = want.abs() * R.U_BF16 + 1.2 * ez + a.abs() * R.ACT_REL
    near(y, want, tol + (res.double().abs() * 2.0 ** -23 if residual else 0), "y")
    if keep:
        near(L.unpack8(z8, dtype=F32), z, R.pack_error(z) + 1.1 * ez + R.blocks(ez).amax(-1)
             .repeat_interleave(32, dim=1)[:, :n] * 2.0 ** -17, "z8")
    assert L.status() == 0


@pytest.mark.parametrize("rows,k,n", LINEAR)
@pytest.mark.parametrize("act,gap", [(None, 0), ("gelu", 0), ("silu", 3), ("relu", 8)])
def test_linear_backward_input(cuda_device, rows, k, n, act, gap):
    dy = rand(1, rows, n, gap=gap)
    w = rand(2, n, k, scale=n ** -0.5, gap=gap)
    p = L.pack8(rand(3, rows, k, scale=2.0)) if act else None
    dx = L.linear_backward_input(dy, w, pre=p, activation=act)
    want, e = dy.double() @ w.double(), product_error(dy, w, n)
    if act:
        s = R.slope(vals(p), act)
        e = e * 1.2 + want.abs() * 3 * R.ACT_REL
        want = want * s
    near(dx, want, want.abs() * R.U_BF16 + e, "dx")
    assert L.status() == 0


@pytest.mark.parametrize("rows,k,n", LINEAR + [(16384, 64, 64), (5000, 40, 200)])
@pytest.mark.parametrize("act,packed,gd,gap", [
    (None, False, BF, 0), (None, True, F32, 0), ("gelu", True, BF, 3), ("silu", True, BF, 8),
    ("relu", True, F32, 1)])
def test_linear_backward_weight(cuda_device, rows, k, n, act, packed, gd, gap):
    """Into a flat gradient, `gap` elements from an aligned address."""
    dy = rand(1, rows, n, gap=gap)
    x = rand(2, rows, k, scale=2.0, gap=gap)
    a = x.double()
    if packed:
        x = L.pack8(x)
        a = R.act(vals(x), act)
    flat = torch.full((gap + n * k + n + 4,), 9.0, dtype=gd, device="cuda")
    dw, db = flat[gap:gap + n * k].view(n, k), flat[gap + n * k:gap + n * k + n]
    assert L.linear_backward_weight(dy, x, activation=act, dweight=dw, dbias=db) is dw
    d = dy.double()
    want = d.t() @ a
    mag = d.abs().t() @ a.abs()
    # an activation's value is rounded to bfloat16 first
    e = mag * ((rows + 2) * 2.0 ** -23 + (R.U_BF16 + R.ACT_REL if act in ("gelu", "silu") else 0))
    near(dw, want, want.abs() * R.u_of(gd) + e, "dw")
    s = d.sum(0)
    near(db, s, s.abs() * R.u_of(gd) + d.abs().sum(0) * (rows + 2) * 2.0 ** -23, "db")
    assert bool((flat[:gap] == 9).all()) and bool((flat[gap + n * k + n:] == 9).all())
    assert L.status() == 0


def test_linear_large_tiles_every_layout(cuda_device):
    """Sizes that fill the GPU with the widest tiles, ragged in each direction."""
    rows, k, n = 5003, 1288, 3592
    x, w, dy = rand(1, rows, k), rand(2, n, k, scale=0.03), rand(3, rows, n, scale=1e-3)
    z, e = x.double() @ w.double().t(), product_error(x, w.t(), k)
    near(L.linear(x, w), z, z.abs() * R.U_BF16 + e, "y")
    want = dy.double() @ w.double()
    near(L.linear_backward_input(dy, w), want, want.abs() * R.U_BF16 + product_error(dy, w, n), "dx")
    want = dy.double().t() @ x.double()
    near(L.linear_backward_weight(dy, x), want,
         want.abs() * R.U_BF16 + product_error(dy.t(), x, rows), "dw")
    assert L.status() == 0


@pytest.mark.parametrize("m,n,k", [(4100, 1276, 3592), (4096, 1280, 3584)])
def test_linear_tiles_left_over(cuda_device, m, n, k):
    """A few more tiles than the GPU takes at one time and a long contraction: the
    last ones go out in a launch of their own.  m x n outputs, contraction k."""
    act, pre = "silu", L.pack8(rand(9, m, n, scale=2.0))
    x, w, b, res = rand(1, m, k), rand(2, n, k, scale=0.03), rand(3, n), rand(4, m, n)
    z, e = x.double() @ w.double().t() + b.double(), product_error(x, w.t(), k)
    a = R.act(z, act)
    y, z8 = L.linear(x, w, bias=b, residual=res, activation=act, keep_pre=True)
    want = a + res.double()
    near(y, want, want.abs() * R.U_BF16 + 1.2 * e + z.abs() * 2.0 ** -23 + a.abs() * R.ACT_REL
         + res.double().abs() * 2.0 ** -23, "y")
    near(L.unpack8(z8, dtype=F32), z, R.pack_error(z) + 1.1 * e + z.abs() * 2.0 ** -23
         + R.blocks(e).amax(-1).repeat_interleave(32, dim=1)[:, :n] * 2.0 ** -17, "z8")
    w2 = rand(5, k, n, scale=0.03)
    want, e, s = x.double() @ w2.double(), product_error(x, w2, k), R.slope(vals(pre), act)
    near(L.linear_backward_input(x, w2, pre=pre, activation=act), want * s,
         (want * s).abs() * R.U_BF16 + e * 1.2 + want.abs() * 3 * R.ACT_REL, "dx")
    dy, x2 = rand(6, k, m, scale=0.01), rand(7, k, n)
    want, e = dy.double().t() @ x2.double(), product_error(dy.t(), x2, k)
    near(L.linear_backward_weight(dy, x2), want, want.abs() * R.U_BF16 + e, "dw")
    near(L.linear_backward_weight(dy, x2, grad_dtype=F32), want, want.abs() * R.U_F32 + e, "dw32")
    assert L.status() == 0


@pytest.mark.parametrize("m,n,k,act", [
    (4090, 1272, 72, None), (4090, 1272, 72, "gelu"), (4864, 1100, 40, "relu"), (4700, 1149, 300, "silu"),
    (20224, 256, 1800, "gelu")])
def test_linear_other_tilings(cuda_device, m, n, k, act):
    """Products whose tiles go out in one round of wider ones, and (the last case)
    with tiles left over where wider ones do not help."""
    xf, wf, b = rand(1, m, k), rand(2, n, k, scale=0.03), rand(3, n)
    z, e = xf.double() @ wf.double().t() + b.double(), product_error(xf, wf.t(), k)
    if act:
        y, z8 = L.linear(xf, wf, bias=b, activation=act, keep_pre=True)
        near(L.unpack8(z8, dtype=F32), z, R.pack_error(z) + 1.1 * e + z.abs() * 2.0 ** -23
             + R.blocks(e).amax(-1).repeat_interleave(32, dim=1)[:, :n] * 2.0 ** -17, "z8")
    else:
        y = L.linear(xf, wf, bias=b)
    want = R.act(z, act) if act else z
    near(y, want, want.abs() * R.U_BF16 + 1.2 * e + z.abs() * 2.0 ** -23 + want.abs() * R.ACT_REL, "y")
    pre = L.pack8(rand(9, m, n, scale=2.0)) if act else None
    x, w2 = rand(1, m, k), rand(5, k, n, scale=0.03)
    want, e = x.double() @ w2.double(), product_error(x, w2, k)
    if act:
        e = e * 1.2 + want.abs() * 3 * R.ACT_REL
        want = want * R.slope(vals(pre), act)
    near(L.linear_backward_input(x, w2, pre=pre, activation=act), want, want.abs() * R.U_BF16 + e, "dx")
    dy, x2 = rand(6, k, m, scale=0.01), rand(7, k, n)
    want, e = dy.double().t() @ x2.double(), product_error(dy.t(), x2, k)
    near(L.linear_backward_weight(dy, x2), want, want.abs() * R.U_BF16 + e, "dw")
    near(L.linear_backward_weight(dy, x2, grad_dtype=F32), want, want.abs() * R.U_F32 + e, "dw32")
    assert L.status() == 0


def test_linear_gradients_against_differences(cuda_device):
    """d/dt of sum(c * act-linear(x)) with the input made by gelu from z: the
    64-bit formula's central differences along random directions of z and w."""
    rows, k, n = 40, 96, 72
    z8 = L.pack8(rand(1, rows, k))
    z, w, c = vals(z8), rand(2, n, k, scale=0.1), rand(3, rows, n)
    dz = L.linear_backward_input(c, w, pre=z8, activation="gelu").double()
    dw = L.linear_backward_weight(c, z8, activation="gelu", grad_dtype=F32).double()
    f = lambda a, b: float((c.double() * (R.act(a, "gelu") @ b.t())).sum())  # noqa: E731
    for s in range(4):
        v, u, t = rand(10 + s, rows, k).double(), rand(20 + s, n, k).double(), 1e-5
        num = (f(z + t * v, w.double()) - f(z - t * v, w.double())) / (2 * t)
        assert abs(num - float((dz * v).sum())) <= float((dz * v).abs().sum()) * R.U_BF16 + 1e-4
        num = (f(z, w.double() + t * u) - f(z, w.double() - t * u)) / (2 * t)
        assert abs(num - float((dw * u).sum())) <= 2 * float((dw * u).abs().sum()) * R.U_BF16 + 1e-4


def test_linear_leading_dimensions_and_in_place_residual(cuda_device):
    x, w = rand(1, 2, 5, 64), rand(2, 48, 64, scale=0.1)
    res = rand(3, 2, 5, 48)
    want = L.linear(x, w, residual=res)
    assert want.shape == (2, 5, 48)
    got = L.linear(x, w, residual=res, out=res)
    assert got is res and torch.equal(got, want)


def test_empty_batches(cuda_device):
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    w = rand(1, 24, 16)
    assert L.linear(e(0, 16), w).shape == (0, 24)
    assert L.linear_backward_input(e(0, 24), w).shape == (0, 16)
    db = torch.full((24,), 3.0, dtype=BF, device="cuda")
    dw = L.linear_backward_weight(e(0, 24), e(0, 16), dbias=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    p = L.pack8(e(0, 40))
    assert p.q.shape == (0, 40) and p.scale.shape == (0, 2) and L.unpack8(p).shape == (0, 40)
    wn, g = torch.ones(40, device="cuda"), torch.full((40,), 2.0, device="cuda")
    o = L.add_rmsnorm(e(0, 40), wn, pack=True)
    assert o.y.shape == (0, 40)
    L.add_rmsnorm_backward(e(0, 40), e(0, 40), wn, o.rstd, dweight=g)
    assert bool((g == 0).all())


def test_non_finite_values_stay_in_their_rows(cuda_device):
    x, w = rand(1, 200, 320), rand(2, 136, 320, scale=0.05)
    want = L.linear(x, w, activation="silu")
    x[3, 7], x[150, 0] = float("inf"), float("nan")
    got, z8 = L.linear(x, w, activation="silu", keep_pre=True)
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[3] = keep[150] = False
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[150]).all()) and bool(torch.isnan(L.unpack8(z8)[150]).all())
    assert not bool(torch.isfinite(got[3].float()).all())


def test_repeatable_and_on_another_stream(cuda_device):
    """Equal bits call after call, on a stream of the caller's, and replayed from
    a captured graph."""
    x, w, dy = rand(1, 300, 1283), rand(2, 257, 1283, scale=0.03), rand(3, 300, 257)
    wn = torch.ones(1283, device="cuda")

    def all_of():
        o = L.add_rmsnorm(x, wn, pack=True)
        y, z8 = L.linear(o.y, w, activation="gelu", keep_pre=True)
        db = torch.empty(257, dtype=BF, device="cuda")
        dz = L.activation_grad(dy, z8, "gelu")
        dw = L.linear_backward_weight(dz, o.y8, dbias=db)
        dx = L.linear_backward_input(dz, w)
        g = torch.empty(1283, device="cuda")
        return y, dw, db, dx, L.add_rmsnorm_backward(dx, o.h, wn, o.rstd, dweight=g), g

    first = all_of()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            again = all_of()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


@pytest.mark.parametrize("call", [
    lambda x, w: L.pack8(x.half()), lambda x, w: L.pack8(x.t()), lambda x, w: L.pack8(x.cpu()),
    lambda x, w: L.unpack8(L.pack8(x), dtype=torch.float16),
    lambda x, w: L.unpack8(L.pack8(x), activation="tanh"),
    lambda x, w: L.unpack8(L.Packed8(L.pack8(x).q, L.pack8(x).scale[:, :1])),
    lambda x, w: L.activation_grad(x[:4], L.pack8(x), "gelu"),
    lambda x, w: L.add_rmsnorm(x, torch.ones(63, device="cuda")),
    lambda x, w: L.add_rmsnorm(x, torch.ones(64, device="cuda"), residual=x.float()),
    lambda x, w: L.linear(x, w[:, :32]), lambda x, w: L.linear(x, w.float()),
    lambda x, w: L.linear(x, w, bias=torch.zeros(3, device="cuda", dtype=BF)),
    lambda x, w: L.linear(x, w, activation="gelu_erf"),
    lambda x, w: L.linear(x, w, out=x),
    lambda x, w: L.linear_backward_input(x, w),
    lambda x, w: L.linear_backward_input(x[:, :48], w, activation="gelu"),
    lambda x, w: L.linear_backward_weight(x[:, :48], x, activation="gelu"),
    lambda x, w: L.linear_backward_weight(x[:, :48], x, dweight=w.half()),
    lambda x, w: L.linear(x.unsqueeze(0).expand(3, 8, 64).transpose(0, 1), w),
])
def test_refusals(cuda_device, call):
    with pytest.raises((ValueError, pkg.ScapeError)):
        call(rand(1, 8, 64), rand(2, 48, 64))
