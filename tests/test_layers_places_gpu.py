"""Where outputs may lie: slices with a row stride, beside their inputs in one
buffer, and in the place of an input; every result equal to that of a call with
outputs of its own, nothing written beside it."""
import pytest
import torch

from sparse_communication_sharded_gb300 import ScapeError
from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def slices(rows, widths, dtype, gap):
    """Neighbouring column ranges of one buffer of sevens, `gap` columns apart."""
    buf = torch.full((rows, sum(widths) + gap * len(widths)), 7.0, dtype=dtype, device="cuda")
    views, at = [], 0
    for w in widths:
        views.append(buf[:, at:at + w])
        at += w + gap
    return buf, views


@pytest.mark.parametrize("rows,k,n", [(1, 64, 72), (4, 96, 40), (7, 40, 33), (300, 264, 136), (2500, 192, 2304)])
@pytest.mark.parametrize("gap", [8, 3])
def test_slices_of_the_inputs_buffer(cuda_device, rows, k, n, gap):
    buf, (x, y, res) = slices(rows, (k, n, n), BF, gap)
    x.copy_(rand(1, rows, k))
    res.copy_(rand(2, rows, n))
    before = buf.clone()
    w, b = rand(3, n, k, scale=0.1), rand(4, n)
    want = L.linear(x, w, bias=b, residual=res, activation="silu")
    assert L.linear(x, w, bias=b, residual=res, activation="silu", out=y) is y
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert torch.equal(buf, before)
    assert torch.equal(L.linear(x, w, bias=b, residual=res, out=res), L.linear(x, w, bias=b, residual=before[:, -n - gap:][:, :n]))
    dy, dx = y, x
    dy.copy_(rand(5, rows, n))
    p = L.pack8(rand(6, rows, k))
    want = L.linear_backward_input(dy, w, pre=p, activation="gelu")
    assert torch.equal(L.linear_backward_input(dy, w, pre=p, activation="gelu", out=dx), want)
    assert bool((buf[:, k:k + gap] == 7).all())


@pytest.mark.parametrize("rows,k,n", [(3, 64, 72), (8, 33, 40), (300, 264, 136), (2500, 192, 2304), (4096, 1280, 1280)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [8, 3])
def test_weight_gradient_with_a_row_stride(cuda_device, rows, k, n, dtype, gap):
    dy, x = rand(1, rows, n), rand(2, rows, k)
    buf = torch.full((n, k + gap), 7.0, dtype=dtype, device="cuda")
    db = torch.empty(n, dtype=dtype, device="cuda")
    for a, act in ((x, None), (L.pack8(x), "relu")):
        want = L.linear_backward_weight(dy, a, activation=act, grad_dtype=dtype)
        L.linear_backward_weight(dy, a, activation=act, dweight=buf[:, :k], dbias=db)
        assert torch.equal(buf[:, :k], want)
        assert bool((buf[:, k:] == 7).all())
        assert bool(torch.isfinite(db.float()).all())


@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 33), (300, 1280), (77, 1283), (3, 9000)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [16, 8, 3])
def test_8_bit_values_with_a_row_stride(cuda_device, rows, cols, dtype, gap):
    """q cut out of a wider buffer, outputs too."""
    x = rand(1, rows, cols, dtype=dtype)
    p = L.pack8(x)
    wide = torch.zeros(rows, cols + gap, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide.view(torch.uint8)[:, :cols].copy_(p.q.view(torch.uint8))
    s = L.Packed8(wide[:, :cols], p.scale)
    buf, (a, b) = slices(rows, (cols, cols), dtype, gap)
    want = L.unpack8(p, dtype=dtype, activation="gelu")
    assert torch.equal(L.unpack8(s, dtype=dtype, activation="gelu", out=a), want)
    b.copy_(rand(2, rows, cols, dtype=dtype))
    want = L.activation_grad(b, p, "gelu")
    assert torch.equal(L.activation_grad(b, s, "gelu", out=a), want)
    assert torch.equal(L.activation_grad(b, s, "gelu", out=b), want)
    assert bool((buf[:, cols:cols + gap] == 7).all()) and bool((buf[:, 2 * cols + gap:] == 7).all())
    if dtype == BF:
        dy = rand(3, rows, 40)
        assert torch.equal(L.linear_backward_weight(dy, s, activation="silu"),
                           L.linear_backward_weight(dy, p, activation="silu"))
        w = rand(4, 40, cols, scale=0.1)
        assert torch.equal(L.linear_backward_input(dy, w, pre=s, activation="silu"),
                           L.linear_backward_input(dy, w, pre=p, activation="silu"))


@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 33), (300, 512), (130, 1024), (33, 1280), (77, 1283), (6, 5632), (3, 9000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_in_the_place_of_an_input(cuda_device, rows, cols, dtype):
    x, res, w = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype), rand(3, cols, dtype=F32)
    want = L.add_rmsnorm(x, w, residual=res, pack=True)
    lib, t = C.load(), C.SCAPE_BF16 if dtype == BF else C.SCAPE_F32
    st = torch.cuda.current_stream().cuda_stream
    for place in (0, 1):
        a = [x.clone(), res.clone()]
        y, rstd, q = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty_like(want.y8.q.view(torch.uint8))
        s = torch.empty_like(want.y8.scale)
        assert lib.scape_layer_add_rmsnorm(a[0].data_ptr(), cols, a[1].data_ptr(), cols, w.data_ptr(), C.SCAPE_F32, rows,
                                           cols, 1e-5, t, y.data_ptr(), cols, a[place].data_ptr(), cols,
                                           rstd.data_ptr(), q.data_ptr(), cols, s.data_ptr(), st) == C.SCAPE_OK
        assert torch.equal(a[place], want.h) and torch.equal(y, want.y) and torch.equal(rstd, want.rstd)
        assert torch.equal(q, want.y8.q.view(torch.uint8)) and torch.equal(s, want.y8.scale)
    dy, dh = rand(4, rows, cols, dtype=dtype), rand(5, rows, cols, dtype=dtype)
    dw = torch.empty(cols, device="cuda")
    dx = L.add_rmsnorm_backward(dy, want.h, w, want.rstd, dh=dh, dweight=dw)
    again = torch.empty_like(dw)
    own = dh.clone()
    assert torch.equal(L.add_rmsnorm_backward(dy, want.h, w, want.rstd, dh=own, dweight=again, out=own), dx)
    assert torch.equal(again, dw)
    buf, (a, b, c) = slices(rows, (cols, cols, cols), dtype, 5)
    a.copy_(dy), b.copy_(dh)
    L.add_rmsnorm_backward(a, want.h, w, want.rstd, dh=b, dweight=again, out=c)
    # other alignments may sum in another order: a few roundings of 2^-24 apart before the last one
    assert torch.allclose(c.float(), dx.float(), rtol=2.0 ** -7 if dtype == BF else 1e-5, atol=1e-5)
    assert bool((buf[:, cols:cols + 5] == 7).all()) and bool((buf[:, -5:] == 7).all())


def test_outputs_over_inputs_are_refused(cuda_device):
    x, w = rand(1, 16, 64), rand(2, 64, 64)
    keep = x.clone()
    for call in (lambda: L.linear(x, w, out=x), lambda: L.linear_backward_input(x, w, out=x),
                 lambda: L.linear(x, w, out=w[:16]),
                 lambda: L.linear_backward_weight(x, x, dweight=w, dbias=w[0]),
                 lambda: L.add_rmsnorm_backward(x, x, w[0], torch.ones(16, device="cuda"), out=x)):
        with pytest.raises(ScapeError, match="overlap"):
            call()
    assert torch.equal(x, keep)
