"""Matrices whose rows start on 16 bytes but do not end there: what lies beside them
in a wider buffer is neither written nor multiplied."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def wide(seed, rows, cols, pitch, scale=1.0):
    """A slice of a buffer whose other columns hold NaN, and its contiguous copy's bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((rows, pitch), NAN, dtype=BF, device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, device="cuda", generator=g) * scale).to(BF)
    return buf[:, :cols]


def copy_of(t):
    """The same values in rows of the same kind of alignment with zeros beside them."""
    buf = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


@pytest.mark.parametrize("cols", [1281, 1284, 1286, 1287])
@pytest.mark.parametrize("rows", [3, 8, 200, 4090])
def test_products(cuda_device, rows, cols):
    k = n = cols
    pitch = 1288
    x, w, dy = wide(1, rows, k, pitch), wide(2, n, k, pitch, k ** -0.5), wide(3, rows, n, pitch)
    clean = [copy_of(t) for t in (x, w, dy)]

    def run(x, w, dy, out):
        y = torch.full((rows, pitch), 7.0, dtype=BF, device="cuda")
        dx, dw = y.clone(), torch.full((n, pitch), 7.0, dtype=BF, device="cuda")
        dw32 = dw.float()
        L.linear(x, w, activation="silu", out=y[:, :n])
        L.linear_backward_input(dy, w, out=dx[:, :k])
        L.linear_backward_weight(dy, x, dweight=dw[:, :k])
        L.linear_backward_weight(dy, x, dweight=dw32[:, :k])
        out.extend([y, dx, dw, dw32])

    got, want = [], []
    run(x, w, dy, got)
    run(*clean, want)
    for a, b in zip(got, want):
        assert bool(torch.isfinite(a.float()).all())
        assert torch.equal(a, b)
        assert bool((a[:, cols:] == 7).all())
    z = torch.nn.functional.silu(x.double() @ w.double().t())
    assert float((got[0][:, :n].double() - z).abs().max()) < 0.05


@pytest.mark.parametrize("cols", [33, 1281, 1286, 5625])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_other_operators(cuda_device, cols, dtype):
    rows, pitch = 37, -(-cols // 16) * 16
    x, res = wide(1, rows, cols, pitch).to(dtype), None
    buf = torch.full((rows, pitch), NAN, dtype=dtype, device="cuda")
    buf[:, :cols] = x
    x = buf[:, :cols]
    clean = copy_of(x)
    w = torch.ones(cols, device="cuda")
    a, b = L.add_rmsnorm(x, w, residual=res, pack=True), L.add_rmsnorm(clean, w, residual=res, pack=True)
    assert torch.equal(a.y, b.y) and torch.equal(a.y8.q.view(torch.uint8), b.y8.q.view(torch.uint8))
    p, q = L.pack8(x), L.pack8(clean)
    assert torch.equal(p.q.view(torch.uint8), q.q.view(torch.uint8)) and torch.equal(p.scale, q.scale)
    g, h = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    for f in (lambda t, o, s: L.unpack8(p, dtype=dtype, activation="gelu", out=o),
              lambda t, o, s: L.activation_grad(t, p, "gelu", out=o),
              lambda t, o, s: L.add_rmsnorm_backward(t, t, w, a.rstd, dh=t, dweight=s, out=o)):
        o1, o2 = (torch.full((rows, pitch), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        f(x, o1[:, :cols], g)
        f(clean, o2[:, :cols], h)
        assert torch.equal(o1, o2) and bool((o1[:, cols:] == 7).all()) and bool(torch.isfinite(o1).all())
    assert torch.equal(g, h)
