"""The norm of a set of gradients and their clipping against 64-bit sums."""
import math

import pytest
import torch

from sparse_communication_sharded_gb300 import ScapeError
from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def grads_of(seed, sizes, dtype, offset=0, scale=1e-3):
    """Views of a flat vector, one behind the other (dtype None: of both types in turn,
    each in a vector of its own)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype is None:
        return [(torch.randn(n + offset, device="cuda", generator=g) * scale).to((BF, F32)[i % 2])[offset:]
                for i, n in enumerate(sizes)]
    flat = (torch.randn(sum(sizes) + offset, device="cuda", generator=g) * scale).to(dtype)
    return list(torch.split(flat[offset:], sizes))


SETS = [[1], [7], [0, 5, 0], [8192], [8193, 1, 4095], [100000], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10], [33] * 100,
        [2000003, 17, 300000], [1] * 800, [4097] * 1700]


def check_norm(got, grads):
    want, rel = R.norm(grads)
    assert got.dtype == F32 and got.dim() == 0
    if want >= 2.0 ** 128 - 2.0 ** 103:  # rounds to infinity: past float32's range by half a step
        assert float(got) == math.inf
        return
    assert abs(float(got) - want) <= rel * want, (float(got), want)


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", [BF, F32, None])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_norm(cuda_device, sizes, dtype, offset):
    grads = grads_of(len(sizes), sizes, dtype, offset)
    a = L.grad_norm(grads)
    check_norm(a, grads)
    assert torch.equal(a, L.grad_norm(tuple(grads)))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-22, 1e-12, 1.0, 1e12, 1e19, 3e30, 1e37])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_over_the_whole_range(cuda_device, scale, dtype):
    """Squares leave float32's range on either side; the norm does not."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.randn(50000, device="cuda", generator=g) * scale).to(dtype)
    x[1000:40000] = 0.0
    check_norm(L.grad_norm([x]), [x])
    check_norm(L.grad_norm([x, torch.zeros(9000, device="cuda"), x[:77]]), [x, x[:77]])
    mixed = torch.cat([x, (torch.randn(3000, device="cuda", generator=g) * scale * 1e-15).to(dtype)])
    check_norm(L.grad_norm([mixed]), [mixed])


def test_norm_of_nothing_and_of_what_is_not_finite(cuda_device):
    assert float(L.grad_norm([torch.zeros(0, device="cuda")])) == 0
    assert float(L.grad_norm([torch.zeros(100000, device="cuda", dtype=BF)])) == 0
    x = torch.ones(30000, device="cuda")
    x[12345] = -math.inf
    assert float(L.grad_norm([x])) == math.inf
    x[20000] = math.nan
    assert math.isnan(float(L.grad_norm([x, x])))


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (F32, BF), (BF, F32), (None, BF)])
@pytest.mark.parametrize("offset,into", [(0, 0), (1, 3), (8, 1)])
@pytest.mark.parametrize("over", [0.5, 4.0])
def test_clip(cuda_device, sizes, dtype, out, offset, into, over):
    grads = grads_of(len(sizes) + 1, sizes, dtype, offset)
    before = [g.clone() for g in grads]
    norm, rel = R.norm(grads)
    flat = torch.full((into + sum(sizes) + 5,), 7.0, dtype=out, device="cuda")
    outs = list(torch.split(flat[into:into + sum(sizes)], sizes))
    max_norm = float(torch.tensor(norm / over, dtype=F32))
    check_norm(L.clip_grad_norm(grads, max_norm, out=outs), before)
    factor = min(1.0, max_norm / (norm + 1e-6))
    for g, b, o in zip(grads, before, outs):
        assert torch.equal(g, b)
        want = b.double() * factor
        assert bool(((o.double() - want).abs() <= want.abs() * (R.U(out) + rel + 2 * R.E) + 1e-44).all())
    flat[into:into + sum(sizes)] = 7.0
    assert bool((flat == 7).all())
    if dtype is not None and out is dtype:
        assert torch.equal(L.clip_grad_norm(grads, max_norm), L.clip_grad_norm(before, 1e30))
        for g, b in zip(grads, before):
            want = b.double() * factor
            assert bool(((g.double() - want).abs() <= want.abs() * (R.U(out) + rel + 2 * R.E) + 1e-44).all())
        if over < 1:
            assert all(torch.equal(g, b) for g, b in zip(grads, before))


def test_factor_as_it_comes_out(cuda_device):
    x = torch.tensor([3.0, 4.0, 0.0], device="cuda")
    for bad, norm in ((math.inf, math.inf), (math.nan, math.nan)):
        y = x.clone()
        y[2] = bad
        got = L.clip_grad_norm([y], 1.0)
        assert float(got) == norm or (math.isnan(norm) and math.isnan(float(got)))
        if norm == math.inf:
            assert y[:2].tolist() == [0.0, 0.0] and math.isnan(float(y[2]))
        else:
            assert bool(torch.isnan(y).all())
    y = x.clone()
    assert float(L.clip_grad_norm([y], 0.0)) == 5.0 and not bool(y.any())
    y = x.clone()
    L.clip_grad_norm([y], math.inf)
    assert torch.equal(y, x)
    y = torch.zeros(9, device="cuda")
    assert float(L.clip_grad_norm([y], 0.0, eps=0.0)) == 0 and bool(torch.isnan(y).all())  # 0 / 0


def test_order_of_dimensions(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn(70, 30, device="cuda", generator=g)
    b = torch.randn(4, 5, 6, 7, device="cuda", generator=g).to(memory_format=torch.channels_last)
    grads = [a.t(), b]
    want = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads]
    assert out[0].stride() == grads[0].stride() and out[1].stride() == b.stride()
    norm = L.clip_grad_norm(grads, 1.0, out=out)
    check_norm(norm, want)
    for o, w in zip(out, want):
        assert bool(torch.allclose(o, w / float(norm), rtol=1e-5))
    with pytest.raises(ValueError):
        L.clip_grad_norm(grads, 1.0, out=[torch.empty(30, 70, device="cuda"), out[1]])


def test_refusals(cuda_device):
    x, y = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for bad in (lambda: L.grad_norm([]), lambda: L.grad_norm(x), lambda: L.grad_norm([x, None]),
                lambda: L.grad_norm([x.half()]), lambda: L.grad_norm([x.cpu()]), lambda: L.grad_norm([x[::2]]),
                lambda: L.grad_norm([x.view(8, 8)[:, :4]]), lambda: L.grad_norm([x[:1].expand(5)]),
                lambda: L.grad_norm(7), lambda: L.grad_norm([x.clone().requires_grad_()]),
                lambda: L.clip_grad_norm([x], 1.0, out=[x, y]), lambda: L.clip_grad_norm([x], 1.0, out=[y[:32]]),
                lambda: L.clip_grad_norm([x], "a"), lambda: L.clip_grad_norm([x], 1.0, out=[y.half()])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: L.clip_grad_norm([x], -1.0), lambda: L.clip_grad_norm([x], math.nan),
                lambda: L.clip_grad_norm([x], 1.0, eps=-1.0), lambda: L.clip_grad_norm([x], 1.0, eps=math.inf),
                lambda: L.clip_grad_norm([x, x], 1.0), lambda: L.clip_grad_norm([x[:40], x[30:]], 1.0),
                lambda: L.clip_grad_norm([x, y], 1.0, out=[y, x]), lambda: L.clip_grad_norm([x], 1.0, out=[x.view(BF)[:64]]),
                lambda: L.clip_grad_norm([x[:32], x[32:]], 1.0, out=[y[:32], y[16:48]]),
                lambda: L.clip_grad_norm([x[:32]], 1.0, out=[x[16:48]])):
        with pytest.raises(ScapeError):
            bad()
    assert float(L.grad_norm([x, x])) == 0  # read twice is fine


def test_written_tensors_count_as_modified(cuda_device):
    x, y = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    a, b = x._version, y._version
    L.clip_grad_norm([x], 1.0, out=[y])
    assert x._version == a and y._version > b
    L.clip_grad_norm([x], 1.0)
    assert x._version > a
