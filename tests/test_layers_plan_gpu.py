"""Products through every kernel and tile width that the choice of tiles can make,
each with the sizes that lead there and a check that they still do."""
import ctypes

import pytest
import torch

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORWARD, INPUT_GRAD, WEIGHT_GRAD = 0, 1, 2
FEW, SPLIT, PAIRS, REST = 0, 1, 2, 3


def plan(product, rows, k, n, keep=False):
    v = [ctypes.c_int() for _ in range(3)]
    assert C.load().scape_layer_linear_plan(product, rows, k, n, keep, *[ctypes.byref(x) for x in v]) == C.SCAPE_OK
    return tuple(x.value for x in v)


def rand(seed, *shape, scale=1.0, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape[:-1], shape[-1] + gap, device="cuda", generator=g) * scale).to(BF)[..., :shape[-1]]


def near(got, want, tol, what):
    assert bool(torch.isfinite(got.float()).all()), what
    over = ((got.double() - want).abs() - tol).max()
    assert float(over) <= 0, f"{what}: over by {float(over):.3g}"


def sums(a, b, k):
    """32-bit sums of k exact products, in any order, cut or rounded."""
    return (a.double().abs() @ b.double().abs()) * (k + 2) * 2.0 ** -23


def check_forward(rows, k, n, act, residual, keep, gap):
    x, w, b = rand(1, rows, k), rand(2, n, k, scale=k ** -0.5), rand(3, n)
    res = rand(4, rows, n, gap=gap) if residual else None
    out = torch.full((rows, n + gap), 7.0, dtype=BF, device="cuda")
    r = L.linear(x, w, bias=b, residual=res, activation=act, keep_pre=keep, out=out[:, :n])
    z, e = x.double() @ w.double().t() + b.double(), sums(x, w.t(), k)
    e = e + z.abs() * 2.0 ** -23
    a = R.act(z, act)
    want = a + res.double() if residual else a
    tol = want.abs() * R.U_BF16 + 1.2 * e + a.abs() * R.ACT_REL + (res.double().abs() * 2.0 ** -23 if residual else 0)
    near(out[:, :n], want, tol, "y")
    assert bool((out[:, n:] == 7).all())
    if keep:
        near(L.unpack8(r[1], dtype=F32), z, R.pack_error(z) + 1.1 * e + R.blocks(e).amax(-1)
             .repeat_interleave(32, dim=1)[:, :n] * 2.0 ** -17, "z8")
    assert L.status() == 0


@pytest.mark.parametrize("rows,k,n,expected", [
    (4, 96, 200, (FEW, 0, 0)), (166, 179, 8, (SPLIT, 64, 1)), (9, 767, 39, (SPLIT, 64, 2)), (17, 1283, 41, (SPLIT, 64, 4)),
    (24, 2162, 22, (SPLIT, 64, 8)), (409, 9, 2510, (SPLIT, 128, 1)), (17581, 10, 9, (PAIRS, 128, 0)),
    (3049, 8, 821, (PAIRS, 160, 0)), (8071, 9, 352, (PAIRS, 192, 0)), (14739, 8, 201, (PAIRS, 224, 0)),
    (1135, 9, 3789, (PAIRS, 256, 0)), (14399, 705, 261, (PAIRS, 320, 0)), (14387, 662, 326, (PAIRS, 384, 0)),
    (22152, 1967, 8, (REST, 128, 4)), (20182, 2059, 8, (REST, 128, 8)), (23131, 2024, 235, (REST, 256, 2)),
    (21166, 1225, 231, (REST, 256, 4)), (19520, 2039, 133, (REST, 256, 8))])
def test_forward(cuda_device, rows, k, n, expected):
    assert plan(FORWARD, rows, k, n) == expected
    check_forward(rows, k, n, None, True, False, 0)
    if plan(FORWARD, rows, k, n, True) == expected:
        check_forward(rows, k, n, "gelu", False, True, 0)
    check_forward(rows, k, n, "silu", True, False, 2)


@pytest.mark.parametrize("n", [1500, 1496, 1498, 1497])
@pytest.mark.parametrize("gap", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("act", [None, "relu"])
def test_forward_output_rows_of_any_alignment(cuda_device, n, gap, act):
    """Rows that start on 16, 8, 4 and 2 bytes, of tiles by pairs; a last tile whose
    columns end inside a 32-column box, at odd places too."""
    assert plan(FORWARD, 4090, 40, n)[0] == PAIRS
    check_forward(4090, 40, n, act, True, act is not None, gap)


def check_input_grad(rows, k, n, act, gap):
    dy, w = rand(1, rows, n), rand(2, n, k, scale=n ** -0.5)
    p = L.pack8(rand(3, rows, k, scale=2.0)) if act else None
    out = torch.full((rows, k + gap), 7.0, dtype=BF, device="cuda")
    L.linear_backward_input(dy, w, pre=p, activation=act, out=out[:, :k])
    want, e = dy.double() @ w.double(), sums(dy, w, n)
    if act:
        e = e * 1.2 + want.abs() * 3 * R.ACT_REL
        want = want * R.slope(R.values(p.q.view(torch.uint8), p.scale), act)
    near(out[:, :k], want, want.abs() * R.U_BF16 + e, "dx")
    assert bool((out[:, k:] == 7).all())
    assert L.status() == 0


@pytest.mark.parametrize("rows,k,n,expected", [
    (3, 96, 200, (FEW, 0, 0)), (166, 179, 8, (SPLIT, 64, 1)), (130, 10, 466, (SPLIT, 64, 2)), (9, 86, 1112, (SPLIT, 64, 4)),
    (44, 10, 2028, (SPLIT, 64, 8)), (1331, 867, 8, (SPLIT, 128, 1)), (17581, 10, 9, (PAIRS, 128, 0)),
    (2340, 908, 9, (PAIRS, 160, 0)), (2480, 1025, 9, (PAIRS, 192, 0)), (610, 4149, 8, (PAIRS, 224, 0)),
    (16967, 157, 9, (PAIRS, 256, 0)), (14542, 267, 343, (PAIRS, 320, 0)), (3849, 1310, 394, (PAIRS, 384, 0)),
    (21718, 8, 1928, (REST, 128, 4)), (20843, 10, 2172, (REST, 128, 8)), (22811, 130, 2104, (REST, 256, 2)),
    (19845, 134, 1219, (REST, 256, 4)), (20043, 134, 2162, (REST, 256, 8))])
def test_input_gradient(cuda_device, rows, k, n, expected):
    assert plan(INPUT_GRAD, rows, k, n) == expected
    check_input_grad(rows, k, n, None, 0)
    check_input_grad(rows, k, n, "gelu", 2)


@pytest.mark.parametrize("rows,k,n,expected", [
    (7, 169, 88, (FEW, 0, 0)), (166, 179, 8, (SPLIT, 64, 1)), (780, 20, 27, (SPLIT, 64, 2)), (1114, 8, 292, (SPLIT, 64, 4)),
    (8191, 12, 10, (SPLIT, 64, 8)), (10, 3249, 277, (SPLIT, 128, 1)), (9, 2723, 558, (PAIRS, 128, 0)),
    (10, 1255, 1803, (PAIRS, 160, 0)), (9, 603, 4065, (PAIRS, 192, 0)), (9, 3542, 776, (PAIRS, 224, 0)),
    (9, 2916, 1073, (PAIRS, 256, 0)), (327, 3214, 1315, (PAIRS, 320, 0)), (394, 1329, 3866, (PAIRS, 384, 0)),
    (1952, 773, 2768, (REST, 128, 4)), (2007, 776, 2609, (REST, 128, 8)), (2031, 2583, 3610, (REST, 256, 2)),
    (1228, 2110, 4122, (REST, 256, 4)), (2735, 1559, 2696, (REST, 256, 8))])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradient(cuda_device, rows, k, n, expected, dtype):
    assert plan(WEIGHT_GRAD, rows, k, n) == expected
    dy = rand(1, rows, n)
    for x, act in ((rand(2, rows, k), None), (L.pack8(rand(2, rows, k, scale=2.0)), "relu")):
        a = x.double() if act is None else R.act(R.values(x.q.view(torch.uint8), x.scale), act)
        db = torch.empty(n, dtype=dtype, device="cuda")
        dw = L.linear_backward_weight(dy, x, activation=act, dbias=db, grad_dtype=dtype)
        want = dy.double().t() @ a
        near(dw, want, want.abs() * R.u_of(dtype) + sums(dy.t(), a, rows), "dw")
        s = dy.double().sum(0)
        near(db, s, s.abs() * R.u_of(dtype) + dy.double().abs().sum(0) * (rows + 2) * 2.0 ** -24, "db")
    assert L.status() == 0
