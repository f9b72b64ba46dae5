"""C entry points with a workspace of exactly the size that they ask for, inside a
larger buffer: nothing beside it is written, and results are right."""
import ctypes

import pytest
import torch

from sparse_communication_sharded_gb300 import _scape as C
from tests import _tokens_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIDE, MARK = 8192, 0xA5
DT = {BF: C.SCAPE_BF16, F32: C.SCAPE_F32}


class Space:
    def __init__(self, n):
        self.n, self.all = n, torch.full((n + 2 * SIDE,), MARK, dtype=torch.uint8, device="cuda")
        self.p = self.all.data_ptr() + SIDE

    def check(self):
        assert bool((self.all[:SIDE] == MARK).all()) and bool((self.all[SIDE + self.n:] == MARK).all())


def run(rc):
    assert rc == C.SCAPE_OK, C.load().scape_layer_last_error().decode()
    torch.cuda.synchronize()


@pytest.mark.parametrize("tensors", [1, 47, 48, 49, 388, 768, 769, 1537])
@pytest.mark.parametrize("numel", [1, 5000])
def test_norm(cuda_device, tensors, numel):
    lib = C.load()
    g = torch.Generator(device="cuda").manual_seed(tensors)
    t = [torch.randn(numel + i % 3, device="cuda", generator=g).to(BF if i % 2 else F32) for i in range(tensors)]
    t.insert(tensors // 2, torch.empty(0, device="cuda"))
    n = len(t)
    ptr = (ctypes.c_void_p * n)(*[v.data_ptr() or None for v in t])
    size = (ctypes.c_int64 * n)(*[v.numel() for v in t])
    kind = (ctypes.c_int * n)(*[DT[v.dtype] for v in t])
    need = ctypes.c_size_t()
    assert lib.scape_layer_grad_norm_workspace(n, size, ctypes.byref(need)) == C.SCAPE_OK
    want, tol = R.norm(t)
    st = torch.cuda.current_stream().cuda_stream
    norm, ws = torch.zeros(1, device="cuda"), Space(need.value)
    run(lib.scape_layer_grad_norm(n, ptr, size, kind, norm.data_ptr(), ws.p, ws.n, st))
    ws.check()
    assert abs(float(norm) - want) <= tol * want
    norm.zero_()
    into = [torch.empty_like(v, dtype=F32) for v in t]
    out = (ctypes.c_void_p * n)(*[v.data_ptr() or None for v in into])
    f32 = (ctypes.c_int * n)(*[C.SCAPE_F32] * n)
    run(lib.scape_layer_clip_grads(n, ptr, size, kind, out, f32, want / 2, 0.0, norm.data_ptr(), ws.p, ws.n, st))
    ws.check()
    assert abs(float(norm) - want) <= tol * want
    for a, b in zip(t, into):
        # the factor by the norm's error, its rounding, and the product's
        assert bool(((b.double() - a.double() / 2).abs() <= a.double().abs() * (tol + 2 * R.E)).all())


@pytest.mark.parametrize("count,vocab,cols", [(1, 1, 1), (17, 5, 1), (33, 9, 8200), (579, 3, 700), (1000, 50, 1283),
                                              (5000, 7, 2600), (16 * 4 * 9 + 1, 1, 641), (8191, 999, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [0, 3])
def test_embedding_gradient(cuda_device, count, vocab, cols, dtype, gap):
    """Whole numbers' sums, which are exact; tokens that repeat over many tiles."""
    lib = C.load()
    g = torch.Generator(device="cuda").manual_seed(count)
    dy = torch.randint(-3, 4, (count, cols + gap), device="cuda", generator=g).to(dtype)[:, :cols]
    t = torch.randint(-1, vocab, (count,), device="cuda", generator=g)
    t[count // 3:2 * count // 3] = vocab // 2
    need = ctypes.c_size_t()
    assert lib.scape_layer_embedding_bwd_workspace(count, vocab, cols, ctypes.byref(need)) == C.SCAPE_OK
    dw, ws = torch.full((vocab, cols), 5.0, device="cuda"), Space(need.value)
    want = torch.zeros(vocab + 1, cols, device="cuda", dtype=torch.float64)
    want.index_add_(0, torch.where(t < 0, vocab, t), dy.double())
    for accumulate in (0, 1):
        run(lib.scape_layer_embedding_bwd(dy.data_ptr(), cols + gap, DT[dtype], t.data_ptr(), 8, count, vocab, cols, 1.0,
                                          accumulate, dw.data_ptr(), cols, C.SCAPE_F32, ws.p, ws.n,
                                          torch.cuda.current_stream().cuda_stream))
        ws.check()
        assert torch.equal(dw.double(), want[:vocab] * (1 + accumulate))


@pytest.mark.parametrize("rows,vocab", [(1, 40), (32, 2000), (64, 33), (33, 5001), (256, 1000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_loss_elsewhere(cuda_device, rows, vocab, dtype):
    lib = C.load()
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, device="cuda", generator=g).to(dtype)
    t = torch.randint(-1, vocab, (rows,), device="cuda", generator=g)
    out = torch.empty(rows, vocab + 1, device="cuda", dtype=dtype)[:, 1:]
    args = (x.data_ptr(), vocab, DT[dtype])
    need = ctypes.c_size_t()
    assert lib.scape_layer_token_loss_workspace(*args, rows, vocab, out.data_ptr(), vocab + 1, ctypes.byref(need)) == C.SCAPE_OK
    assert need.value >= 8 * rows  # lse in two numbers
    loss, ws = torch.empty(rows, device="cuda"), Space(need.value)
    run(lib.scape_layer_token_loss(*args, t.data_ptr(), 8, rows, vocab, None, 0.5, loss.data_ptr(), out.data_ptr(), vocab + 1,
                                   ws.p, ws.n, torch.cuda.current_stream().cuda_stream))
    ws.check()
    o = R.Rows(x, t)
    want, tol = o.gradient(torch.full((rows,), -0.5, device="cuda"), dtype)
    assert bool(((out.double() - want).abs() <= tol).all())
    lp, tol = o.logprob()
    assert bool(((loss.double() + 0.5 * lp).abs() <= 0.5 * tol + lp.abs() * R.E).all())
