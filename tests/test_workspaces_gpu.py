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
