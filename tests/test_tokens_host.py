"""Refusals of the C ABI of the operators on tokens, logits and sets of gradients,
before any GPU work, on any host; and the binding's, of tensors that are not the
GPU's."""
import ctypes

import pytest
import torch

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B
from sparse_communication_sharded_gb300 import layers as L

A = 1 << 20  # an aligned address that no refused call reads
BF, F32 = C.SCAPE_BF16, C.SCAPE_F32


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def refused(lib, rc, word):
    assert rc == C.SCAPE_EINVAL
    assert word in lib.scape_layer_last_error().decode()


def test_embedding(lib):
    def f(tokens=A, tb=8, count=4, w=2 * A, ldw=64, wd=BF, vocab=10, cols=64, y=3 * A, ldy=64, d=BF):
        return lib.scape_layer_embedding(tokens, tb, count, w, ldw, wd, vocab, cols, 1.0, y, ldy, d, None)
    refused(lib, f(wd=7), "dtype")
    refused(lib, f(d=-1), "dtype")
    refused(lib, f(tb=2), "token_bytes")
    refused(lib, f(tokens=None), "tokens")
    refused(lib, f(tokens=A + 4), "tokens")
    refused(lib, f(count=-1), "range")
    refused(lib, f(count=1 << 31), "range")
    refused(lib, f(vocab=0), "vocab")
    refused(lib, f(vocab=-5), "range")
    refused(lib, f(cols=(1 << 30) + 1, ldw=1 << 31, ldy=1 << 31), "range")
    refused(lib, f(w=None), "weight")
    refused(lib, f(w=2 * A + 1), "weight")
    refused(lib, f(ldw=63), "stride")
    refused(lib, f(y=None), "y")
    refused(lib, f(ldy=10), "stride")
    refused(lib, f(y=2 * A + 64), "overlap")
    refused(lib, f(y=A, ldy=64), "overlap")
    assert f(count=0, tokens=None, y=None) == C.SCAPE_OK
    assert f(cols=0, y=None) == C.SCAPE_OK


def test_embedding_backward(lib):
    n = ctypes.c_size_t()
    assert lib.scape_layer_embedding_bwd_workspace(100, 10, 64, ctypes.byref(n)) == C.SCAPE_OK
    need = n.value
    assert need >= 100 * 8 + 11 * 4 + 7 * 2 * 64 * 4
    assert lib.scape_layer_embedding_bwd_workspace(0, 10, 64, ctypes.byref(n)) == C.SCAPE_OK and n.value == 0
    refused(lib, lib.scape_layer_embedding_bwd_workspace(1, 1, 1, None), "bytes")
    refused(lib, lib.scape_layer_embedding_bwd_workspace(1 << 32, 1, 1, ctypes.byref(n)), "range")

    def f(dy=A, lddy=64, d=BF, tokens=2 * A, tb=4, count=100, vocab=10, cols=64, dw=3 * A, lddw=64, wd=F32, ws=4 * A,
          nb=need):
        return lib.scape_layer_embedding_bwd(dy, lddy, d, tokens, tb, count, vocab, cols, 1.0, 0, dw, lddw, wd, ws, nb,
                                             None)
    refused(lib, f(d=3), "dtype")
    refused(lib, f(wd=3), "dtype")
    refused(lib, f(dy=None), "dy")
    refused(lib, f(lddy=60), "stride")
    refused(lib, f(tokens=None), "tokens")
    refused(lib, f(tb=1), "token_bytes")
    refused(lib, f(vocab=0), "vocab")
    refused(lib, f(dw=None), "dweight")
    refused(lib, f(dw=3 * A + 2), "dweight")
    refused(lib, f(lddw=63), "stride")
    refused(lib, f(ws=None), "workspace")
    refused(lib, f(ws=4 * A + 16), "workspace")
    refused(lib, f(nb=need - 1), "small")
    refused(lib, f(dw=A), "overlap")
    refused(lib, f(ws=3 * A), "overlap")
    assert f(cols=0) == C.SCAPE_OK


def test_logprobs(lib):
    def f(x=A, ldx=64, d=BF, t=2 * A, tb=8, rows=4, vocab=64, top=0, lp=3 * A, lse=4 * A, ent=None, tl=None, tt=None):
        return lib.scape_layer_token_logprobs(x, ldx, d, t, tb, rows, vocab, top, lp, lse, ent, tl, tt, None)
    refused(lib, f(d=9), "dtype")
    refused(lib, f(x=None), "logits")
    refused(lib, f(ldx=63), "stride")
    refused(lib, f(t=None), "targets")
    refused(lib, f(t=2 * A + 4), "targets")
    refused(lib, f(tb=16), "token_bytes")
    refused(lib, f(rows=-1), "range")
    refused(lib, f(vocab=(1 << 30) + 1, ldx=1 << 31), "range")
    refused(lib, f(vocab=0), "vocab")
    refused(lib, f(top=33), "top")
    refused(lib, f(top=-1), "top")
    refused(lib, f(vocab=4, top=5), "top")
    refused(lib, f(vocab=(1 << 22) + 1, ldx=(1 << 22) + 1, top=1), "too large")
    refused(lib, f(lp=None), "logprob")
    refused(lib, f(lse=4 * A + 2), "lse")
    refused(lib, f(ent=5), "entropy")
    refused(lib, f(top=3), "top_logprob")
    refused(lib, f(top=3, tl=5 * A), "top_token")
    refused(lib, f(top=3, tl=5 * A, tt=6 * A + 4), "top_token")
    refused(lib, f(lse=3 * A), "overlap")
    refused(lib, f(lp=A + 16), "overlap")
    assert f(rows=0, x=None) == C.SCAPE_OK


def test_gradients_of_logits(lib):
    def f(x=A, ldx=64, t=2 * A, rows=4, vocab=64, lse=3 * A, dlp=4 * A, ent=None, dent=None, dx=5 * A, lddx=64):
        return lib.scape_layer_token_logprobs_bwd(x, ldx, F32, t, 8, rows, vocab, lse, dlp, ent, dent, dx, lddx, None)
    refused(lib, f(x=None), "logits")
    refused(lib, f(lse=None), "lse")
    refused(lib, f(dlp=None), "dlogprob")
    refused(lib, f(dent=6 * A), "entropy")
    refused(lib, f(dx=None), "dlogits")
    refused(lib, f(lddx=3), "stride")
    refused(lib, f(dx=A + 4), "overlap")
    refused(lib, f(dx=A, lddx=65), "overlap")
    refused(lib, f(dx=3 * A), "overlap")
    assert f(rows=0) == C.SCAPE_OK
    n = ctypes.c_size_t()

    def g(x=A, t=2 * A, rows=4, vocab=64, w=3 * A, loss=4 * A, dx=5 * A, ws=6 * A, nb=1 << 20):
        return lib.scape_layer_token_loss(x, vocab, BF, t, 8, rows, vocab, w, 1.0, loss, dx, vocab, ws, nb, None)
    refused(lib, g(x=None), "logits")
    refused(lib, g(t=None), "targets")
    refused(lib, g(w=3 * A + 1), "weight")
    refused(lib, g(loss=None), "loss")
    refused(lib, g(dx=None), "dlogits")
    refused(lib, g(dx=A + 2), "overlap")
    refused(lib, g(loss=5 * A), "overlap")
    assert g(rows=0) == C.SCAPE_OK
    refused(lib, lib.scape_layer_token_loss_workspace(A, 64, BF, 4, 64, A, 64, None), "bytes")
    # a row that no cluster of blocks holds
    wide = 1 << 21
    assert lib.scape_layer_token_loss_workspace(A, wide, F32, 4, wide, 2 * A, wide, ctypes.byref(n)) == C.SCAPE_OK
    assert n.value >= 16
    refused(lib, g(vocab=wide, dx=100 * A, ws=None), "workspace")
    refused(lib, g(vocab=wide, dx=100 * A, nb=8), "small")


def arrays(ptrs, numel, dtype):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int * n)(*dtype))


def test_sets_of_gradients(lib):
    n = ctypes.c_size_t()
    _, numel, _ = arrays([A, A], [100, 5], [0, 0])
    assert lib.scape_layer_grad_norm_workspace(2, numel, ctypes.byref(n)) == C.SCAPE_OK and n.value >= 16
    refused(lib, lib.scape_layer_grad_norm_workspace(2, numel, None), "bytes")
    refused(lib, lib.scape_layer_grad_norm_workspace(2, None, ctypes.byref(n)), "host_numel")
    refused(lib, lib.scape_layer_grad_norm_workspace(-1, numel, ctypes.byref(n)), "n is below")

    def f(ptrs=(A, 2 * A), numel=(100, 5), dtype=(F32, BF), norm=3 * A, ws=4 * A, nb=4096):
        p, m, d = arrays(ptrs, numel, dtype)
        return lib.scape_layer_grad_norm(len(ptrs), p, m, d, norm, ws, nb, None)
    refused(lib, f(ptrs=(A, None)), "NULL")
    refused(lib, f(ptrs=(A + 2, 2 * A)), "misaligned")
    refused(lib, f(numel=(-1, 5)), "range")
    refused(lib, f(numel=(1 << 60, 5)), "range")
    refused(lib, f(dtype=(4, 0)), "dtype")
    refused(lib, f(norm=None), "norm")
    refused(lib, f(ws=None), "workspace")
    refused(lib, f(nb=8), "small")
    refused(lib, f(norm=A + 4), "overlap")
    refused(lib, f(ws=A, norm=3 * A), "overlap")
    refused(lib, lib.scape_layer_grad_norm(2, None, numel, None, A, A, 4096, None), "array")

    def g(ptrs=(A, 2 * A), numel=(100, 5), dtype=(F32, BF), out=None, odt=None, top=1.0, eps=0.0, norm=3 * A):
        p, m, d = arrays(ptrs, numel, dtype)
        o, _, q = arrays(out, numel, odt) if out else (None, None, None)
        return lib.scape_layer_clip_grads(len(ptrs), p, m, d, o, q, top, eps, norm, 4 * A, 4096, None)
    refused(lib, g(top=-1.0), "max_norm")
    refused(lib, g(top=float("nan")), "max_norm")
    refused(lib, g(eps=-1.0), "eps")
    refused(lib, g(eps=float("inf")), "eps")
    refused(lib, g(out=(5 * A, None), odt=(F32, F32)), "output")
    refused(lib, g(out=(5 * A, 6 * A), odt=(F32, 5)), "dtype")
    refused(lib, g(ptrs=(A, A)), "overlap")                                 # in place, twice
    refused(lib, g(ptrs=(A, A + 396)), "overlap")
    refused(lib, g(out=(A, 6 * A), odt=(BF, F32)), "overlap")               # its own place in another type
    refused(lib, g(out=(2 * A, 6 * A), odt=(F32, F32)), "overlap")          # another's
    refused(lib, g(out=(5 * A, 5 * A + 199), odt=(F32, F32)), "misaligned")
    refused(lib, g(out=(5 * A, 5 * A + 196), odt=(F32, F32)), "overlap")
    refused(lib, g(out=(3 * A, 6 * A), odt=(F32, F32)), "overlap")          # the norm


def test_tensors_of_the_host():
    t, x = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8)
    f = torch.zeros(4)
    for bad in (lambda: L.embedding(t, x), lambda: L.embedding_backward(x, t, x), lambda: L.token_logprobs(x, t),
                lambda: L.token_logprobs_backward(x, t, f, f), lambda: L.token_loss(x, t, 1.0),
                lambda: L.grad_norm([x]), lambda: L.clip_grad_norm([x], 1.0), lambda: L.grad_norm([]),
                lambda: L.embedding(3, x), lambda: L.token_logprobs_backward(x, t, f, f, dentropy=f)):
        with pytest.raises(ValueError):
            bad()
