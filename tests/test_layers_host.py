"""The training-layer C ABI's refusals, before any GPU work, on any host."""
import ctypes

import pytest

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B

A = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def refused(lib, rc, word):
    assert rc == C.SCAPE_EINVAL
    assert word in lib.scape_layer_last_error().decode()


def test_pack_refusals(lib):
    f = lib.scape_layer_pack8
    refused(lib, f(A, 64, 7, 2, 64, A, 64, A, None), "dtype")
    refused(lib, f(A, 64, C.SCAPE_BF16, -1, 64, A, 64, A, None), "range")
    refused(lib, f(None, 64, C.SCAPE_BF16, 2, 64, A, 64, A, None), "x")
    refused(lib, f(A + 1, 64, C.SCAPE_BF16, 2, 64, A, 64, A, None), "x")
    refused(lib, f(A, 63, C.SCAPE_BF16, 2, 64, A, 64, A, None), "stride")
    refused(lib, f(A, 64, C.SCAPE_BF16, 2, 64, A, 64, None, None), "scale")
    assert f(None, 0, C.SCAPE_BF16, 0, 64, None, 0, None, None) == C.SCAPE_OK  # no rows


def test_unpack_and_act_grad_refusals(lib):
    refused(lib, lib.scape_layer_unpack8(A, 64, A, 2, 64, 9, A, 64, C.SCAPE_BF16, None), "activation")
    refused(lib, lib.scape_layer_unpack8(A, 64, None, 2, 64, 0, A, 64, C.SCAPE_BF16, None), "scale")
    refused(lib, lib.scape_layer_unpack8(A, 64, A, 2, 64, 0, None, 64, C.SCAPE_BF16, None), "y")
    refused(lib, lib.scape_layer_act_grad(A, 64, A, 60, A, 2, 64, 1, A, 64, C.SCAPE_F32, None), "q")


def test_norm_refusals(lib):
    def f(x=A, ldx=64, w=A, wd=C.SCAPE_F32, rows=2, cols=64, eps=1e-5, dt=C.SCAPE_BF16, y=A, q=None,
          s=None):
        return lib.scape_layer_add_rmsnorm(x, ldx, None, 0, w, wd, rows, cols, eps, dt, y, 64, None,
                                           0, None, q, 64, s, None)
    refused(lib, f(x=None), "x")
    refused(lib, f(ldx=10), "stride")
    refused(lib, f(w=None), "weight")
    refused(lib, f(wd=5), "dtype")
    refused(lib, f(eps=-1.0), "eps")
    refused(lib, f(eps=float("nan")), "eps")
    refused(lib, f(y=None), "y")
    refused(lib, f(q=A), "scale")
    assert f(rows=0) == C.SCAPE_OK
    n = ctypes.c_size_t()
    assert lib.scape_layer_add_rmsnorm_bwd_workspace(8, 64, ctypes.byref(n)) == C.SCAPE_OK
    assert n.value >= 64 * 4

    def b(rstd=A, ws=A, nbytes=n.value, dw=A):
        return lib.scape_layer_add_rmsnorm_bwd(A, 64, A, 64, A, C.SCAPE_F32, rstd, None, 0, 8, 64,
                                               C.SCAPE_BF16, A, 64, dw, C.SCAPE_BF16, ws, nbytes,
                                               None)
    refused(lib, b(rstd=None), "rstd")
    refused(lib, b(ws=None), "workspace")
    refused(lib, b(ws=A + 16), "workspace")
    refused(lib, b(nbytes=n.value - 1), "small")
    refused(lib, b(dw=A + 1), "dweight")


def test_linear_refusals(lib):
    n = ctypes.c_size_t(9)
    assert lib.scape_layer_linear_workspace(A, 64, A, 64, 8, 64, 32, ctypes.byref(n)) == C.SCAPE_OK
    assert n.value == 0  # aligned operands need none
    assert lib.scape_layer_linear_workspace(A, 65, A, 64, 16, 64, 32, ctypes.byref(n)) == C.SCAPE_OK
    assert n.value >= 16 * 64 * 2
    assert lib.scape_layer_linear_workspace(A, 65, A, 64, 4, 64, 32, ctypes.byref(n)) == C.SCAPE_OK
    assert n.value == 0  # few rows are read in place whatever their alignment

    def f(x=A, ldx=64, rows=16, k=64, act=0, y=A, ws=None, nbytes=0):
        return lib.scape_layer_linear(x, ldx, A, 64, None, None, 0, rows, k, 32, act, y, 32, None, 0,
                                      None, ws, nbytes, None)
    refused(lib, f(x=None), "x")
    refused(lib, f(k=0), "k")
    refused(lib, f(act=-1), "activation")
    refused(lib, f(y=A + 1), "y")
    refused(lib, f(rows=1 << 31), "range")
    refused(lib, f(ldx=65), "workspace")
    refused(lib, f(ldx=65, ws=A, nbytes=16), "small")
    assert f(rows=0, x=None) == C.SCAPE_OK

    def i(n=32, act=0, q=None):
        return lib.scape_layer_linear_bwd_input(A, 32, A, 64, q, 64, None, act, 8, 64, n, A, 64, None,
                                                0, None)
    refused(lib, i(n=0), "n")
    refused(lib, i(act=2), "scale")

    def w(x=A, q=None, act=0, dw=A, gd=C.SCAPE_BF16, ws=None, nbytes=0):
        return lib.scape_layer_linear_bwd_weight(A, 32, x, 64, q, 64, None, act, 8, 64, 32, dw, 64,
                                                 None, gd, ws, nbytes, None)
    refused(lib, w(x=A, q=A), "both")
    refused(lib, w(act=1), "activation")
    refused(lib, w(x=None), "scale")
    refused(lib, w(dw=None), "dweight")
    refused(lib, w(gd=3), "dtype")


def test_null_outputs(lib):
    refused(lib, lib.scape_layer_status(None, None), "host_status")
    refused(lib, lib.scape_layer_linear_workspace(A, 64, A, 64, 8, 64, 32, None), "bytes")
