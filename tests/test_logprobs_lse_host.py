"""Refusals of the C ABI of the log probabilities with a log-sum-exp of two numbers,
before any GPU work, on any host."""
import pytest

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B

A = 1 << 20  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def refused(lib, rc, word):
    assert rc == C.SCAPE_EINVAL
    assert word in lib.scape_layer_last_error().decode()


def test_forward(lib):
    def f(rows=4, lp=3 * A, lse=4 * A, rest=5 * A, ent=6 * A, x=A):
        return lib.scape_layer_token_logprobs_rest(x, 64, C.SCAPE_BF16, 2 * A, 8, rows, 64, 0, lp, lse, rest, ent, None,
                                                   None, None)
    refused(lib, f(rest=5 * A + 2), "lse_rest")
    refused(lib, f(rest=4 * A), "overlap")
    refused(lib, f(rest=6 * A + 12), "overlap")
    refused(lib, f(rest=A + 64), "overlap")
    refused(lib, f(lse=None), "lse")
    assert f(rows=0, x=None) == C.SCAPE_OK


def test_backward(lib):
    def f(rows=4, lse=3 * A, rest=4 * A, dx=6 * A):
        return lib.scape_layer_token_logprobs_rest_bwd(A, 64, C.SCAPE_F32, 2 * A, 8, rows, 64, lse, rest, 5 * A, None,
                                                       None, dx, 64, None)
    refused(lib, f(rest=4 * A + 1), "lse_rest")
    refused(lib, f(dx=4 * A), "overlap")
    refused(lib, f(lse=None), "lse")
    assert f(rows=0) == C.SCAPE_OK
