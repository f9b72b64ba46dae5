"""How much memory the norm of a set of gradients asks for, on any host."""
import ctypes

import pytest

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


def workspace(lib, numel):
    n = ctypes.c_size_t()
    assert lib.scape_layer_grad_norm_workspace(len(numel), (ctypes.c_int64 * len(numel))(*numel),
                                               ctypes.byref(n)) == C.SCAPE_OK
    return n.value


# 64 bits a block, of which one launch has 4 an SM at most (of 256 SMs at most), and a
# launch takes 768 tensors that are not empty
LAUNCH = 8 * 4 * 256


@pytest.mark.parametrize("tensors,launches", [(1, 1), (48, 1), (49, 1), (219, 1), (388, 1), (768, 1), (769, 2), (2000, 3)])
def test_a_few_blocks_a_launch(lib, tensors, launches):
    need = workspace(lib, [1 << 24] * tensors)
    assert need <= launches * LAUNCH
    assert workspace(lib, [0, 1 << 24] * tensors) == need  # empty ones take nothing
    assert workspace(lib, [1 << 26] * tensors) == need


def test_of_tensors_as_large_as_can_be(lib):
    """Their pieces' numbers end a launch's table before its tensors do."""
    assert workspace(lib, [1 << 38] * 64) <= 5 * LAUNCH
    assert workspace(lib, []) == 0 and workspace(lib, [0, 0]) == 0
    assert workspace(lib, [1]) >= 8
