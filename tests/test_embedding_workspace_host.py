"""How much memory the embedding's gradient asks for, part by part, on any host."""
import ctypes

import pytest

from sparse_communication_sharded_gb300 import _scape as C
from sparse_communication_sharded_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return C.load()


@pytest.mark.parametrize("count", [1, 16, 17, 100, 8192, 65537])
@pytest.mark.parametrize("vocab", [1, 10, 50304])
@pytest.mark.parametrize("cols", [1, 64, 640, 641, 1283, 8192])
def test_room_for_every_part(lib, count, vocab, cols):
    """16 bytes a position, 4 a row of the table and one more, and for every 16 positions
    a counter for each 640 columns (160 threads with 4 each) and two sums of all columns
    in 32 bits; no more than 256 bytes beside each."""
    n = ctypes.c_size_t()
    assert lib.scape_layer_embedding_bwd_workspace(count, vocab, cols, ctypes.byref(n)) == C.SCAPE_OK
    tiles = -(-count // 16)
    parts = [16 * count, 4 * (vocab + 1), 4 * tiles * -(-cols // 640), 8 * tiles * (-(-cols // 8) * 8)]
    assert sum(parts) <= n.value <= sum(parts) + 4 * 256
