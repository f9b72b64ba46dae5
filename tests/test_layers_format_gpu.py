"""The 8-bit format at the ends of its range: what is packed there is read back as
the format's value, rounded to the type."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _layers_oracle as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def read(p, dtype, stride):
    """Aligned rows, or rows that every kernel reads element by element."""
    if not stride:
        return L.unpack8(p, dtype=dtype)
    out = torch.empty(p.q.shape[0], p.q.shape[1] + stride, dtype=dtype, device="cuda")[:, :p.q.shape[1]]
    return L.unpack8(p, dtype=dtype, out=out)


@pytest.mark.parametrize("stride", [0, 3])
@pytest.mark.parametrize("cols", [64, 40, 39])
def test_every_value_of_every_scale(cuda_device, cols, stride):
    """All 254 finite bytes under every scale that pack8 writes, 1 to 247."""
    finite = torch.tensor([b for b in range(256) if b & 127 != 127], dtype=torch.uint8, device="cuda")
    n = -(-254 // cols)
    q = torch.nn.functional.pad(finite, (0, n * cols - 254)).view(n, cols).repeat(247, 1)
    code = torch.arange(1, 248, dtype=torch.uint8, device="cuda").repeat_interleave(n)[:, None]
    p = L.Packed8(q.view(torch.float8_e4m3fn), code.expand(-1, -(-cols // 32)).contiguous())
    want = R.values(q, p.scale)
    # float32 and bfloat16 share their range, 2^128 on is infinity; a value has 4 significant bits
    far = want.abs() >= 2.0 ** 128
    assert bool(far.any())
    for dtype, step in ((F32, 2.0 ** -149), (BF, 2.0 ** -133)):
        w = torch.where(want.abs() < 2.0 ** -120, torch.round(want / step) * step, want)
        w = torch.where(far, torch.copysign(torch.full_like(w, float("inf")), want), w)
        assert torch.equal(read(p, dtype, stride).double(), w)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("stride", [0, 3])
def test_packed_and_read_back_at_the_ends(cuda_device, dtype, stride):
    big, tiny = torch.finfo(dtype).max, 2.0 ** (-133 if dtype == BF else -149)
    rows = [[big], [-big], [248 * 2.0 ** 120], [247 * 2.0 ** 120], [tiny], [-tiny, 3 * tiny], [2.0 ** -126, tiny]]
    x = torch.zeros(len(rows), 40, dtype=torch.float64)
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r, dtype=torch.float64)
    x = x.to("cuda").to(dtype)
    p = L.pack8(x)
    v, code = R.pack8(x.double())
    assert torch.equal(p.scale, code)
    got = read(p, dtype, stride).double()
    inf = float("inf")
    assert got[0, 0] == inf and got[1, 0] == -inf
    # bfloat16's steps there are 2^120: 248 lies in the middle and goes to the even 256
    assert got[2, 0] == inf and got[3, 0] == 240 * 2.0 ** 120
    step = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
    assert torch.equal(got[4:], torch.round(v[4:] / step) * step)
