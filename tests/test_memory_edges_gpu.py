"""Inputs that begin and end where their memory does, with tokens and targets just
outside the vocabulary on both sides: whatever is none or out of range, and whatever
lies beside a row's ends, is not read."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R
from tests.test_embedding_gpu import near as near_rows
from tests.test_logprobs_gpu import near
from tests.test_logprobs_lse_gpu import bounds

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
BYTES = 12 << 20  # torch's allocator gives as much a piece of device memory of its own


def alone(rows, cols, dtype, seed):
    assert rows * cols * torch.finfo(dtype).bits // 8 == BYTES
    torch.cuda.empty_cache()
    t = torch.empty(rows, cols, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    return t.copy_(torch.randn(rows, cols, device="cuda", generator=g) * 2)


def beside(rows, cols, dtype, off):
    """Rows that start off elements into a wider buffer's."""
    return torch.zeros(rows, cols + 8, dtype=dtype, device="cuda")[:, off:off + cols]


@pytest.mark.parametrize("cols", [3, 1 << 12, 1 << 15, 1 << 20])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 3, 7])
def test_logits(cuda_device, cols, dtype, off):
    rows = BYTES // (torch.finfo(dtype).bits // 8) // cols
    x = alone(rows, cols, dtype, cols)
    g = torch.Generator(device="cuda").manual_seed(off)
    dlp, dent = (torch.randn(rows, device="cuda", generator=g) for _ in range(2))
    for i in range(1, 9):
        t = torch.randint(0, cols, (rows,), device="cuda", generator=g)
        t[0], t[-1] = -i, cols + i - 1
        out = beside(rows, cols, dtype, off)
        r = L.token_logprobs(x, t, entropy=True, lse_rest=True, top=min(2, cols) if i == 1 else 0)
        few = torch.tensor(sorted({0, 1, rows // 2, rows - 2, rows - 1}), device="cuda")
        xs, ts, gs, hs = x[few], t[few], dlp[few], dent[few]
        o = R.Rows(xs, ts)
        near(r.logprob[few], *o.logprob(), "log probabilities")
        L.token_logprobs_backward(x, t, r.lse, dlp, r.entropy, dent, out=out, lse_rest=r.lse_rest)
        part = type("Part", (), {"entropy": r.entropy[few]})
        near(out[few], *bounds(xs, ts, gs, dtype, part, hs), "gradient from two numbers")
        L.token_logprobs_backward(x, t, r.lse, dlp, r.entropy, dent, out=out)
        near(out[few], *o.gradient(gs, dtype, r.entropy[few], hs, own_lse=r.lse[few]), "gradient")
        L.token_logprobs_backward(x, t, r.lse, dlp, out=out)
        near(out[few], *o.gradient(gs, dtype, own_lse=r.lse[few]), "gradient without the entropy's")
        L.token_loss(x, t, dlp, out=out)
        near(out[few], *o.gradient(-gs, dtype), "loss")


@pytest.mark.parametrize("cols", [3, 1 << 10, 1 << 17])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 7])
def test_tables_and_their_gradients(cuda_device, cols, dtype, off):
    rows = BYTES // (torch.finfo(dtype).bits // 8) // cols
    w = alone(rows, cols, dtype, cols)
    g = torch.Generator(device="cuda").manual_seed(off)
    t = torch.randint(0, rows, (64,), device="cuda", generator=g)
    t[:6] = torch.tensor([0, rows - 1, -1, rows, -2, rows + 1], device="cuda")
    y = beside(64, cols, dtype, off)
    L.embedding(t, w, out=y)
    near_rows(y, *R.embedding(t, w, 1.0, dtype))
    # the same memory as the gradient of rows that were looked up
    ids = torch.randint(-1, 41, (rows,), device="cuda", generator=g)
    ids[0], ids[-1] = 39, 0
    dw = beside(40, cols, F32, off)
    L.embedding_backward(w, ids, dw)
    near_rows(dw, *R.embedding_backward(w, ids, torch.zeros(40, cols, device="cuda"), 1.0, F32))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [0, 1, 7])
def test_gradients(cuda_device, dtype, off):
    n = BYTES // (torch.finfo(dtype).bits // 8)
    t = alone(1, n, dtype, off).view(-1)
    want, tol = R.norm([t])
    assert abs(float(L.grad_norm([t])) - want) <= tol * want
    for out_type in (BF, F32):
        out = torch.zeros(n + 8, dtype=out_type, device="cuda")[off:off + n]
        assert abs(float(L.clip_grad_norm([t], want / 2, out=[out], eps=0.0)) - want) <= tol * want
        w = t.double() / 2
        assert bool(((out.double() - w).abs() <= w.abs() * (R.U(out_type) + tol + 2 * R.E) * 1.01).all())
