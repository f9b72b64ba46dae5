"""Calls of the embedding's gradient whose tokens the call before them has just
written: its kernels start before that call's have ended, and have to see all of it."""
import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,vocab,cols", [(20000, 520, 16), (3000, 2600, 40), (64, 131072, 8)])
def test_tokens_from_the_call_before(cuda_device, rows, vocab, cols):
    """The likeliest tokens of changing logits at one address, which token_logprobs
    writes over and over at one place.  Whole numbers' sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    logits = [torch.randn(rows, vocab, device="cuda", generator=g).bfloat16() for _ in range(3)]
    x = torch.empty_like(logits[0])
    targets = torch.zeros(rows, dtype=torch.int64, device="cuda")
    dy = torch.randint(-4, 5, (rows, cols), device="cuda", generator=g).float()
    want = []
    for v in logits:
        w = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda")
        first = torch.where(v == v.amax(1, keepdim=True), torch.arange(vocab, device="cuda"), vocab).amin(1)
        want.append(w.index_add_(0, first, dy.double()))
    dw = [torch.empty(vocab, cols, device="cuda") for _ in range(12)]
    torch.cuda.synchronize()
    for i in range(12):
        x.copy_(logits[i % 3])
        token = L.token_logprobs(x, targets, top=1).top_token[:, 0]
        L.embedding_backward(dy, token, dw[i])
        del token  # its place is the next call's
    torch.cuda.synchronize()
    for i in range(12):
        assert torch.equal(dw[i].double(), want[i % 3]), i
