"""README.md's lines on tokens, logits and gradients, run as they stand there: what the
scoring gives belongs to the logits, not to what a call has put in their place."""
import os
import re

import pytest
import torch

from sparse_communication_sharded_gb300 import layers as L
from tests import _tokens_oracle as R
from tests.test_logprobs_gpu import near

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def code(word):
    """The indented lines of each paragraph that has the word, in their order."""
    with open(README) as f:
        text = f.read()
    found = [p for p in re.findall(r"(?:^    .*\n)+", text, re.M) if word in p]
    assert found
    return "\n".join(re.sub(r"^    ", "", p, flags=re.M) for p in found)


def test_tokens_logits_and_gradients(cuda_device):
    g = torch.Generator(device="cuda").manual_seed(1)
    n, vocab, hidden = 50, 301, 64
    table = torch.randn(vocab, hidden, device="cuda", generator=g).bfloat16()
    tokens = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    targets = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    logits0 = (torch.randn(n, vocab, device="cuda", generator=g) * 3).bfloat16()
    dlogprob, dentropy = (torch.randn(n, device="cuda", generator=g) for _ in range(2))
    flat = torch.zeros(vocab * hidden, device="cuda")
    s = dict(torch=torch, L=L, tokens=tokens, targets=targets, table=table, hidden=hidden, count=n,
             blocks=lambda x: (logits0.clone(), None), blocks_backward=lambda d, kept: d[:, :hidden].contiguous(),
             g_flat=flat, g_table=flat.view(vocab, hidden), dlogprob=dlogprob, dentropy=dentropy)
    exec(code("L.token_l"), s)
    o = R.Rows(logits0, targets)
    near(s["r"].logprob, *o.logprob(), "log probabilities")
    near(s["r"].entropy, *o.entropy_and_tol(), "entropies")
    assert torch.equal(s["r"].top_token, o.top_k(5)[0])
    assert torch.equal(s["d"], L.token_logprobs_backward(logits0, targets, s["r"].lse, dlogprob, s["r"].entropy, dentropy,
                                                         lse_rest=s["r"].lse_rest))
    lp, tol = o.logprob()
    near(s["loss"], -lp / n, tol / n + lp.abs() / n * 2 * R.E, "loss")
