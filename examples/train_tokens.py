"""A small language model trained with the layer operators and the sharded sparse
optimizer on one GPU.

Tokens go in through a table that is the output layer's weight as well, through
the residual feed-forward blocks of train_blocks.py, and out as logits, whose loss
and gradient are one call; the table's gradient is the output layer's with the
lookup's added.  Every worker's flat gradient is clipped by its norm before
Scape.step() takes it.  The text is made up: a word's successor is mostly fixed.

    python examples/train_tokens.py [--workers 4] [--steps 30] [--hidden 256] [--vocab 1000]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from sparse_communication_sharded_gb300 import Scape, layers as L  # noqa: E402
from train_blocks import Blocks  # noqa: E402


class TokenModel(Blocks):
    """Blocks whose output layer's weight is the embedding table too."""

    def __init__(self, n_blocks, hidden, ffn, vocab):
        super().__init__(n_blocks, hidden, ffn, vocab)
        self.scale = hidden ** 0.5

    def logits(self, p, tokens):
        return self.forward(p, L.embedding(tokens, p["head"], scale=self.scale))

    def loss_and_gradients(self, p, tokens, targets, weight, g):
        """Every position's loss; gradients of their sum into the views g."""
        logits, kept = self.logits(p, tokens)
        loss, dlogits = L.token_loss(logits, targets, weight, out=logits)
        dx = self.backward(p, dlogits, kept, g)
        L.embedding_backward(dx, tokens, g["head"], scale=self.scale, accumulate=True)
        return loss


def text(gen, count, vocab, device):
    """Tokens and their successors: 7 in 8 follow from the token, the others are any;
    every 16th position has none (an end)."""
    tokens = torch.randint(0, vocab, (count,), device=device, generator=gen)
    after = (tokens * 5 + 3) % vocab
    other = torch.randint(0, vocab, (count,), device=device, generator=gen)
    targets = torch.where(torch.rand(count, device=device, generator=gen) < 0.125, other, after)
    targets[15::16] = -1
    return tokens, targets


def train(workers=4, steps=30, hidden=256, blocks=2, tokens=512, vocab=1000, sparsity=0.9, lr=2e-3, max_norm=1.0,
          seed=0, device="cuda:0"):
    """Returns (mean loss, the workers' largest gradient norm) of every step, for how much
    of the last batch the usual successor is the likeliest, and the mean entropy."""
    model = TokenModel(blocks, hidden, 4 * hidden, vocab)
    params = model.init(device, seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    grads = [torch.empty(params.numel(), dtype=torch.bfloat16, device=device) for _ in range(workers)]
    opt = Scape(params, workers, sparsity, layer_numel=model.numel, lr=lr, weight_decay=0.0)
    log = []
    for _ in range(steps):
        p = model.views(params.bfloat16())
        total, norms = 0.0, []
        for w in range(workers):
            ids, targets = text(gen, tokens, vocab, device)
            weight = 1.0 / (tokens - tokens // 16)  # of the positions that have a target
            loss = model.loss_and_gradients(p, ids, targets, weight, model.views(grads[w]))
            total = total + loss.sum() / workers
            norms.append(L.clip_grad_norm([grads[w]], max_norm))
        # a product that gave up a wait has left gradients that nobody may use
        if L.status():
            raise RuntimeError("a matrix product did not finish: gradients of this step are incomplete")
        opt.step(grads)
        opt.refresh_mask()
        log.append((float(total), float(torch.stack(norms).max())))
    opt.close()
    r = L.token_logprobs(model.logits(model.views(params.bfloat16()), ids)[0], (ids * 5 + 3) % vocab, entropy=True, top=1)
    hits = float((r.top_token[:, 0] == (ids * 5 + 3) % vocab).float().mean())
    return log, hits, float(r.entropy.mean())


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--workers", type=int, default=4)
    a.add_argument("--steps", type=int, default=30)
    a.add_argument("--hidden", type=int, default=256)
    a.add_argument("--vocab", type=int, default=1000)
    a = a.parse_args()
    log, hits, entropy = train(a.workers, a.steps, a.hidden, vocab=a.vocab)
    for i, (loss, norm) in enumerate(log):
        print(f"step {i:3d}  loss {loss:.4f}  largest gradient norm {norm:.3f}")
    print(f"successor found for {100 * hits:.1f}% of the last batch, mean entropy {entropy:.3f}")
