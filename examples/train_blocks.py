"""Training with the layer operators and the sharded sparse optimizer on one GPU.

A stack of residual feed-forward blocks (RMS norm, linear + gelu, linear), W
data-parallel workers one after the other: each worker's forward pass keeps the
block inputs, and of the activations only 8 bits a value; its backward pass
writes every gradient into the worker's flat bfloat16 vector, and Scape.step()
takes the W vectors.

    python examples/train_blocks.py [--workers 4] [--steps 30] [--hidden 256]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_communication_sharded_gb300 import Scape, layers as L  # noqa: E402

EPS = 1e-5


class Blocks:
    """Shapes, flat layout and passes of the stack.  Parameters are one flat
    float32 vector; a pass takes its bfloat16 copy."""

    def __init__(self, n_blocks, hidden, ffn, out):
        self.n_blocks = n_blocks
        self.shapes = []
        for i in range(n_blocks):
            self.shapes += [(f"norm{i}", (hidden,)), (f"w1_{i}", (ffn, hidden)), (f"b1_{i}", (ffn,)),
                            (f"w2_{i}", (hidden, ffn)), (f"b2_{i}", (hidden,))]
        self.shapes += [("norm", (hidden,)), ("head", (out, hidden)), ("head_b", (out,))]
        self.numel = [math.prod(s) for _, s in self.shapes]

    def views(self, flat):
        """Each parameter's view of a flat vector (parameters or gradients)."""
        parts = torch.split(flat, self.numel)
        return {name: p.view(shape) for (name, shape), p in zip(self.shapes, parts)}

    def init(self, device, seed):
        g = torch.Generator(device=device).manual_seed(seed)
        flat = torch.randn(sum(self.numel), device=device, generator=g) * 0.02
        for name, v in self.views(flat).items():
            if name.startswith("norm"):
                v.fill_(1.0)
            elif "b" in name:
                v.zero_()
        return flat

    def forward(self, p, x):
        """Output and what the backward pass needs: for each block the normed sum
        (bfloat16), its row factors, and two 8-bit checkpoints."""
        kept = []
        delta, stream = x, None
        for i in range(self.n_blocks):
            n = L.add_rmsnorm(delta, p[f"norm{i}"], residual=stream, eps=EPS, pack=True)
            stream = n.h
            hidden, z8 = L.linear(n.y, p[f"w1_{i}"], bias=p[f"b1_{i}"], activation="gelu",
                                  keep_pre=True)
            delta = L.linear(hidden, p[f"w2_{i}"], bias=p[f"b2_{i}"])
            kept.append((n.h, n.rstd, n.y8, z8))
        n = L.add_rmsnorm(delta, p["norm"], residual=stream, eps=EPS, pack=True)
        kept.append((n.h, n.rstd, n.y8, None))
        return L.linear(n.y, p["head"], bias=p["head_b"]), kept

    def backward(self, p, dout, kept, g):
        """Gradients of everything into the views g; returns the input's."""
        h, rstd, y8, _ = kept[-1]
        L.linear_backward_weight(dout, y8, dweight=g["head"], dbias=g["head_b"])
        dy = L.linear_backward_input(dout, p["head"])
        # d: the gradient of the sum, which is that of delta and of the stream
        d = L.add_rmsnorm_backward(dy, h, p["norm"], rstd, dweight=g["norm"])
        for i in reversed(range(self.n_blocks)):
            h, rstd, y8, z8 = kept[i]
            L.linear_backward_weight(d, z8, activation="gelu", dweight=g[f"w2_{i}"], dbias=g[f"b2_{i}"])
            dz = L.linear_backward_input(d, p[f"w2_{i}"], pre=z8, activation="gelu")
            L.linear_backward_weight(dz, y8, dweight=g[f"w1_{i}"], dbias=g[f"b1_{i}"])
            dy = L.linear_backward_input(dz, p[f"w1_{i}"])
            d = L.add_rmsnorm_backward(dy, h, p[f"norm{i}"], rstd, dh=d, dweight=g[f"norm{i}"], out=dy)
        return d


def train(workers=4, steps=30, hidden=256, blocks=3, tokens=512, out=64, sparsity=0.9, lr=2e-3, seed=0,
          device="cuda:0"):
    """Mean squared error against a random teacher; returns the loss of every step."""
    model = Blocks(blocks, hidden, 4 * hidden, out)
    params = model.init(device, seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    teacher = torch.randn(hidden, out, device=device, generator=gen) / hidden ** 0.5
    grads = [torch.empty(params.numel(), dtype=torch.bfloat16, device=device) for _ in range(workers)]
    opt = Scape(params, workers, sparsity, layer_numel=model.numel, lr=lr, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        p = model.views(params.bfloat16())
        total = 0.0
        for w in range(workers):
            x = torch.randn(tokens, hidden, device=device, generator=gen).bfloat16()
            y, kept = model.forward(p, x)
            err = y.float() - torch.tanh(x.float() @ teacher)
            total = total + err.square().mean() / workers
            model.backward(p, (err * (2.0 / err.numel())).bfloat16(), kept, model.views(grads[w]))
        # a product that gave up a wait has left gradients that nobody may use
        if L.status():
            raise RuntimeError("a matrix product did not finish: gradients of this step are incomplete")
        opt.step(grads)
        opt.refresh_mask()
        losses.append(float(total))
    opt.close()
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--workers", type=int, default=4)
    a.add_argument("--steps", type=int, default=30)
    a.add_argument("--hidden", type=int, default=256)
    a = a.parse_args()
    for i, v in enumerate(train(a.workers, a.steps, a.hidden)):
        print(f"step {i:3d}  loss {v:.5f}")
