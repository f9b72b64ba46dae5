"""The operators on tokens, logits and sets of gradients in 64 bits, for the GPU
tests, each with a bound on what a 32-bit computation may be off by.  Shares no code
with the package.

U(t): half a step of type t relative to the value.  E = 2^-24, a rounding in 32 bits.
An exponential 2^a in hardware is off by 2^-22 of itself, and a's roundings (the
difference from the row's largest, its product with log2 e and that constant's own)
by 3 E |d| more.  A thread adds up no more than vocab / 64 + 64 terms in a row, sums
over lanes and blocks included.  Differences may be taken from a number below the row's
largest by ln 1024 at most (a larger term of a sum makes the kernel raise it): B = 7
more in the size of every difference and of the logarithm of their exponentials' sum."""
import math

import torch

E = 2.0 ** -24
B = 7.0


def U(dtype):
    return torch.finfo(dtype).eps / 2


def embedding(tokens, w, scale, dtype):
    """(values, tolerance): one rounding of the product, one to the type."""
    t = tokens.long()
    y = w.double()[t.clamp(0, w.shape[0] - 1)] * scale
    y[t < 0] = 0.0
    y[t >= w.shape[0]] = math.nan
    return y, y.abs() * (U(dtype) + E) + 1e-44


def embedding_backward(dy, tokens, old, scale, dtype):
    """Sums of n rows are off by n roundings of the sum of magnitudes at most; then the
    product, the sum with what was there, and the type."""
    vocab, cols = old.shape
    t = tokens.long().flatten()
    d = dy.double().reshape(-1, cols)
    keep = (t >= 0) & (t < vocab)
    t, d = t[keep], d[keep]
    z = torch.zeros(vocab, cols, dtype=torch.float64, device=dy.device)
    s, m = z.clone().index_add_(0, t, d), z.clone().index_add_(0, t, d.abs())
    n = torch.bincount(t, minlength=vocab)[:, None]
    want = s * scale + old.double()
    tol = want.abs() * U(dtype) + abs(scale) * m * (n + 1) * E + want.abs() * E
    return want, tol + 1e-44


class Rows:
    """Everything about rows of logits x (any float type)."""

    def __init__(self, x, targets):
        self.x = x.double()
        self.t = targets.long()
        rows, self.vocab = self.x.shape
        self.none = self.t < 0
        self.bad = self.t >= self.vocab
        self.empty = (self.x == -math.inf).all(1)
        top = self.x.amax(1)
        self.top = torch.where(self.empty, 0.0, top)
        self.d = self.x - self.top[:, None]
        e = torch.exp(self.d)
        self.s = e.sum(1)
        self.lse = self.top + torch.log(self.s)  # -inf where empty
        self.p = torch.where(self.empty[:, None], 0.0, e / self.s[:, None])
        self.pd = torch.where(self.p > 0, self.p * self.d, 0.0)
        self.ln_s = torch.where(self.empty, 0.0, torch.log(self.s))
        # not x - lse: beside a mask's lowest value even 64 bits lose ln S
        self.logp = self.d - self.ln_s[:, None]
        self.entropy = torch.where(self.empty, 0.0, self.ln_s - self.pd.sum(1))
        # relative error of S
        self.chain = (self.vocab / 64 + 64) * E
        self.ds = self.chain + 2.0 ** -22 + 3 * E * (self.pd.abs().sum(1) + B)
        self.at = (torch.arange(rows, device=x.device), self.t.clamp(0, self.vocab - 1))

    def logprob(self):
        v = self.logp[self.at]
        v = torch.where(self.none, 0.0, torch.where(self.bad, math.nan, v))
        tol = self.ds + 2 * E * (self.d[self.at].abs() + self.ln_s + 2 * B + v.abs())
        return v, torch.where(torch.isfinite(tol), tol, 0.0)

    def lse_and_tol(self):
        return self.lse, torch.where(self.empty, 0.0, self.ds + 2 * E * (self.ln_s + B + self.lse.abs()))

    def entropy_and_tol(self):
        a = torch.where(self.p > 0, self.p * (self.d.abs() + B) * (self.chain + 2.0 ** -22 + 4 * E * (self.d.abs() + B)), 0.0).sum(1)
        mean = self.pd.sum(1).abs()
        return self.entropy, self.ds * (1 + mean + B) + a + 4 * E * (self.ln_s + mean + 2 * B)

    def top_k(self, k):
        """Columns and logits in falling order, equal ones by column."""
        value, place = torch.sort(self.x, dim=1, descending=True, stable=True)
        v = (value[:, :k] - self.top[:, None]) - self.ln_s[:, None]
        tol = self.ds[:, None] + 2 * E * (self.d.gather(1, place[:, :k]).abs() + self.ln_s[:, None] + 2 * B + v.abs())
        return place[:, :k], v, torch.where(torch.isfinite(tol), tol, 0.0)

    def gradient(self, dlogprob, dtype, entropy=None, dentropy=None, own_lse=None):
        """own_lse: the float32 log-sum-exp that the call is given (else its own sums)."""
        logp, p = self.logp, self.p
        off = self.ds[:, None] + 3 * E * (self.d.abs() + B)
        if own_lse is not None:
            # (a number of 4096 or more has too few digits left: own sums then)
            far = (own_lse.abs() > 4096) & ~self.empty
            lse = torch.where(self.empty | far, 0.0, own_lse.double())
            logp = torch.where(far[:, None], logp, self.x - lse[:, None])
            p = torch.exp(logp)
            off = torch.where(far[:, None], off, 2.0 ** -22 + 3 * E * logp.abs())
        g = torch.where(self.none, 0.0, torch.where(self.bad, math.nan, dlogprob.double()))[:, None]
        one = torch.zeros_like(p)
        one[self.at] = torch.where(self.none, 0.0, 1.0).to(p.dtype)
        # 1 - p at the target without a difference
        left = torch.where(one > 0, -torch.expm1(logp), -p)
        dx = g * torch.where(one > 0, left, -p)
        rel = torch.where(p > 0, off + 3 * E, 0.0)
        tol = (g.abs() * (p * rel + (one > 0) * left.abs() * 4 * E))
        if dentropy is not None:
            h = dentropy.double()[:, None]
            lh = torch.where(p > 0, logp + entropy.double()[:, None], 0.0)
            dx = dx - h * p * lh
            size = torch.where(p > 0, logp.abs() + entropy.double().abs()[:, None], 0.0)
            tol = tol + h.abs() * p * size * (torch.where(p > 0, off, 0.0) + 5 * E)
        # 2^a below 2^-126 is 0, and its product's roundings there
        tiny = 2.0 ** -120 * (1 + g.abs() + (0 if dentropy is None else dentropy.double().abs()[:, None] * 256))
        return dx, tol + dx.abs() * U(dtype) + tiny


def norm(grads):
    """(norm, relative tolerance): no more than 32 roundings in a short sum of squares
    and the joining of eight, half of that in the root, and one to 32 bits."""
    s = sum(float(g.double().square().sum()) for g in grads if g.numel())
    return math.sqrt(s), 24 * E
