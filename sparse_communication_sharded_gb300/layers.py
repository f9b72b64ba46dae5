"""Training-layer operators over torch tensors (include/scape_layers.h).

The gradients that Scape.step() reads are made with these on the same GPU:
the residual RMS norm, activation checkpoints in 8 bits, and the linear layer
with bias, activation and residual in its epilogue, each with its gradient; the
embedding and the log probabilities of tokens (or a loss) at a language model's
ends, with theirs; and the gradients' norm and clipping before the step.
Every computation is a kernel of libscape.so; PyTorch provides device memory
and the current stream, on which all work is enqueued.

A tensor of any number of dimensions is taken as rows of its last one: its
last dimension has unit stride and the others collapse to one row stride
(slices of a wider buffer are fine).  Outputs are new contiguous tensors
unless given, and given ones share no memory with what the call reads unless
said.  ValueError: an argument's type, shape, layout or device; ScapeError:
what the library refuses.

Nothing is recorded for autograd: the gradients are operators of their own
(*_backward).  A tensor that requires grad is refused while autograd records
(ValueError); under torch.no_grad() or in an autograd.Function it is taken.
Tensors written in place (out, dweight, dbias) count as modified.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os
from typing import NamedTuple

import torch

from . import build as _build
from ._layers import ACTIVATIONS

BLOCK = 32  # columns that share a scale (SCAPE_PACK_BLOCK)

_binding = None


def _lib():
    """The binding (csrc/layers_torch.cpp); raises if it has not been built, or for
    another torch."""
    global _binding
    if _binding is None:
        if not os.path.exists(_build.BINDING):
            raise ImportError(f"{_build.BINDING} not found: build it with "
                              "`python -m sparse_communication_sharded_gb300.build`")
        why = _build.binding_mismatch()
        if why:
            raise ImportError(f"{_build.BINDING} was {why}: build it again with "
                              "`python -m sparse_communication_sharded_gb300.build`")
        name = "_layers_torch"
        loader = importlib.machinery.ExtensionFileLoader(name, _build.BINDING)
        spec = importlib.util.spec_from_file_location(name, _build.BINDING, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _binding = module
    return _binding


class Packed8(NamedTuple):
    """8-bit values q (float8_e4m3fn) and one scale byte for 32 columns of a
    row: value = q * 2^(scale - 127)."""
    q: torch.Tensor
    scale: torch.Tensor

    @property
    def shape(self):
        return self.q.shape


class NormOutput(NamedTuple):
    """y and its 8-bit form (None unless asked for); h, the normed sum (x itself
    without a residual); rstd, one float32 a row."""
    y: torch.Tensor
    h: torch.Tensor
    rstd: torch.Tensor
    y8: Packed8 | None


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}")
    return act


# ------------------------------------------------------------------ 8-bit checkpoints
def pack8(x: torch.Tensor) -> Packed8:
    """x (float32 or bfloat16) in 8 bits: blocks of 32 columns with a
    power-of-two scale each.  Infinities and NaN become NaN."""
    return Packed8(*_lib().pack8(x))


def unpack8(p: Packed8, dtype=torch.bfloat16, activation=None, out=None) -> torch.Tensor:
    """The values of p, through an activation (None, "relu", "gelu" in its tanh
    form, or "silu").  Without one the result is exact in either dtype, up to
    3.3e38 (a magnitude packed from above that is read as infinity) and, in
    bfloat16, down to its smallest step 2^-133."""
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    return _lib().unpack8(p, dtype is torch.bfloat16, _activation(activation), out)


def activation_grad(dy: torch.Tensor, pre: Packed8, activation, out=None) -> torch.Tensor:
    """dy * activation'(z) for an activation whose input z was kept as `pre`.
    out may be dy."""
    return _lib().activation_grad(dy, pre, _activation(activation), out)


# ------------------------------------------------------------------ residual RMS norm
def add_rmsnorm(x, weight, residual=None, eps=1e-5, pack=False) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last
    dimension.  x, residual, h and y share a dtype (float32 or bfloat16); weight
    is of either.  pack: also y in 8 bits, rounded from the 32-bit y."""
    y, h, rstd, q, scale = _lib().add_rmsnorm(x, weight, residual, eps, pack)
    return NormOutput(y, x if h is None else h, rstd, Packed8(q, scale) if pack else None)


def add_rmsnorm_backward(dy, h, weight, rstd, dh=None, dweight=None, out=None) -> torch.Tensor:
    """The gradient of x (and of residual, the same): dh is the gradient that
    reaches h from elsewhere.  dweight, a vector of float32 or bfloat16 (a slice
    of a flat gradient, say), receives the weight's.  out may be dy or dh."""
    return _lib().add_rmsnorm_backward(dy, h, weight, rstd, dh, dweight, out)


# ------------------------------------------------------------------ linear layer
def linear(x, weight, bias=None, residual=None, activation=None, keep_pre=False, out=None):
    """activation(x weight^T + bias) + residual, bfloat16, weight [n, k].
    keep_pre: returns (y, z8) with z8 the value before the activation in 8 bits.
    out may be residual."""
    r = _lib().linear(x, weight, bias, residual, _activation(activation), keep_pre, out)
    return (r[0], Packed8(r[1], r[2])) if keep_pre else r


def linear_backward_input(dy, weight, pre=None, activation=None, out=None) -> torch.Tensor:
    """dy weight, the gradient of a linear layer's input; with `pre` (and its
    activation) taken on through the activation that made that input from the
    value kept as `pre`."""
    if (pre is None) != (activation is None):
        raise ValueError("pre and activation must be given together")
    return _lib().linear_backward_input(dy, weight, pre, _activation(activation), out)


def linear_backward_weight(dy, x, activation=None, dweight=None, dbias=None, grad_dtype=None):
    """The gradient of a linear layer's weight, dy^T a, for its input a: a
    bfloat16 tensor, or a Packed8 (through an activation).  Written into dweight
    [n, k] (a view of a flat gradient, say; new, of grad_dtype, if None), and the
    bias gradient into dbias [n] if given.  Both float32 or both bfloat16."""
    if activation is not None and not isinstance(x, tuple):
        raise ValueError("an activation is applied to a Packed8 input only")
    if grad_dtype is not None:
        if grad_dtype is not torch.bfloat16 and grad_dtype is not torch.float32:
            raise ValueError("grad_dtype must be torch.float32 or torch.bfloat16")
        if dweight is not None and dweight.dtype is not grad_dtype:
            raise ValueError("dweight is not of grad_dtype")
    return _lib().linear_backward_weight(dy, x, _activation(activation), dweight, dbias,
                                         grad_dtype is torch.float32)


# ------------------------------------------------------------------ tokens
def embedding(tokens, weight, scale=1.0, dtype=None, out=None) -> torch.Tensor:
    """scale * weight[tokens], a row of zeros for a token below 0 (none).  tokens:
    contiguous int64 or int32; weight [vocabulary, columns] and the result float32 or
    bfloat16 each (the result weight's unless dtype or out says otherwise).  A token
    outside the vocabulary gives a row of NaN."""
    if dtype is not None and dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    kind = 0 if dtype is None else 1 if dtype is torch.bfloat16 else 2
    return _lib().embedding(tokens, weight, scale, kind, out)


def embedding_backward(dy, tokens, dweight, scale=1.0, accumulate=False) -> torch.Tensor:
    """The gradient of embedding's weight, written into dweight [vocabulary, columns]
    (a view of a flat gradient, say), which is returned: scale times the sum of dy's
    rows of each token, zeros where there are none.  accumulate: added to what
    dweight holds, for a table that is the output layer's weight as well.  Sums
    are in 32 bits and in the same order in every call; tokens below 0 or outside
    the vocabulary add nothing."""
    return _lib().embedding_backward(dy, tokens, dweight, scale, accumulate)


class _TokenLogprobs(NamedTuple):
    logprob: torch.Tensor
    lse: torch.Tensor
    entropy: torch.Tensor | None
    top_logprob: torch.Tensor | None
    top_token: torch.Tensor | None


class TokenLogprobs(_TokenLogprobs):
    """Each of the rows' leading shape, float32: the targets' log probabilities, the
    logits' log-sum-exp, the entropies (None unless asked for); the `top` largest
    logits' log probabilities and columns (int64), in falling order, in one more
    dimension (None unless asked for).  Beside these five, lse_rest: what lse's rounding
    leaves of the log-sum-exp, for token_logprobs_backward (None unless asked for).  The
    float32 ones are parts of one allocation."""
    lse_rest: torch.Tensor | None = None


def token_logprobs(logits, targets, entropy=False, top=0, lse_rest=False) -> TokenLogprobs:
    """Log probabilities of the targets (contiguous int64 or int32, of the logits'
    leading shape) under softmax(logits), logits float32 or bfloat16.  A target below
    0 stands for none and gives 0; one outside the vocabulary gives NaN.  top: 0 to
    32 (of up to 4194304 columns); of equal logits the lower column comes first.  A
    logit of -infinity has probability 0; in a row of nothing else every log
    probability is -infinity and the entropy 0."""
    values = _lib().token_logprobs(logits, targets, entropy, top, lse_rest)
    if not lse_rest:
        return TokenLogprobs(*values)
    r = TokenLogprobs(*values[:5])
    r.lse_rest = values[5]
    return r


def token_logprobs_backward(logits, targets, lse, dlogprob, entropy=None, dentropy=None,
                            out=None, lse_rest=None) -> torch.Tensor:
    """The gradient of the logits, from that of the log probabilities and, if given,
    that of the entropies (with the entropies themselves).  lse, lse_rest, dlogprob,
    entropy and dentropy: contiguous float32, one a row.  out may be logits.  lse_rest
    is what token_logprobs gives if asked: without it probabilities are off by lse's rounding, 2^-24
    |lse| of themselves, and a target with nearly all of it has no gradient left."""
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropies that token_logprobs gave")
    return _lib().token_logprobs_backward(logits, targets, lse, dlogprob, entropy, dentropy, out, lse_rest)


def token_loss(logits, targets, weight, out=None):
    """(loss, dlogits): each row's -weight * log probability of its target, and the
    gradient of their sum, with the logits read once.  weight: a number, or
    contiguous float32, one a row; 1 / the number of targets makes the sum a mean.  A
    row whose target is below 0 (none) has neither, whatever its logits.  out
    (the gradient) may be logits."""
    if isinstance(weight, torch.Tensor):
        return _lib().token_loss(logits, targets, weight, 0.0, out)
    return _lib().token_loss(logits, targets, None, float(weight), out)


# ------------------------------------------------------------------ gradients
def grad_norm(grads) -> torch.Tensor:
    """sqrt of the sum of all elements' squares over a list of float32 or bfloat16
    tensors on one device, as a float32 scalar there.  A tensor's elements lie
    together in memory, in any order of its dimensions."""
    return _lib().grad_norm(grads)


def clip_grad_norm(grads, max_norm, out=None, eps=1e-6) -> torch.Tensor:
    """Multiplies every tensor by min(1, max_norm / (norm + eps)) and returns the norm
    from before, without waiting for it.  In place, or into the tensors of `out`, of
    the same shapes and strides and of either type: float32 sums over
    several batches go into a worker's flat bfloat16 gradient so."""
    return _lib().clip_grad_norm(grads, max_norm, eps, out)


def status() -> int:
    """How many waits inside matrix-product kernels on the current device were given
    up since the last call (0: none): the output of a product that gave up is
    incomplete, and its call returned without an error.  Synchronises the current
    stream and answers for the work on it; ask before gradients are used."""
    return _lib().status()
