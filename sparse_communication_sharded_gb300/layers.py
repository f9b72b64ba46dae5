"""Training-layer operators over torch tensors (include/scape_layers.h).

The gradients that Scape.step() reads are made with these on the same GPU:
the residual RMS norm, activation checkpoints in 8 bits, and the linear layer
with bias, activation and residual in its epilogue, each with its gradient.
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


def status() -> int:
    """How many waits inside matrix-product kernels on the current device were given
    up since the last call (0: none): the output of a product that gave up is
    incomplete, and its call returned without an error.  Synchronises the current
    stream and answers for the work on it; ask before gradients are used."""
    return _lib().status()
