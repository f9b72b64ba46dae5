"""Training-layer operators over torch tensors (include/scape_layers.h).

The gradients that Scape.step() reads are made with these on the same GPU:
the residual RMS norm, activation checkpoints in 8 bits, and the linear layer
with bias, activation and residual in its epilogue, each with its gradient.
Every computation is a kernel of libscape.so; PyTorch provides device memory
and the current stream, on which all work is enqueued.

A tensor of any number of dimensions is taken as rows of its last one: its
last dimension has unit stride and the others collapse to one row stride
(slices of a wider buffer are fine).  Outputs are new contiguous tensors
unless given.  ValueError: an argument's type, shape, layout or device;
ScapeError: what the library refuses.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _scape as C
from ._layers import ACTIVATIONS

BLOCK = 32  # columns that share a scale (SCAPE_PACK_BLOCK)

_DTYPES = {torch.float32: C.SCAPE_F32, torch.bfloat16: C.SCAPE_BF16}
_E4M3 = torch.float8_e4m3fn


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


def _call(fn, dev, *args):
    """One library call on `dev` and its current stream."""
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if rc != C.SCAPE_OK:
        raise C.ScapeError(rc, C.load().scape_layer_last_error().decode())


def _workspace(fn, dev, *args):
    n = ctypes.c_size_t()
    rc = fn(*args, ctypes.byref(n))
    if rc != C.SCAPE_OK:
        raise C.ScapeError(rc, C.load().scape_layer_last_error().decode())
    if n.value == 0:
        return None, 0, None
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    return ws.data_ptr(), n.value, ws


def _rows(t, name, dtypes, shape=None, device=None):
    """(rows, columns, row stride) of a tensor seen as a matrix."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, not one of {list(dtypes)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    nd = t.dim()
    if nd == 0:
        raise ValueError(f"{name} has no dimension")
    cols = t.shape[-1]
    if nd == 2:
        rows, ld = t.shape[0], t.stride(0)
    elif t.is_contiguous():
        rows, ld = (t.numel() // cols if cols else 0), cols
    else:
        rows, ld = _collapse(t, name)
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")
    if rows <= 1 or cols == 0:
        ld = max(ld, cols)
    elif ld < cols:
        raise ValueError(f"{name} has overlapping rows")
    return rows, cols, ld


def _collapse(t, name):
    """Rows and row stride of a strided tensor of more than two dimensions, whose
    leading dimensions must step through memory as one."""
    rows, ld = 1, None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise ValueError(f"{name}: the leading dimensions do not collapse to one row stride")
        rows *= n
    return rows, t.shape[-1] if ld is None else ld


def _vector(t, name, dtypes, n, device):
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor on {device} of one of {list(dtypes)}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    return t.data_ptr()


def _packed(p, name, shape, device):
    """(q pointer, row stride, scale pointer)."""
    if not isinstance(p, Packed8):
        raise ValueError(f"{name} must be a Packed8")
    _, cols, ld = _rows(p.q, f"{name}.q", (_E4M3,), shape, device)
    want = (*p.q.shape[:-1], -(-cols // BLOCK))
    s = p.scale
    if s.dtype != torch.uint8 or s.device != p.q.device or s.shape != want or not s.is_contiguous():
        raise ValueError(f"{name}.scale must be a contiguous uint8 tensor of shape {want}")
    return p.q.data_ptr(), ld, s.data_ptr()


def _new_packed(shape, device):
    return Packed8(torch.empty(shape, dtype=_E4M3, device=device),
                   torch.empty((*shape[:-1], -(-shape[-1] // BLOCK)), dtype=torch.uint8,
                               device=device))


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}") from None


def _output(out, name, shape, dtype, device):
    """The given output (checked) or a new one, and its row stride."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device), shape[-1]
    return out, _rows(out, name, (dtype,), shape, device)[2]


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ 8-bit checkpoints
def pack8(x: torch.Tensor) -> Packed8:
    """x (float32 or bfloat16) in 8 bits: blocks of 32 columns with a
    power-of-two scale each.  Infinities and NaN become NaN."""
    rows, cols, ld = _rows(x, "x", _DTYPES)
    p = _new_packed(x.shape, x.device)
    _call(C.load().scape_layer_pack8, x.device, x.data_ptr(), ld, _DTYPES[x.dtype], rows, cols,
          p.q.data_ptr(), cols, p.scale.data_ptr())
    return p


def unpack8(p: Packed8, dtype=torch.bfloat16, activation=None, out=None) -> torch.Tensor:
    """The values of p, through an activation (None, "relu", "gelu" in its tanh
    form, or "silu").  Without one the result is exact in either dtype."""
    act = _activation(activation)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be torch.float32 or torch.bfloat16")
    q, ldq, scale = _packed(p, "p", None, None)
    rows, cols, _ = _rows(p.q, "p.q", (_E4M3,))
    out, ldo = _output(out, "out", p.q.shape, dtype, p.q.device)
    _call(C.load().scape_layer_unpack8, p.q.device, q, ldq, scale, rows, cols, act,
          out.data_ptr(), ldo, _DTYPES[dtype])
    return out


def activation_grad(dy: torch.Tensor, pre: Packed8, activation, out=None) -> torch.Tensor:
    """dy * activation'(z) for an activation whose input z was kept as `pre`.
    out may be dy."""
    act = _activation(activation)
    rows, cols, ld = _rows(dy, "dy", _DTYPES)
    q, ldq, scale = _packed(pre, "pre", dy.shape, dy.device)
    out, ldo = _output(out, "out", dy.shape, dy.dtype, dy.device)
    _call(C.load().scape_layer_act_grad, dy.device, dy.data_ptr(), ld, q, ldq, scale, rows, cols,
          act, out.data_ptr(), ldo, _DTYPES[dy.dtype])
    return out


# ------------------------------------------------------------------ residual RMS norm
def add_rmsnorm(x, weight, residual=None, eps=1e-5, pack=False) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight over the last
    dimension.  x, residual, h and y share a dtype (float32 or bfloat16); weight
    is of either.  pack: also y in 8 bits, rounded from the 32-bit y."""
    rows, cols, ldx = _rows(x, "x", _DTYPES)
    dev = x.device
    w = _vector(weight, "weight", _DTYPES, cols, dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    h, ldr = x, cols
    if residual is not None:
        _, _, ldr = _rows(residual, "residual", (x.dtype,), x.shape, dev)
        h = torch.empty(x.shape, dtype=x.dtype, device=dev)
    p = _new_packed(x.shape, dev) if pack else None
    _call(C.load().scape_layer_add_rmsnorm, dev, x.data_ptr(), ldx, _ptr(residual), ldr, w,
          _DTYPES[weight.dtype], rows, cols, eps, _DTYPES[x.dtype], y.data_ptr(), cols,
          None if residual is None else h.data_ptr(), cols, rstd.data_ptr(),
          p.q.data_ptr() if p else None, cols, p.scale.data_ptr() if p else None)
    return NormOutput(y, h, rstd, p)


def add_rmsnorm_backward(dy, h, weight, rstd, dh=None, dweight=None, out=None) -> torch.Tensor:
    """The gradient of x (and of residual, the same): dh is the gradient that
    reaches h from elsewhere.  dweight, a vector of float32 or bfloat16 (a slice
    of a flat gradient, say), receives the weight's.  out may be dy or dh."""
    rows, cols, ldy = _rows(dy, "dy", _DTYPES)
    dev, dt = dy.device, _DTYPES[dy.dtype]
    _, _, ldh = _rows(h, "h", (dy.dtype,), dy.shape, dev)
    w = _vector(weight, "weight", _DTYPES, cols, dev)
    if rstd.dtype != torch.float32 or rstd.device != dev or rstd.numel() != rows or not rstd.is_contiguous():
        raise ValueError(f"rstd must be a contiguous float32 tensor of {rows} elements")
    ldd = _rows(dh, "dh", (dy.dtype,), dy.shape, dev)[2] if dh is not None else cols
    out, ldo = _output(out, "out", dy.shape, dy.dtype, dev)
    lib = C.load()
    ws = (None, 0, None)
    if dweight is not None:
        _vector(dweight, "dweight", _DTYPES, cols, dev)
        ws = _workspace(lib.scape_layer_add_rmsnorm_bwd_workspace, dev, rows, cols)
    _call(lib.scape_layer_add_rmsnorm_bwd, dev, dy.data_ptr(), ldy, h.data_ptr(), ldh, w,
          _DTYPES[weight.dtype], rstd.data_ptr(), _ptr(dh), ldd, rows, cols, dt, out.data_ptr(),
          ldo, _ptr(dweight), C.SCAPE_F32 if dweight is None else _DTYPES[dweight.dtype], ws[0],
          ws[1])
    return out


# ------------------------------------------------------------------ linear layer
_BF16 = (torch.bfloat16,)


def _weight(weight, device):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a matrix")
    return _rows(weight, "weight", _BF16, None, device)


def linear(x, weight, bias=None, residual=None, activation=None, keep_pre=False, out=None):
    """activation(x weight^T + bias) + residual, bfloat16, weight [n, k].
    keep_pre: returns (y, z8) with z8 the value before the activation in 8 bits.
    out may be residual."""
    act = _activation(activation)
    rows, k, ldx = _rows(x, "x", _BF16)
    dev = x.device
    n, kw, ldw = _weight(weight, dev)
    if kw != k:
        raise ValueError(f"weight has {kw} columns, x has {k}")
    shape = (*x.shape[:-1], n)
    b = None if bias is None else _vector(bias, "bias", _BF16, n, dev)
    ldr = n if residual is None else _rows(residual, "residual", _BF16, shape, dev)[2]
    out, ldo = _output(out, "out", shape, torch.bfloat16, dev)
    p = _new_packed(shape, dev) if keep_pre else None
    lib = C.load()
    xp, wp = x.data_ptr(), weight.data_ptr()
    ws = _workspace(lib.scape_layer_linear_workspace, dev, xp, ldx, wp, ldw, rows, k, n)
    _call(lib.scape_layer_linear, dev, xp, ldx, wp, ldw, b, _ptr(residual), ldr, rows, k, n, act,
          out.data_ptr(), ldo, p.q.data_ptr() if p else None, n,
          p.scale.data_ptr() if p else None, ws[0], ws[1])
    return (out, p) if keep_pre else out


def linear_backward_input(dy, weight, pre=None, activation=None, out=None) -> torch.Tensor:
    """dy weight, the gradient of a linear layer's input; with `pre` (and its
    activation) taken on through the activation that made that input from the
    value kept as `pre`."""
    act = _activation(activation)
    if (pre is None) != (act == 0):
        raise ValueError("pre and activation must be given together")
    rows, n, ldy = _rows(dy, "dy", _BF16)
    dev = dy.device
    nw, k, ldw = _weight(weight, dev)
    if nw != n:
        raise ValueError(f"weight has {nw} rows, dy has {n} columns")
    shape = (*dy.shape[:-1], k)
    q, ldq, scale = (None, k, None) if pre is None else _packed(pre, "pre", shape, dev)
    out, ldo = _output(out, "out", shape, torch.bfloat16, dev)
    lib = C.load()
    dp, wp = dy.data_ptr(), weight.data_ptr()
    ws = _workspace(lib.scape_layer_linear_bwd_input_workspace, dev, dp, ldy, wp, ldw, rows, k, n)
    _call(lib.scape_layer_linear_bwd_input, dev, dp, ldy, wp, ldw, q, ldq, scale, act, rows, k, n,
          out.data_ptr(), ldo, ws[0], ws[1])
    return out


def linear_backward_weight(dy, x, activation=None, dweight=None, dbias=None, grad_dtype=None):
    """The gradient of a linear layer's weight, dy^T a, for its input a: a
    bfloat16 tensor, or a Packed8 (through an activation).  Written into dweight
    [n, k] (a view of a flat gradient, say; new, of grad_dtype, if None), and the
    bias gradient into dbias [n] if given.  Both float32 or both bfloat16."""
    act = _activation(activation)
    rows, n, ldy = _rows(dy, "dy", _BF16)
    dev = dy.device
    packed = isinstance(x, Packed8)
    k = x.shape[-1] if packed or isinstance(x, torch.Tensor) and x.dim() else 0
    shape = (*dy.shape[:-1], k)
    xp, ldx, q, ldq, scale = None, k, None, k, None
    if packed:
        q, ldq, scale = _packed(x, "x", shape, dev)
    else:
        if act:
            raise ValueError("an activation is applied to a Packed8 input only")
        ldx = _rows(x, "x", _BF16, shape, dev)[2]
        xp = x.data_ptr()
    if dweight is None:
        dweight = torch.empty((n, k), dtype=grad_dtype or torch.bfloat16, device=dev)
    elif grad_dtype is not None and dweight.dtype != grad_dtype:
        raise ValueError("dweight is not of grad_dtype")
    ldw = _rows(dweight, "dweight", _DTYPES, (n, k), dev)[2]
    db = None if dbias is None else _vector(dbias, "dbias", (dweight.dtype,), n, dev)
    lib = C.load()
    dp = dy.data_ptr()
    ws = _workspace(lib.scape_layer_linear_bwd_weight_workspace, dev, dp, ldy, xp, ldx, rows, k, n)
    _call(lib.scape_layer_linear_bwd_weight, dev, dp, ldy, xp, ldx, q, ldq, scale, act, rows, k,
          n, dweight.data_ptr(), ldw, db, _DTYPES[dweight.dtype], ws[0], ws[1])
    return dweight


def status() -> int:
    """Nonzero if a matrix-product kernel on the current device gave up a wait
    since the last call (its output is then incomplete).  Synchronises the
    current stream."""
    v = ctypes.c_int()
    rc = C.load().scape_layer_status(ctypes.byref(v), torch.cuda.current_stream().cuda_stream)
    if rc != C.SCAPE_OK:
        raise C.ScapeError(rc, C.load().scape_layer_last_error().decode())
    return v.value
