"""The training-layer operators in 64 bits, for the GPU tests: plain formulas on
double tensors, and the 8-bit block format from its definition.  Shares no code
with the package."""
import math

import torch

BLOCK = 32
EPS64 = 2.0 ** -52
U_BF16 = 2.0 ** -8     # largest relative error of one rounding to bfloat16
U_F32 = 2.0 ** -24


def u_of(dtype):
    return U_BF16 if dtype == torch.bfloat16 else U_F32


def blocks(x):
    rows, cols = x.shape
    p = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=x.dtype, device=x.device)
    p[:, :cols] = x
    return p.view(rows, -1, BLOCK)


def pack8(x):
    """(values, codes) of a double matrix: the least code >= 1 whose scale takes
    the largest finite magnitude to 448 or less; nearest e4m3, ties to even;
    infinities and NaN become NaN."""
    rows, cols = x.shape
    b = blocks(x)
    fin = torch.isfinite(b)
    top = torch.where(fin, b.abs(), 0.0).amax(-1)
    code = torch.ones_like(top)
    # 448 * 2^(code - 127) >= top: count the codes that are too small
    m, e = torch.frexp(top)                      # top = m 2^e, m in [0.5, 1)
    least = torch.where(m <= 0.875, e - 9, e - 8)  # 448 = 0.875 * 2^9
    code = torch.where(top > 0, (least + 127).clamp_min(1).double(), code)
    s = torch.exp2(code - 127)[..., None]
    t = b / s
    _, te = torch.frexp(torch.where(fin, t, 0.0))
    step = torch.exp2((te - 4).clamp_min(-9).double())
    v = torch.where(fin, torch.round(t / step) * step * s, math.nan)
    return v.view(rows, -1)[:, :cols], code.to(torch.uint8)


def values(q, code):
    """Values of e4m3 bytes q (uint8) and scale codes."""
    b = q.long()
    ex, fr = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(ex == 0, fr * 2.0 ** -9, (1 + fr / 8) * torch.exp2((ex - 7).double()))
    mag = torch.where((b & 127) == 127, math.nan, mag)
    col = torch.arange(q.shape[1], device=q.device) // BLOCK
    return torch.where(b >= 128, -mag, mag) * torch.exp2(code.double() - 127)[:, col]


def pack_error(x):
    """Bound on |value - x|: half a step of e4m3, which is 2^-4 of a value's own
    magnitude or, below 2^-6 scales, 2^-10 scales; a scale is at most the
    block's largest magnitude / 224 (or the smallest scale, 2^-126)."""
    rows, cols = x.shape
    top = blocks(x).abs().amax(-1)
    s = (top / 224).clamp_min(2.0 ** -126).repeat_interleave(BLOCK, dim=1)[:, :cols]
    return x.abs() * 2.0 ** -4 + s * 2.0 ** -10


def act(z, name):
    if name is None:
        return z
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z * torch.sigmoid(z)
    # (1 + tanh u) / 2 is the logistic of 2u, which keeps its digits where it is small
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def slope(z, name):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    du = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * du


# The kernels take the logistic function from the hardware's exponential and
# division, whose documented errors are 2 + floor(|1.16 a|) ulp and 2 ulp; past
# |a| = 24 the result is within 2^-34 of 0 or 1.  A relative 2^-18 covers it
# (30 ulp of 2^-23), and the slope has two such terms of size 1.2 at most.
ACT_REL = 2.0 ** -18


def rms(x, w, eps, res=None):
    h = x if res is None else x + res
    rstd = (h.pow(2).mean(1) + eps).pow(-0.5)
    return h * rstd[:, None] * w, h, rstd


def rms_backward(dy, h, w, rstd, dh=None):
    r = rstd[:, None]
    d, n = dy * w, h * r
    dx = r * (d - n * (d * n).mean(1, keepdim=True))
    return dx if dh is None else dx + dh, (dy * n).sum(0)
