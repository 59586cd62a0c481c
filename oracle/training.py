"""The operators around the update in 64 bits on the CPU, from their definitions (plain and slow; torch for storage)."""
import torch

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
# fraction bits, smallest normal exponent
SHAPE8 = {"e4m3": (3, -6), "e5m2": (2, -14)}


def clip_grads(grads, max_norm, eps=1e-6):
    """(norm, clipped) of a list of tensors."""
    norm = sum(float((g.double() ** 2).sum()) for g in grads) ** 0.5
    coef = max_norm / (norm + eps)
    coef = min(1.0, coef) if coef == coef else coef
    return norm, [g.double() * coef for g in grads]


def rms_norm(x, weight=None, residual=None, eps=1e-6):
    """(y, h, rstd) over the last dimension, unrounded."""
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = ((h * h).mean(dim=-1) + eps) ** -0.5
    y = h * rstd[..., None]
    return (y if weight is None else y * weight.double()), h, rstd


def rms_norm_backward(dy, h, weight, rstd, dresidual=None):
    """(dx, dweight) of y = h rstd(h) weight for 2-D dy, with rstd as given."""
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    g = dy if weight is None else dy * weight.double()
    dx = r * g - h * r ** 3 * (g * h).mean(dim=1, keepdim=True)
    if dresidual is not None:
        dx = dx + dresidual.double()
    return dx, (dy * h * r).sum(dim=0)


def round8(v, fmt):
    """v (finite, at most the largest value of fmt) to the nearest value of fmt, ties to even."""
    bits, low = SHAPE8[fmt]
    _, p = torch.frexp(v)
    step = 2.0 ** (torch.clamp(p - 1, min=low) - bits).double()
    return torch.round(v / step) * step


def exponent8(amax, fmt):
    """The smallest whole e >= -127 with amax <= top * 2^e (0 for amax = 0), by search."""
    e = torch.full(amax.shape, -127, dtype=torch.int64)
    for k in range(-127, 128):
        e = torch.where(amax > TOP[fmt] * 2.0 ** k, k + 1, e)
    return torch.where(amax == 0, 0, e)


def quantize(x, fmt, square=False):
    """(data, exponents): 8-bit values as float64 [rows, cols] and the exponents [rows, ceil(cols / 128)]."""
    x = x.double()
    rows, cols = x.shape
    down = 128 if square else 1
    blocks = -(-cols // 128)
    amax = torch.zeros(rows, blocks, dtype=torch.float64)
    for r0 in range(0, rows, down):
        for kb in range(blocks):
            amax[r0:r0 + down, kb] = x[r0:r0 + down, kb * 128:(kb + 1) * 128].abs().max()
    exps = exponent8(amax, fmt)
    wide = exps.repeat_interleave(128, dim=1)[:, :cols].double()
    return round8(x / 2.0 ** wide, fmt), exps


def values(data, scale_bytes):
    """What 8-bit data (any float8 tensor) with kept scale bytes [groups, rows4, 4] stands for."""
    rows, cols = data.shape
    kb = torch.arange(cols) // 128
    s = scale_bytes[kb // 4, :rows, kb % 4].double().t()
    return data.float().double() * torch.where(s == 255, torch.nan, 2.0 ** (s - 127))


def matmul(a, b, add=None):
    c = a.double() @ b.double().t()
    return c if add is None else c + add.double()
