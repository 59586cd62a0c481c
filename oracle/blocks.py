"""The norms around a block and the gated activation in 64 bits on the CPU, from their definitions (plain and slow)."""
import math

import torch


def block_norm(x, residual, post, pre, gate=None, scale=None, alpha=1.0, eps=1e-6):
    """(y, h, rstd_x, rstd_h), unrounded, of rows x [rows, cols]."""
    x, post, pre = x.double(), post.double(), pre.double()
    rx = ((x * x).mean(dim=1) + eps) ** -0.5
    v = x * rx[:, None] * post
    if scale is not None:
        v = v * scale.double()
    if gate is not None:
        v = v * torch.sigmoid(gate.double())
    h = alpha * residual.double() + v
    rh = ((h * h).mean(dim=1) + eps) ** -0.5
    return h * rh[:, None] * pre, h, rx, rh


def block_norm_backward(dy, x, h, rx, rh, post, pre, gate=None, scale=None, alpha=1.0, dh=None):
    """(dx, dresidual, dgate, dpost, dpre, dscale) with x, h, rx and rh as given."""
    dy, x, h, post, pre = dy.double(), x.double(), h.double(), post.double(), pre.double()
    rx, rh = rx.double()[:, None], rh.double()[:, None]
    scale_ = torch.ones_like(post) if scale is None else scale.double()
    sig = torch.ones(x.shape[0], 1, dtype=torch.float64) if gate is None else torch.sigmoid(gate.double())
    a = dy * pre
    stream = rh * a - h * rh ** 3 * (a * h).mean(dim=1, keepdim=True)
    if dh is not None:
        stream = stream + dh.double()
    t = stream * sig
    b = t * post * scale_
    dx = rx * b - x * rx ** 3 * (b * x).mean(dim=1, keepdim=True)
    dgate = None
    if gate is not None:
        dgate = stream * post * scale_ * x * rx * sig * torch.sigmoid(-gate.double())
        dgate = dgate.sum(dim=1, keepdim=True) if gate.shape[1] != x.shape[1] else dgate
    s = (t * x * rx).sum(dim=0)
    return dx, alpha * stream, dgate, s * scale_, (dy * h * rh).sum(dim=0), None if scale is None else s * post


def activation(g, kind):
    """(f(g), f'(g))."""
    g = g.double()
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    phi = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def gated(gate, up, kind="silu"):
    return activation(gate, kind)[0] * up.double()


def gated_backward(dy, gate, up, kind="silu"):
    """(dgate, dup, y)."""
    f, slope = activation(gate, kind)
    return dy.double() * up.double() * slope, dy.double() * f, f * up.double()
