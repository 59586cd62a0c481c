"""Edges of the norms around a block, the gated activation and 8-bit checkpoints: the ends of the types' ranges, masked gates,
gates that are wide open, where memory lies."""
import math

import pytest
import torch

import oracle.blocks as ref
from test_block_ops import DTYPES, F24, check8_exact, close, dev, gen, gpu, mm, norm_inputs  # noqa: F401

FLT_MAX = torch.finfo(torch.float32).max


def bits32(*words):
    return torch.tensor(words, dtype=torch.int32).view(torch.float32)


# the last values below infinity: from 0x7f7f0000 on all have one scale byte
TOP32 = bits32(0x7f7effff, 0x7f7f0000, 0x7f7f0001, 0x7f7f8000, 0x7f7fffff)


def far_ends(dtype):
    """Rows of 300 values whose blocks' largest magnitudes lie at the ends of the type's range, of either sign."""
    lim = torch.finfo(dtype)
    tops = list(TOP32) + list(-TOP32) if dtype == torch.float32 else [torch.tensor(v) for v in (lim.max, lim.min)]
    x = gen(1, 2 * len(tops), 300)
    for i, v in enumerate(tops):
        x[2 * i, 7], x[2 * i, 131], x[2 * i + 1, 299] = v, -v, v
    return x.to(dtype)


# ---------------------------------------------------------------- the ends of the types' ranges

@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_checkpoints_of_the_largest_finite_values(mm, dtype, fmt):
    t = far_ends(dtype)
    one = torch.ones_like(t)
    a = mm.gated_activation(*dev(t, t.flip(1)), checkpoint=fmt)
    check8_exact(a.kept.gate, t, fmt), check8_exact(a.kept.up, t.flip(1), fmt)
    w = torch.ones(300, device="cuda")
    n = mm.block_norm(*dev(one, one), w, w, gate=t.cuda(), checkpoint=fmt)
    check8_exact(n.kept.gate, t, fmt)
    n = mm.block_norm(*dev(t, one), w, w, checkpoint=fmt)
    check8_exact(n.kept.x, t, fmt)
    n = mm.block_norm(*dev(torch.zeros_like(t), t), w, w, checkpoint=fmt)      # the stream alone
    assert torch.equal(n.h.cpu(), t)
    check8_exact(n.kept.h, t, fmt)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_outputs_of_the_largest_finite_values(mm, fmt):
    """8-bit results whose fp32 values lie above 0x7f7f0000, by rows and by columns."""
    big, one = torch.full((5, 300), FLT_MAX), torch.ones(5, 300)
    big[1], big[2, ::2], big[3], big[4] = TOP32[2], -FLT_MAX, TOP32[3], TOP32[1]
    a = mm.gated_activation(*dev(big.abs(), big.sign()), fp8=fmt)               # the gate is open: y = gate up
    assert torch.equal(a.y.cpu(), big)
    check8_exact(a.q, big, fmt)
    kept = mm.GatedKept(*dev(torch.full_like(big, 30.0), one))                  # f' = 1: dgate = dy up
    d = mm.gated_activation_backward(big.cuda(), kept, fp8=fmt)
    check8_exact(d.dgate_rows, d.dgate.cpu(), fmt), check8_exact(d.dgate_cols, d.dgate.cpu().t(), fmt)
    assert bool(torch.isfinite(d.dgate).all()) and float(d.dgate.abs().max()) > TOP32[1]
    kept = mm.GatedKept(*dev(big.abs(), one))                                   # f = gate: dup = dy gate, y = gate
    d = mm.gated_activation_backward(big.sign().cuda(), kept, fp8=fmt, y_fp8=fmt)
    assert torch.equal(d.dup.cpu(), big)
    check8_exact(d.dup_rows, big, fmt), check8_exact(d.dup_cols, big.t(), fmt), check8_exact(d.y_cols, big.abs().t(), fmt)
    for dtype in (torch.bfloat16, torch.float32):                               # products of 16-bit values: 1.99585 2^127
        g, u = torch.full((3, 200), 1.171875 * 2.0 ** 127), torch.full((3, 200), 1.703125)
        for kind in ("silu", "gelu"):
            a = mm.gated_activation(*dev(g.to(dtype), u.to(dtype)), activation=kind, fp8=fmt, y=False)
            check8_exact(a.q, g * u, fmt)
    pre = bits32(0x7f7f4000)                                                    # a row of one column: y = pre, but for eps
    n = mm.block_norm(*dev(torch.zeros(3, 1), torch.ones(3, 1), pre, pre), fp8=fmt)
    assert bool(torch.isfinite(n.y).all()) and float(n.y.min()) > TOP32[1]
    check8_exact(n.q, n.y.cpu(), fmt)
