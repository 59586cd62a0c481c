"""The operators of a residual network's block and its 8-bit checkpoints (argument checks and marshalling; the work runs
in the library's kernels): the norms behind a block and before the next one with the block's gate and scale, the gated
activation within it, and the transposition of 8-bit matrices.  A block of a training step with 8-bit products, whose
backward pass reads 8-bit copies alone:

    u, v = fp8_matmul(q, Wg_rows), fp8_matmul(q, Wu_rows)            # q: the block's input in 8 bits, kept
    a = gated_activation(u, v, fp8="e4m3", y=False, checkpoint="e4m3")
    x = fp8_matmul(a.q, Wd_rows)
    r = block_norm(x, stream, w_post, w_pre, gate=g, scale=s, fp8="e4m3", y=False, checkpoint="e4m3")
                                                                     # r.h: the new stream, r.q: the next block's input

    g = block_norm_backward(dy, r.kept, w_post, w_pre, scale=s, dh=dstream)
    d, dt = fp8_quantize(g.dx, "e5m2", cols=True)
    b = gated_activation_backward(fp8_matmul(d, Wd_cols), a.kept, fp8="e5m2", dense=False, y_fp8="e4m3")
    dWd = fp8_matmul(dt, b.y_cols)
    qt = fp8_transpose(q)
    dWg, dWu = fp8_matmul(b.dgate_cols, qt), fp8_matmul(b.dup_cols, qt)
    dy = fp8_matmul(b.dup_rows, Wu_cols, add=fp8_matmul(b.dgate_rows, Wg_cols))

What the calls of training.py say of autograd and of `stream=` holds for these too.
"""
from __future__ import annotations

import struct
from typing import NamedTuple, Optional, Union

import torch

from . import binding as _b
from .training import _FMT, _TYPE_FMT, Fp8Tensor, _dt, _fmt_code, _like, _on, _rows

_ACT = {"silu": 0, "gelu": 1}
_NONE8 = (0, 0, 0)

# the argument structs of include/muon_ns.h: pointers and 64-bit integers, 32-bit integers, floats, and padding to 8 bytes
_BLOCK_NORM = struct.Struct("@29q5i2f0q").pack
_BLOCK_NORM_GRAD = struct.Struct("@31q4if0q").pack
_GATED = struct.Struct("@17q4i0q").pack
_GATED_GRAD = struct.Struct("@29q5i0q").pack


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _out8(q: Optional[Fp8Tensor]):
    return _NONE8 if q is None else (q.data.data_ptr(), q.scale.data_ptr(), q._ld())


def _vectors(post, pre, scale, cols, device):
    """post_weight, pre_weight and the scale (or None): contiguous [cols] of one type."""
    shape, kind = (cols,), post.dtype
    if post.shape == shape == pre.shape and pre.dtype == kind and post.device == device == pre.device \
            and post.is_contiguous() and pre.is_contiguous() \
            and (scale is None or scale.shape == shape and scale.dtype == kind and scale.device == device and scale.is_contiguous()):
        return
    for name, t in (("post_weight", post), ("pre_weight", pre), ("scale", scale)):
        if t is None:
            continue
        if t.shape != shape or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name} must be a contiguous [{cols}] tensor on {device}")
        if t.dtype != kind:
            raise TypeError(f"{name} is {t.dtype}: the weights and the scale have one dtype, {kind}")


def _required(**tensors):
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")


def _stride(t, like, cols, name) -> int:
    """Row stride of a tensor of `like`'s shape, dtype and device."""
    _like(t, like, name)
    return cols if t.is_contiguous() else _rows(t, name)[1]


def _per_row(gate, like) -> bool:
    """Whether a gate is one of each row."""
    if gate.shape == like.shape:
        return False
    if gate.shape != (*like.shape[:-1], 1):
        raise ValueError(f"gate must be {list(like.shape)} or {[*like.shape[:-1], 1]}, not {list(gate.shape)}")
    return True


def _kept(name, t, dy, rows, cols):
    """(data pointer, scale pointer, row stride, 8-bit format or None) of a kept matrix."""
    if isinstance(t, Fp8Tensor):
        if t.data.shape != (rows, cols) or t.data.device != dy.device:
            raise ValueError(f"{name} must be an 8-bit [{rows}, {cols}] matrix on {dy.device}")
        return t.data.data_ptr(), t.scale.data_ptr(), t._ld(), _TYPE_FMT[t.data.dtype]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor or an Fp8Tensor")
    return t.data_ptr(), 0, _stride(t, dy, cols, name), None


def _tensors(*kept):
    """The tensors of kept matrices, for their lifetime on another stream."""
    out = []
    for t in kept:
        out += (t.data, t.scale) if isinstance(t, Fp8Tensor) else (t,)
    return out


def _vector(n, device):  # one allocation each: views of a new one cost the host twice as much
    return torch.empty(n, dtype=torch.float32, device=device)


def _new(like, device):
    return torch.empty_like(like) if like.is_contiguous() else torch.empty(like.shape, dtype=like.dtype, device=device)


# ---------------------------------------------------------------- norms around a block

class BlockNormKept(NamedTuple):
    """What block_norm_backward needs of the forward pass: x, h and the gate as tensors, or x, h and a gate of every
    element in 8 bits; and the two norms' factors, fp32 [rows]."""
    x: Union[torch.Tensor, Fp8Tensor]
    h: Union[torch.Tensor, Fp8Tensor]
    gate: Union[torch.Tensor, Fp8Tensor, None]
    rstd_x: torch.Tensor
    rstd_h: torch.Tensor


class BlockNormOutput(NamedTuple):
    y: Optional[torch.Tensor]     # normalised stream
    h: torch.Tensor               # the stream
    q: Optional[Fp8Tensor]        # y in 8 bits, [rows, cols]
    kept: BlockNormKept


class BlockNormGrads(NamedTuple):
    dx: torch.Tensor
    dresidual: torch.Tensor
    dgate: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]   # fp32 [cols], as the next two
    dpre_weight: Optional[torch.Tensor]
    dscale: Optional[torch.Tensor]


def block_norm(x: torch.Tensor, residual: torch.Tensor, post_weight: torch.Tensor, pre_weight: torch.Tensor,
               gate: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, alpha: float = 1.0,
               eps: float = 1e-6, fp8: Optional[str] = None, y: bool = True, checkpoint: Optional[str] = None,
               stream=None) -> BlockNormOutput:
    """A block's output x joins the residual stream and the next block's norm follows (C-ABI muon_block_norm):

        h = alpha residual + sigmoid(gate) scale rms(x) post_weight        y = rms(h) pre_weight

    with rms(v) = v / sqrt(mean(v^2) + eps) over the last dimension.  x and residual are bf16, fp16 or fp32 of one shape;
    gate (or None) holds logits of x's type, one for each element or, with a last dimension of 1, for each row; the
    weights and scale (or None) are [cols] of one type.  `fp8` ("e4m3" or "e5m2") asks for y in 8 bits as well, `y=False`
    leaves out the other y.  What the gradient needs is in `kept`: x, h and gate themselves, or with `checkpoint` 8-bit
    copies of them (a gate of each row stays as it is).

    With `checkpoint` a gate of every element is shut by a finite value: an infinity makes its block of 128 NaN in 8 bits, and
    the type's lowest value leaves the block's other gates 0 there; -100 does neither."""
    _required(x=x, residual=residual, post_weight=post_weight, pre_weight=pre_weight)
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least 1")
    if not (y or fp8):
        raise ValueError("neither y nor an 8-bit copy is asked for")
    rows, ldx = _rows(x, "x")
    cols = shape[-1]
    ldr = _stride(residual, x, cols, "residual")
    dev, per_row, ldg = x.device, 0, 0
    if gate is not None:
        if gate.dtype != x.dtype or gate.device != dev:
            raise ValueError("gate must have the dtype and device of x")
        per_row = 1 if _per_row(gate, x) else 0
        ldg = cols if not per_row and gate.is_contiguous() else _rows(gate, "gate")[1]
    _vectors(post_weight, pre_weight, scale, cols, dev)
    codes = (_dt(x, "x"), _dt(post_weight, "post_weight"), per_row, 0 if fp8 is None else _fmt_code(fp8),
             0 if checkpoint is None else _fmt_code(checkpoint))
    return _on(stream, dev, (x, residual, gate, post_weight, scale, pre_weight), _block_norm, x, ldx, residual, ldr, gate, ldg,
               post_weight, scale, pre_weight, rows, codes, float(alpha), float(eps), fp8, y, checkpoint, dev)


def _block_norm(x, ldx, residual, ldr, gate, ldg, post, scale, pre, rows, codes, alpha, eps, fp8, y, checkpoint, dev, st):
    cols = x.shape[-1]
    h, out = _new(x, dev), _new(x, dev) if y else None
    rstd_x, rstd_h = _vector(rows, dev), _vector(rows, dev)
    q = None if fp8 is None else Fp8Tensor.empty(rows, cols, fp8, dev)
    x8 = h8 = gate8 = None
    kept = BlockNormKept(x, h, gate, rstd_x, rstd_h)
    if checkpoint is not None:
        x8, h8 = Fp8Tensor.empty(rows, cols, checkpoint, dev), Fp8Tensor.empty(rows, cols, checkpoint, dev)
        if gate is not None and not codes[2]:
            gate8 = Fp8Tensor.empty(rows, cols, checkpoint, dev)
        kept = BlockNormKept(x8, h8, gate if gate8 is None else gate8, rstd_x, rstd_h)
    _b._check(_b.load().muon_block_norm(_BLOCK_NORM(
        x.data_ptr(), ldx, residual.data_ptr(), ldr, _ptr(gate), ldg, post.data_ptr(), _ptr(scale), pre.data_ptr(),
        _ptr(out), cols, h.data_ptr(), cols, rstd_x.data_ptr(), rstd_h.data_ptr(), *_out8(q), *_out8(x8), *_out8(h8), *_out8(gate8), rows, cols,
        *codes, alpha, eps), st))
    return BlockNormOutput(out, h, q, kept)


def block_norm_backward(dy: torch.Tensor, kept: BlockNormKept, post_weight: torch.Tensor, pre_weight: torch.Tensor,
                        scale: Optional[torch.Tensor] = None, alpha: float = 1.0, dh: Optional[torch.Tensor] = None,
                        dweights: bool = True, stream=None) -> BlockNormGrads:
    """Gradient of block_norm (C-ABI muon_block_norm_backward) from what it kept.

    `dh` is what reaches h on its way past the second norm.  dx, dresidual and dgate have the types of the forward pass;
    the gradients of the weights and of the scale are fp32 [cols], or None with `dweights=False`."""
    _required(dy=dy, post_weight=post_weight, pre_weight=pre_weight)
    shape = dy.shape
    if not shape or shape[-1] < 1:
        raise ValueError("dy needs a last dimension of at least 1")
    cols, dev = shape[-1], dy.device
    rows, lddy = _rows(dy, "dy")
    lddh = 0 if dh is None else _stride(dh, dy, cols, "dh")
    x, h, gate, rstd_x, rstd_h = kept
    kx, kh = _kept("kept.x", x, dy, rows, cols), _kept("kept.h", h, dy, rows, cols)
    kg, per_row, fmts = (0, 0, 0, kx[3]), 0, {kx[3], kh[3]}
    if isinstance(gate, Fp8Tensor):
        kg = _kept("kept.gate", gate, dy, rows, cols)
        fmts.add(kg[3])
    elif gate is not None:
        if gate.dtype != dy.dtype or gate.device != dev:
            raise ValueError("kept.gate must have the dtype and device of dy")
        per_row = 1 if _per_row(gate, dy) else 0
        kg = (gate.data_ptr(), 0, _rows(gate, "kept.gate")[1], None)
        if not per_row:
            fmts.add(None)
    if len(fmts) != 1:
        raise ValueError("x, h and a gate of every element are kept as tensors, or all in one 8-bit format")
    for name, t in (("kept.rstd_x", rstd_x), ("kept.rstd_h", rstd_h)):
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be {rows} contiguous float32 values on {dev}")
    _vectors(post_weight, pre_weight, scale, cols, dev)
    codes = (_dt(dy, "dy"), _dt(post_weight, "post_weight"), per_row, kx[3] or 0)
    return _on(stream, dev, (dy, dh, rstd_x, rstd_h, post_weight, scale, pre_weight, *_tensors(x, h, gate)), _block_norm_backward,
               dy, lddy, dh, lddh, kx, kh, kg, gate, rstd_x, rstd_h, post_weight, scale, pre_weight, rows, codes, float(alpha),
               dweights, dev)


def _block_norm_backward(dy, lddy, dh, lddh, kx, kh, kg, gate, rstd_x, rstd_h, post, scale, pre, rows, codes, alpha, dweights,
                         dev, st):
    lib = _b.load()
    cols = dy.shape[-1]
    dx, dresidual = _new(dy, dev), _new(dy, dev)
    dgate, ldgate = None, 0
    if gate is not None:
        dgate = torch.empty((*dy.shape[:-1], 1) if codes[2] else dy.shape, dtype=dy.dtype, device=dev)
        ldgate = 1 if codes[2] else cols
    dpost = dpre = dscale = ws = None
    size = 0
    if dweights:
        dpost, dpre, dscale = _vector(cols, dev), _vector(cols, dev), None if scale is None else _vector(cols, dev)
        size = lib.muon_block_norm_backward_workspace_bytes_for(rows, cols, codes[0])
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _b._check(lib.muon_block_norm_backward(_BLOCK_NORM_GRAD(
        dy.data_ptr(), lddy, _ptr(dh), lddh, *kx[:3], *kh[:3], *kg[:3], rstd_x.data_ptr(), rstd_h.data_ptr(), post.data_ptr(),
        _ptr(scale), pre.data_ptr(), dx.data_ptr(), cols, dresidual.data_ptr(), cols, _ptr(dgate), ldgate, _ptr(dpost), _ptr(dpre), _ptr(dscale), _ptr(ws), size,
        rows, cols, *codes, alpha), st))
    return BlockNormGrads(dx, dresidual, dgate, dpost, dpre, dscale)


# ---------------------------------------------------------------- gated activation

class GatedKept(NamedTuple):
    """What gated_activation_backward needs of the forward pass: both branches, as tensors or in 8 bits."""
    gate: Union[torch.Tensor, Fp8Tensor]
    up: Union[torch.Tensor, Fp8Tensor]


class GatedOutput(NamedTuple):
    y: Optional[torch.Tensor]
    q: Optional[Fp8Tensor]        # y in 8 bits, [rows, cols]
    kept: GatedKept


class GatedGrads(NamedTuple):
    dgate: Optional[torch.Tensor]
    dup: Optional[torch.Tensor]
    dgate_rows: Optional[Fp8Tensor]   # [rows, cols], for the products with the weights
    dgate_cols: Optional[Fp8Tensor]   # transposed, for the weights' gradients
    dup_rows: Optional[Fp8Tensor]
    dup_cols: Optional[Fp8Tensor]
    y_cols: Optional[Fp8Tensor]       # the activation again, transposed


def _activation(name: str) -> int:
    try:
        return _ACT[name]
    except KeyError:
        raise ValueError(f"unknown activation {name!r}: 'silu' or 'gelu'") from None


def gated_activation(gate: torch.Tensor, up: torch.Tensor, activation: str = "silu", fp8: Optional[str] = None, y: bool = True,
                     checkpoint: Optional[str] = None, stream=None) -> GatedOutput:
    """y = f(gate) up, f "silu" (g / (1 + exp(-g))) or "gelu" (g times the normal distribution's function) (C-ABI
    muon_gated_activation).

    gate and up are bf16, fp16 or fp32 of one shape, each with its own row stride (the halves of one product, say).  `fp8`
    ("e4m3" or "e5m2") asks for y in 8 bits as well, `y=False` leaves out the other y.  `kept` is for the gradient: gate
    and up themselves, or with `checkpoint` 8-bit copies of them."""
    _required(gate=gate, up=up)
    if not gate.shape:
        raise ValueError("gate must have at least one dimension")
    act = _activation(activation)
    if not (y or fp8):
        raise ValueError("neither y nor an 8-bit copy is asked for")
    rows, ldg = _rows(gate, "gate")
    ldu = _stride(up, gate, gate.shape[-1], "up")
    codes = (_dt(gate, "gate"), act, 0 if fp8 is None else _fmt_code(fp8), 0 if checkpoint is None else _fmt_code(checkpoint))
    return _on(stream, gate.device, (gate, up), _gated, gate, ldg, up, ldu, rows, codes, fp8, y, checkpoint, gate.device)


def _gated(gate, ldg, up, ldu, rows, codes, fp8, y, checkpoint, dev, st):
    cols = gate.shape[-1]
    out = _new(gate, dev) if y else None
    q = None if fp8 is None else Fp8Tensor.empty(rows, cols, fp8, dev)
    kept = GatedKept(gate, up)
    g8 = u8 = None
    if checkpoint is not None:
        g8, u8 = Fp8Tensor.empty(rows, cols, checkpoint, dev), Fp8Tensor.empty(rows, cols, checkpoint, dev)
        kept = GatedKept(g8, u8)
    _b._check(_b.load().muon_gated_activation(_GATED(
        gate.data_ptr(), ldg, up.data_ptr(), ldu, _ptr(out), cols, *_out8(q), *_out8(g8), *_out8(u8), rows, cols, *codes), st))
    return GatedOutput(out, q, kept)


def gated_activation_backward(dy: torch.Tensor, kept: GatedKept, activation: str = "silu", dense: bool = True,
                              fp8: Optional[str] = None, y_fp8: Optional[str] = None, stream=None) -> GatedGrads:
    """Gradient of gated_activation (C-ABI muon_gated_activation_backward) from what it kept, in one pass.

    `dense` asks for dgate and dup in dy's type; `fp8` for both in 8 bits, along their columns and transposed, as the
    products that follow read them; `y_fp8` for the activation again, transposed in 8 bits, for the gradient of the
    weight behind it."""
    _required(dy=dy)
    if not dy.shape:
        raise ValueError("dy must have at least one dimension")
    act = _activation(activation)
    if not (dense or fp8 or y_fp8):
        raise ValueError("no gradient is asked for")
    rows, lddy = _rows(dy, "dy")
    gate, up = kept
    kg, ku = _kept("kept.gate", gate, dy, rows, dy.shape[-1]), _kept("kept.up", up, dy, rows, dy.shape[-1])
    if kg[3] != ku[3]:
        raise ValueError("gate and up are kept as tensors, or both in one 8-bit format")
    codes = (_dt(dy, "dy"), act, kg[3] or 0, 0 if fp8 is None else _fmt_code(fp8), 0 if y_fp8 is None else _fmt_code(y_fp8))
    return _on(stream, dy.device, (dy, *_tensors(gate, up)), _gated_backward, dy, lddy, kg, ku, rows, codes, dense, fp8, y_fp8,
               dy.device)


def _gated_backward(dy, lddy, kg, ku, rows, codes, dense, fp8, y_fp8, dev, st):
    cols = dy.shape[-1]
    dgate, dup = (_new(dy, dev), _new(dy, dev)) if dense else (None, None)
    by_rows = by_cols = (None, None)
    if fp8 is not None:
        by_rows = Fp8Tensor.empty(rows, cols, fp8, dev), Fp8Tensor.empty(rows, cols, fp8, dev)
        by_cols = Fp8Tensor.empty(cols, rows, fp8, dev), Fp8Tensor.empty(cols, rows, fp8, dev)
    y_cols = None if y_fp8 is None else Fp8Tensor.empty(cols, rows, y_fp8, dev)
    _b._check(_b.load().muon_gated_activation_backward(_GATED_GRAD(
        dy.data_ptr(), lddy, *kg[:3], *ku[:3], _ptr(dgate), cols, _ptr(dup), cols, *_out8(by_rows[0]), *_out8(by_cols[0]),
        *_out8(by_rows[1]), *_out8(by_cols[1]), *_out8(y_cols), rows, cols, *codes), st))
    return GatedGrads(dgate, dup, by_rows[0], by_cols[0], by_rows[1], by_cols[1], y_cols)


# ---------------------------------------------------------------- transposition

def fp8_transpose(q: Fp8Tensor, stream=None) -> Fp8Tensor:
    """An 8-bit matrix [rows, cols] as the 8-bit matrix [cols, rows] of the same format, with scales for 128 of its rows
    (C-ABI muon_fp8_transpose): a checkpoint as the operand of a product that sums over its rows."""
    if not isinstance(q, Fp8Tensor):
        raise TypeError("q must be an Fp8Tensor")
    if not q.data.is_cuda:
        raise ValueError("q must be on a CUDA device")
    return _on(stream, q.data.device, (q.data, q.scale), _transpose, q, q.data.device)


def _transpose(q, dev, st):
    rows, cols = q.data.shape
    out = Fp8Tensor.empty(cols, rows, q.fmt, dev)
    _b._check(_b.load().muon_fp8_transpose(q.data.data_ptr(), q._ld(), q.scale.data_ptr(), rows, cols, _TYPE_FMT[q.data.dtype],
                                           out.data.data_ptr(), out._ld(), out.scale.data_ptr(), st))
    return out
