"""The operators around the Muon update (argument checks and marshalling; the work runs in the library's kernels):
gradient clipping by the global norm, the RMS norm with an 8-bit copy and its gradient, quantisation to 8 bits and the
8-bit matrix product.  One training step of a layer:

    r = rms_norm(x, w_norm, residual=stream, fp8="e4m3")       # r.q feeds the product, r.h is the new stream
    out = fp8_matmul(r.q, W_rows)                              # W_rows, W_cols = fp8_quantize(W, square=True, cols=True)
    dq, dqt = fp8_quantize(dout, "e5m2", cols=True)
    dy = fp8_matmul(dq, W_cols)                                # data gradient
    dW = fp8_matmul(dqt, fp8_quantize(r.y, rows=False, cols=True)[1], torch.float32, add=dW)   # weight gradient
    dx, dw_norm = rms_norm_backward(dy, r.h, w_norm, r.rstd, dresidual=dstream)
    clip_grads(grads, max_norm=1.0)                            # then muon_step

Autograd does not see these calls: their results have no gradient function, whatever the inputs require, and what is
written in place or to `out` keeps its version.  The backward pass is written out, as above.

With `stream=` (a stream of the tensors' device) a call runs there and its results belong to that stream; the caller
orders it after what its inputs wait for, and what reads the results after it.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import NamedTuple, Optional, Sequence

import torch

from . import binding as _b

_DT = {torch.bfloat16: _b.BF16, torch.float32: _b.FP32, torch.float16: _b.FP16}
_FMT = {"e4m3": 0, "e5m2": 1}
_FMT_TYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TYPE_FMT = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_SCALE_TYPES = (torch.float8_e8m0fnu, torch.uint8)


def _dt(t: torch.Tensor, name: str) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}: bfloat16, float16 or float32") from None


def _rows(t: torch.Tensor, name: str):
    """(rows, row stride) of a tensor seen as rows of its last dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, strides = t.shape, t.stride()
    dims = len(shape)
    if dims == 2:  # the ordinary case, without a view
        rows, width = shape
        ld, unit = strides
    else:
        if dims < 1:
            raise ValueError(f"{name} must have at least one dimension")
        width, unit = shape[-1], strides[-1]
        try:
            v = t.view(-1, width) if width else t.reshape(0, 0)
        except RuntimeError:
            raise ValueError(f"{name}: the rows must be evenly spaced (one stride for all leading dimensions)") from None
        rows, ld = v.shape[0], v.stride(0)
    if unit != 1 and width > 1:
        raise ValueError(f"{name}: elements of a row must be consecutive (last stride 1, not {unit})")
    if ld < width:
        if rows > 1:
            raise ValueError(f"{name}: rows overlap (stride {ld} for {width} columns)")
        ld = width
    return rows, ld


def _like(t, ref, name):
    if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{name} must have the shape, dtype and device of the input")


def _on(stream, device, tensors, call, *args):
    """call(*args, stream pointer) with `device` and `stream` (None: its current one) current, so that the tensors made
    within belong to that stream.  The memory of `tensors` (or None among them), which it reads or writes, is not given
    away before a `stream` of the caller's has passed the call."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return call(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return call(*args, torch.cuda.current_stream().cuda_stream)


# ---------------------------------------------------------------- 8-bit matrices

class Fp8Tensor:
    """An 8-bit matrix [rows, cols] whose blocks of 128 columns share a power-of-two scale.

    `data` is float8_e4m3fn or float8_e5m2, 16-byte aligned, with a row stride that is a multiple of 16; `scale` is
    contiguous float8_e8m0fnu (or uint8) [ceil(cols / 512), rows rounded up to 4, 4]: the scale of block kb of row r is
    at [kb // 4, r, kb % 4].  Element (r, c) stands for data[r, c] * scale of block c // 128."""

    __slots__ = ("data", "scale")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor):
        if data.dim() != 2 or data.dtype not in _TYPE_FMT:
            raise TypeError("data must be a 2-D float8_e4m3fn or float8_e5m2 tensor")
        if scale.dtype not in _SCALE_TYPES or not scale.is_contiguous():
            raise TypeError("scale must be a contiguous float8_e8m0fnu or uint8 tensor")
        rows, cols = data.shape
        if tuple(scale.shape) != (-(-cols // 512), -(-rows // 4) * 4, 4):
            raise ValueError(f"scale of a [{rows}, {cols}] matrix is [{-(-cols // 512)}, {-(-rows // 4) * 4}, 4], "
                             f"not {list(scale.shape)}")
        if data.device != scale.device:
            raise ValueError("data and scale must be on one device")
        if data.numel() and ((cols > 1 and data.stride(1) != 1) or (rows > 1 and data.stride(0) < cols)):
            raise ValueError("elements of a row must be consecutive and rows must not overlap")
        if data.numel() and (data.data_ptr() % 16 or (rows > 1 and data.stride(0) % 16)):
            raise ValueError("data must be 16-byte aligned with a row stride that is a multiple of 16")
        if scale.numel() and scale.data_ptr() % 16:
            raise ValueError("scale must be 16-byte aligned")
        self.data, self.scale = data, scale

    @classmethod
    def empty(cls, rows: int, cols: int, fmt: str = "e4m3", device=None) -> "Fp8Tensor":
        """Uninitialised, with the row padding that the product asks for."""
        if fmt not in _FMT_TYPE:
            raise _unknown(fmt)
        self = object.__new__(cls)
        pitch = (cols + 15) // 16 * 16
        data = torch.empty((rows, pitch), dtype=_FMT_TYPE[fmt], device=device or "cuda")
        self.data = data if pitch == cols else data.as_strided((rows, cols), (pitch, 1))
        self.scale = torch.empty(((cols + 511) // 512, (rows + 3) // 4 * 4, 4), dtype=torch.float8_e8m0fnu,
                                 device=data.device)
        return self

    @property
    def shape(self):
        return self.data.shape

    @property
    def fmt(self) -> str:
        return "e5m2" if self.data.dtype == torch.float8_e5m2 else "e4m3"

    def scales(self) -> torch.Tensor:
        """The scales as fp32 [rows, ceil(cols / 128)]."""
        rows, cols = self.data.shape
        s = self.scale.view(torch.float8_e8m0fnu).to(torch.float32)
        return s.permute(1, 0, 2).reshape(s.shape[1], -1)[:rows, :-(-cols // 128)]

    def dequantize(self) -> torch.Tensor:
        """What the matrix stands for, in fp32 (for inspection and tests; the product reads the 8 bits)."""
        cols = self.data.shape[1]
        return self.data.to(torch.float32) * self.scales().repeat_interleave(128, dim=1)[:, :cols]

    def _ld(self) -> int:
        return self.data.stride(0) if self.data.shape[0] > 1 else -(-self.data.shape[1] // 16) * 16

    def __repr__(self):
        return f"Fp8Tensor({list(self.data.shape)}, {self.fmt}, device={self.data.device})"


def _unknown(fmt) -> ValueError:
    return ValueError(f"unknown 8-bit format {fmt!r}: 'e4m3' or 'e5m2'")


def _fmt_code(fmt: str) -> int:
    try:
        return _FMT[fmt]
    except KeyError:
        raise _unknown(fmt) from None


def fp8_quantize(x: torch.Tensor, fmt: str = "e4m3", square: bool = False, rows: bool = True, cols: bool = False,
                 stream=None):
    """x [rows, cols] (bf16, fp16, fp32) in 8 bits (C-ABI muon_fp8_quantize): (along its columns, transposed).

    The first is x as an operand summed over its columns, the second x transposed, summed over x's rows; each is an
    Fp8Tensor, or None where `rows` / `cols` is false.  Scales belong to 128 elements along the summed axis, or with
    `square` to 128 x 128 (weights: both then stand for the same values)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if not (rows or cols):
        raise ValueError("neither rows nor cols is asked for")
    n, ld = _rows(x, "x")
    return _on(stream, x.device, (x,), _quantize, x, n, ld, _dt(x, "x"), _fmt_code(fmt), fmt, 1 if square else 0, rows, cols)


def _quantize(x, n, ld, dt, code, fmt, square, rows, cols, st):
    m, dev = x.shape[1], x.device
    q = qt = None
    args, argst = (None, 0, None), (None, 0, None)
    if rows:
        q = Fp8Tensor.empty(n, m, fmt, dev)
        args = (q.data.data_ptr(), q._ld(), q.scale.data_ptr())
    if cols:
        qt = Fp8Tensor.empty(m, n, fmt, dev)
        argst = (qt.data.data_ptr(), qt._ld(), qt.scale.data_ptr())
    _b._check(_b.load().muon_fp8_quantize(x.data_ptr(), ld, n, m, dt, code, square, *args, *argst, st))
    return q, qt


def fp8_matmul(a: Fp8Tensor, b: Fp8Tensor, out_dtype=torch.bfloat16, add: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a @ b.T (+ add) for 8-bit a [m, k] and b [n, k] (C-ABI muon_fp8_matmul), summed in fp32 and rounded once.

    `add` and `out` are [m, n] of `out_dtype` (bf16, fp16 or fp32; `out` decides where it is given); `out` may be `add`,
    which accumulates."""
    if not isinstance(a, Fp8Tensor) or not isinstance(b, Fp8Tensor):
        raise TypeError("a and b must be Fp8Tensor")
    dev = a.data.device
    if a.data.shape[1] != b.data.shape[1]:
        raise ValueError(f"a has {a.data.shape[1]} columns and b {b.data.shape[1]}: both are summed over them")
    if not a.data.is_cuda:
        raise ValueError("a must be on a CUDA device")
    if b.data.device != dev:
        raise ValueError(f"b is on {b.data.device}, not {dev}")
    return _on(stream, dev, (a.data, a.scale, b.data, b.scale, add, out), _matmul, a, b, out_dtype, add, out, dev)


def _matmul(a, b, out_dtype, add, out, dev, st):
    ad, bd = a.data, b.data
    (m, k), n = ad.shape, bd.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
        ldc = n
    else:
        if out.shape != (m, n) or out.device != dev:
            raise ValueError(f"out must be [{m}, {n}] on {dev}")
        ldc = _rows(out, "out")[1]
    addp, ldadd = None, 0
    if add is not None:
        _like(add, out, "add")
        addp, ldadd = add.data_ptr(), _rows(add, "add")[1]
    _b._check(_b.load().muon_fp8_matmul(
        ad.data_ptr(), a._ld(), a.scale.data_ptr(), _TYPE_FMT[ad.dtype], bd.data_ptr(), b._ld(), b.scale.data_ptr(),
        _TYPE_FMT[bd.dtype], m, n, k, addp, ldadd, out.data_ptr(), ldc, _dt(out, "out"), st))
    return out


def _status_device(stream, device):
    if device is None:
        return torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    device = torch.device(device)
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


def fp8_status(stream=None, device=None) -> int:
    """Synchronise and read/clear the 8-bit product's status (OK, or ERR_TIMEOUT where a kernel gave up on a wait).

    The status is that of `device` (default: the stream's, or the current one): one for all its streams, each report given
    once."""
    return _on(stream, _status_device(stream, device), (), _b.load().muon_fp8_status)


def debug_bounded_wait_fp8(max_cycles: int, stream=None, device=None) -> None:
    """Self-test of fp8_status: a wait on `device` that runs out after `max_cycles`."""
    _b._check(_on(stream, _status_device(stream, device), (), _b.load().muon_debug_bounded_wait_fp8, int(max_cycles)))


# ---------------------------------------------------------------- RMS norm

class RmsNormOutput(NamedTuple):
    y: Optional[torch.Tensor]     # normalised rows
    h: torch.Tensor               # x + residual (x itself without a residual)
    rstd: torch.Tensor            # [rows] fp32, for the gradient
    q: Optional[Fp8Tensor]        # y in 8 bits, [rows, cols]


def _weight(weight, cols, device):
    if weight is None:
        return None, 0
    if weight.dim() != 1 or weight.shape[0] != cols or not weight.is_contiguous() or weight.device != device:
        raise ValueError(f"weight must be a contiguous [{cols}] tensor on {device}")
    return weight.data_ptr(), _dt(weight, "weight")


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor], residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             fp8: Optional[str] = None, y: bool = True, stream=None) -> RmsNormOutput:
    """Root-mean-square norm over the last dimension (C-ABI muon_rms_norm): h = x + residual,
    y = h / sqrt(mean(h^2) + eps) * weight, and with `fp8` ("e4m3" or "e5m2") y in 8 bits as well; `y=False` leaves out
    the 16- or 32-bit y.  x is bf16, fp16 or fp32 with any leading dimensions; weight (or None) may have another of these
    types.  The sum of squares is fp32: a row for which it overflows gets rstd = 0 and y = 0."""
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least 1")
    rows, ldx = _rows(x, "x")
    if not (y or fp8):
        raise ValueError("neither y nor an 8-bit copy is asked for")
    ldr, res = 0, None
    if residual is not None:
        _like(residual, x, "residual")
        ldr, res = _rows(residual, "residual")[1], residual.data_ptr()
    dev = x.device
    wp, wdt = _weight(weight, shape[-1], dev)
    return _on(stream, dev, (x, residual, weight), _rms_norm, x, ldx, res, ldr, wp, wdt, rows, shape[-1], float(eps), fp8, y,
               _dt(x, "x"), dev)


def _rms_norm(x, ldx, res, ldr, wp, wdt, rows, cols, eps, fp8, y, dt, dev, st):
    out = h = q = None
    yp = hp = None
    qa, code = (None, 0, None), 0
    contiguous = x.is_contiguous()
    if y:
        out = torch.empty_like(x) if contiguous else torch.empty(x.shape, dtype=x.dtype, device=dev)
        yp = out.data_ptr()
    if res is not None:
        h = torch.empty_like(x) if contiguous else torch.empty(x.shape, dtype=x.dtype, device=dev)
        hp = h.data_ptr()
    rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    if fp8 is not None:
        code = _fmt_code(fp8)
        q = Fp8Tensor.empty(rows, cols, fp8, dev)
        qa = (q.data.data_ptr(), q._ld(), q.scale.data_ptr())
    _b._check(_b.load().muon_rms_norm(x.data_ptr(), ldx, res, ldr, wp, wdt, rows, cols, eps, yp, cols, hp, cols,
                                      rstd.data_ptr(), *qa, code, dt, st))
    return RmsNormOutput(out, x if h is None else h, rstd, q)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                      dresidual: Optional[torch.Tensor] = None, dweight: bool = True, stream=None):
    """Gradient of rms_norm (C-ABI muon_rms_norm_backward): (dx, dweight).

    dx is the gradient of x and of the residual alike, plus `dresidual`, what reaches h on its way past the norm;
    dweight is fp32 [cols], or None with `dweight=False`."""
    shape = dy.shape
    if not shape or shape[-1] < 1:
        raise ValueError("dy needs a last dimension of at least 1")
    cols = shape[-1]
    rows, lddy = _rows(dy, "dy")
    _like(h, dy, "h")
    ldh = _rows(h, "h")[1]
    lddr, res = 0, None
    if dresidual is not None:
        _like(dresidual, dy, "dresidual")
        lddr, res = _rows(dresidual, "dresidual")[1], dresidual.data_ptr()
    dev = dy.device
    if rstd.dtype != torch.float32 or rstd.numel() != rows or not rstd.is_contiguous() or rstd.device != dev:
        raise ValueError(f"rstd must be {rows} contiguous float32 values on {dev}")
    wp, wdt = _weight(weight, cols, dev)
    return _on(stream, dev, (dy, h, weight, rstd, dresidual), _rms_norm_backward, dy, lddy, h.data_ptr(), ldh, wp, wdt,
               rstd.data_ptr(), res, lddr, rows, cols, dweight, _dt(dy, "dy"), dev)


def _rms_norm_backward(dy, lddy, hp, ldh, wp, wdt, rp, res, lddr, rows, cols, dweight, dt, dev, st):
    lib = _b.load()
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dev)
    dw = dwp = ws = None
    size = 0
    if dweight:
        dw = torch.empty(cols, dtype=torch.float32, device=dev)
        size = lib.muon_rms_norm_backward_workspace_bytes(rows, cols)
        keep = torch.empty(size, dtype=torch.uint8, device=dev)
        dwp, ws = dw.data_ptr(), keep.data_ptr()
    _b._check(lib.muon_rms_norm_backward(dy.data_ptr(), lddy, hp, ldh, wp, wdt, rp, res, lddr, rows, cols, dx.data_ptr(), cols,
                                         dwp, ws, size, dt, st))
    return dx, dw


# ---------------------------------------------------------------- clipping

def _clip(grads, max_norm, out, eps, stream):
    count = len(grads)
    if count == 0:
        raise ValueError("no gradients")
    dev = grads[0].device
    tensor = torch.Tensor
    on = list(map(tensor.get_device, grads))  # -1 on the CPU
    if on[0] < 0 or on.count(on[0]) != count or not all(map(tensor.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous CUDA tensors on one device")
    kinds = [g.dtype for g in grads]
    try:
        dts = array("i", [_DT[k] for k in kinds])
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e.args[0]}: bfloat16, float16 or float32") from None
    numel = list(map(tensor.numel, grads))
    # one host array: gradient pointers, element counts, the outputs' pointers where they are others
    table = list(map(tensor.data_ptr, grads)) + numel
    if out is not None and out is not grads:
        if [o.dtype for o in out] != kinds or list(map(tensor.numel, out)) != numel \
                or list(map(tensor.get_device, out)) != on or not all(map(tensor.is_contiguous, out)):
            raise ValueError("there must be one out per gradient, contiguous, of its size, dtype and device")
        table += map(tensor.data_ptr, out)
    table = array("q", table)
    base = table.buffer_info()[0]
    outs = None if out is None else base if out is grads else base + 16 * count
    tensors = grads if out is None or out is grads else [*grads, *out]
    return _on(stream, dev, tensors, _clip_call, base, outs, base + 8 * count, dts.buffer_info()[0], count, max_norm, eps, dev,
               (table, dts))


def _clip_call(grads, outs, numel, dts, count, max_norm, eps, dev, keep, st):
    lib = _b.load()
    size = lib.muon_clip_workspace_bytes(count)
    ws = torch.empty(size // 4 + 1, dtype=torch.float32, device=dev)  # partial sums, then the norm
    norm = ws.as_strided((), (), size // 4)
    at = ws.data_ptr()
    _b._check(lib.muon_clip_grads(grads, outs, numel, dts, count, max_norm, eps, at + size, at, size, st))
    return norm


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
               eps: float = 1e-6, stream=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (N + eps)), N their global norm, in place or into `out` (C-ABI
    muon_clip_grads), and returns N (a 0-d fp32 tensor on the device; nothing waits for it).

    A tensor is listed once: outputs that share memory with another tensor of the list are refused."""
    return _clip(grads, float(max_norm), grads if out is None else out, float(eps), stream)


def grad_norm(grads: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
    """The global norm of the gradients as a 0-d fp32 tensor on the device."""
    return _clip(grads, 0.0, None, 0.0, stream)
