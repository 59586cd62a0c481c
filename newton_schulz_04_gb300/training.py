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
"""
from __future__ import annotations

import ctypes
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


def _rows(t: torch.Tensor, name: str, cols=None):
    """(rows, row stride) of a tensor seen as rows of its last dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() == 2:  # the ordinary case, without a view
        rows, width = t.shape
        ld = t.stride(0)
        unit = t.stride(1)
    else:
        if t.dim() < 1:
            raise ValueError(f"{name} must have at least one dimension")
        width = t.shape[-1]
        try:
            v = t.view(-1, width) if width else t.reshape(0, 0)
        except RuntimeError:
            raise ValueError(f"{name}: the rows must be evenly spaced (one stride for all leading dimensions)") from None
        rows, ld, unit = v.shape[0], v.stride(0), v.stride(1) if width else 1
    if width > 1 and unit != 1:
        raise ValueError(f"{name}: elements of a row must be consecutive (last stride 1, not {unit})")
    if rows > 1 and ld < width:
        raise ValueError(f"{name}: rows overlap (stride {ld} for {width} columns)")
    if cols is not None and width != cols:
        raise ValueError(f"{name} has {width} columns, {cols} expected")
    return rows, max(ld, width)


def _like(t, ref, name):
    if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{name} must have the shape, dtype and device of the input")


def _same_device(ref, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, not {ref.device}")


def _workspace(workspace, need, device, name="workspace"):
    """(pointer, bytes) of the caller's workspace, or of a new one (returned to be kept alive)."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not (workspace.is_cuda and workspace.is_contiguous() and workspace.device == device):
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


class _on:
    """Makes `stream` (None: the current one) current, so that tensors made within belong to it."""

    def __new__(cls, stream, device):
        if stream is None and device.index == torch.cuda.current_device():
            return _HERE
        return _Guard(stream, device)


class _Here:
    def __enter__(self):
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        return False


class _Guard:
    def __init__(self, stream, device):
        self.stream, self.device = stream, device

    def __enter__(self):
        self.dev = torch.cuda.device(self.device)
        self.dev.__enter__()
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)
        return self.dev.__exit__(*exc)


_HERE = _Here()


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
        self = object.__new__(cls)
        pitch = (cols + 15) // 16 * 16
        data = torch.empty((rows, pitch), dtype=_FMT_TYPE[fmt], device=device or "cuda")
        self.data = data if pitch == cols else data[:, :cols]
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


def _fmt_code(fmt: str) -> int:
    try:
        return _FMT[fmt]
    except KeyError:
        raise ValueError(f"unknown 8-bit format {fmt!r}: 'e4m3' or 'e5m2'") from None


def fp8_quantize(x: torch.Tensor, fmt: str = "e4m3", square: bool = False, rows: bool = True, cols: bool = False,
                 stream=None):
    """x [rows, cols] (bf16, fp16, fp32) in 8 bits (C-ABI muon_fp8_quantize): (along its columns, transposed).

    The first is x as an operand summed over its columns, the second x transposed, summed over x's rows; each is an
    Fp8Tensor, or None where `rows` / `cols` is false.  Scales belong to 128 elements along the summed axis, or with
    `square` to 128 x 128 (weights: both then stand for the same values)."""
    lib = _b.load()
    code = _fmt_code(fmt)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    if not (rows or cols):
        raise ValueError("neither rows nor cols is asked for")
    n, ld = _rows(x, "x")
    m = x.shape[1]
    dt = _dt(x, "x")
    with _on(stream, x.device) as st:
        q = Fp8Tensor.empty(n, m, fmt, x.device) if rows else None
        qt = Fp8Tensor.empty(m, n, fmt, x.device) if cols else None
        _b._check(lib.muon_fp8_quantize(
            x.data_ptr(), ld, n, m, dt, code, 1 if square else 0, q.data.data_ptr() if rows else None,
            q._ld() if rows else 0, q.scale.data_ptr() if rows else None, qt.data.data_ptr() if cols else None,
            qt._ld() if cols else 0, qt.scale.data_ptr() if cols else None, st))
    return q, qt


def fp8_matmul(a: Fp8Tensor, b: Fp8Tensor, out_dtype=torch.bfloat16, add: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a @ b.T (+ add) for 8-bit a [m, k] and b [n, k] (C-ABI muon_fp8_matmul), summed in fp32 and rounded once.

    `add` and `out` are [m, n] of `out_dtype` (bf16, fp16 or fp32; `out` decides where it is given); `out` may be `add`,
    which accumulates.  Where few tiles make the library split k, `workspace` (uint8, fp8_matmul_workspace_bytes) holds
    the parts; a new one is made if None."""
    lib = _b.load()
    if not isinstance(a, Fp8Tensor) or not isinstance(b, Fp8Tensor):
        raise TypeError("a and b must be Fp8Tensor")
    (m, k), (n, kb) = a.data.shape, b.data.shape
    if k != kb:
        raise ValueError(f"a has {k} columns and b {kb}: both are summed over them")
    dev = a.data.device
    if not a.data.is_cuda:
        raise ValueError("a must be on a CUDA device")
    if b.data.device != dev:
        raise ValueError(f"b is on {b.data.device}, not {dev}")
    with _on(stream, dev) as st:
        if out is None:
            out = torch.empty((m, n), dtype=out_dtype, device=dev)
            ldc = n
        else:
            if out.shape != (m, n) or out.device != dev:
                raise ValueError(f"out must be [{m}, {n}] on {dev}")
            ldc = _rows(out, "out")[1]
        dt = _dt(out, "out")
        ldadd = 0
        if add is not None:
            _like(add, out, "add")
            ldadd = _rows(add, "add")[1]
        need = lib.muon_fp8_matmul_workspace_bytes(m, n, k)
        ws = size = None
        if need:
            keep, ws, size = _workspace(workspace, need, dev)
        _b._check(lib.muon_fp8_matmul(
            a.data.data_ptr(), a._ld(), a.scale.data_ptr(), _TYPE_FMT[a.data.dtype], b.data.data_ptr(), b._ld(),
            b.scale.data_ptr(), _TYPE_FMT[b.data.dtype], m, n, k, None if add is None else add.data_ptr(), ldadd,
            out.data_ptr(), ldc, dt, ws, size or 0, st))
    return out


def fp8_matmul_workspace_bytes(m: int, n: int, k: int) -> int:
    """Bytes of workspace that fp8_matmul uses for a product of these sizes (0: none)."""
    return int(_b.load().muon_fp8_matmul_workspace_bytes(int(m), int(n), int(k)))


def fp8_status(stream=None) -> int:
    """Synchronise and read/clear the 8-bit product's status (OK, or ERR_TIMEOUT where a kernel gave up on a wait)."""
    return _b.load().muon_fp8_status(ctypes.c_void_p(_b._stream_ptr(stream)))


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
    types."""
    lib = _b.load()
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x needs a last dimension of at least 1")
    cols = x.shape[-1]
    rows, ldx = _rows(x, "x")
    dt = _dt(x, "x")
    code = _fmt_code(fp8) if fp8 is not None else 0
    if not (y or fp8):
        raise ValueError("neither y nor an 8-bit copy is asked for")
    ldr, res = 0, None
    if residual is not None:
        _like(residual, x, "residual")
        ldr, res = _rows(residual, "residual")[1], residual.data_ptr()
    wp, wdt = _weight(weight, cols, x.device)
    with _on(stream, x.device) as st:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device) if y else None
        h = torch.empty(x.shape, dtype=x.dtype, device=x.device) if residual is not None else None
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
        q = Fp8Tensor.empty(rows, cols, fp8, x.device) if fp8 is not None else None
        _b._check(lib.muon_rms_norm(
            x.data_ptr(), ldx, res, ldr, wp, wdt, rows, cols, eps, out.data_ptr() if y else None, cols,
            h.data_ptr() if h is not None else None, cols, rstd.data_ptr(), q.data.data_ptr() if q is not None else None,
            q._ld() if q is not None else 0, q.scale.data_ptr() if q is not None else None, code, dt, st))
    return RmsNormOutput(out, x if h is None else h, rstd, q)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                      dresidual: Optional[torch.Tensor] = None, dweight: bool = True, stream=None):
    """Gradient of rms_norm (C-ABI muon_rms_norm_backward): (dx, dweight).

    dx is the gradient of x and of the residual alike, plus `dresidual`, what reaches h on its way past the norm;
    dweight is fp32 [cols], or None with `dweight=False`."""
    lib = _b.load()
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError("dy needs a last dimension of at least 1")
    cols = dy.shape[-1]
    rows, lddy = _rows(dy, "dy")
    dt = _dt(dy, "dy")
    _like(h, dy, "h")
    ldh = _rows(h, "h")[1]
    lddr, res = 0, None
    if dresidual is not None:
        _like(dresidual, dy, "dresidual")
        lddr, res = _rows(dresidual, "dresidual")[1], dresidual.data_ptr()
    if rstd.dtype != torch.float32 or rstd.numel() != rows or not rstd.is_contiguous() or rstd.device != dy.device:
        raise ValueError(f"rstd must be {rows} contiguous float32 values on {dy.device}")
    wp, wdt = _weight(weight, cols, dy.device)
    with _on(stream, dy.device) as st:
        dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
        dw = ws = size = None
        if dweight:
            dw = torch.empty(cols, dtype=torch.float32, device=dy.device)
            keep, ws, size = _workspace(None, lib.muon_rms_norm_backward_workspace_bytes(rows, cols), dy.device)
        _b._check(lib.muon_rms_norm_backward(
            dy.data_ptr(), lddy, h.data_ptr(), ldh, wp, wdt, rstd.data_ptr(), res, lddr, rows, cols, dx.data_ptr(), cols,
            dw.data_ptr() if dweight else None, ws, size or 0, dt, st))
    return dx, dw


# ---------------------------------------------------------------- clipping

def _clip(grads, max_norm, out, eps, stream):
    lib = _b.load()
    count = len(grads)
    if count == 0:
        raise ValueError("no gradients")
    dev = grads[0].device
    for g in grads:
        if not g.is_cuda or g.device != dev or not g.is_contiguous():
            raise ValueError("gradients must be contiguous CUDA tensors on one device")
    P = ctypes.c_void_p * count
    try:
        dts = (ctypes.c_int32 * count)(*[_DT[g.dtype] for g in grads])
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e.args[0]}: bfloat16, float16 or float32") from None
    ptrs = P(*[g.data_ptr() for g in grads])
    numel = (ctypes.c_int64 * count)(*[g.numel() for g in grads])
    if out is None:
        outs = None
    elif out is grads:
        outs = ptrs
    else:
        if len(out) != count:
            raise ValueError("out and the gradients must have the same length")
        for g, o in zip(grads, out):
            if o.shape != g.shape or o.dtype != g.dtype or o.device != dev or not o.is_contiguous():
                raise ValueError("each out must be contiguous with its gradient's shape, dtype and device")
        outs = P(*[o.data_ptr() for o in out])
    with _on(stream, dev) as st:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        need = lib.muon_clip_workspace_bytes(count)
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        _b._check(lib.muon_clip_grads(ptrs, outs, numel, dts, count, max_norm, eps, norm.data_ptr(), ws.data_ptr(), need,
                                      st))
    return norm


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
               eps: float = 1e-6, stream=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (N + eps)), N their global norm, in place or into `out` (C-ABI
    muon_clip_grads), and returns N (a 0-d fp32 tensor on the device; nothing waits for it)."""
    return _clip(grads, float(max_norm), grads if out is None else out, float(eps), stream)


def grad_norm(grads: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
    """The global norm of the gradients as a 0-d fp32 tensor on the device."""
    return _clip(grads, 0.0, None, 0.0, stream)
