"""The operators that stand around the Muon update in a training step with 8-bit products, as measurable cases.

A step normalises the residual stream and quantises it (rms_norm), multiplies 8-bit operands whose blocks of 128
share a power-of-two scale (fp8_matmul; fp8_quantize lays weights, activations and gradients out for it, both ways),
and clips the gradients by their global norm (clip_grads) before the update.  `run` computes a case in plain torch
operations, or with `own` set through the package's entry points.

An 8-bit operand [rows, cols] is a float8 tensor whose rows are padded to a multiple of 16 bytes, with its scales
as [ceil(cols / 512), rows rounded up to 4, 4] powers of two (float8_e8m0fnu): the scale of block kb of row r is
at [kb // 4, r, kb % 4].  Scales of no row or block are 1.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # largest finite values: both 1.75 * 2^k
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # gradients of sixteen 128 x 256 fp32 matrices: the smallest model, where the launch counts
        {"name": "clip 16 small fp32", "op": "clip", "count": 16, "rows": 128, "cols": 256, "dtype": "fp32",
         "std": 1e-2, "max_norm": 1.0},
        # 48 matrices of 512 x 2048: the many-small-matrices workload
        {"name": "clip 48 middling bf16", "op": "clip", "count": 48, "rows": 512, "cols": 2048, "dtype": "bf16",
         "std": 1e-3, "max_norm": 1.0},
        # four 4096 x 14336 matrices: most of one layer of the d = 4096 model
        {"name": "clip 4 large bf16", "op": "clip", "count": 4, "rows": 4096, "cols": 14336, "dtype": "bf16",
         "std": 1e-3, "max_norm": 1.0},
        # a single token through the norm of the d = 4096 model
        {"name": "norm 1 token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "residual": True,
         "fmt": "e4m3"},
        # a training batch of 8192 tokens
        {"name": "norm 8192 tokens", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "residual": True,
         "fmt": "e4m3"},
        # its gradient, at an odd number of tokens
        {"name": "norm gradient 8191 tokens", "op": "norm_grad", "rows": 8191, "cols": 4096, "dtype": "bf16",
         "residual": True},
        # the up projection's weight after an update, for the forward product and, transposed, for the data gradient
        {"name": "quantize weight", "op": "quantize", "rows": 4096, "cols": 14336, "dtype": "bf16", "square": True,
         "fmt": "e4m3"},
        # a ragged fp32 gradient, along both axes
        {"name": "quantize ragged gradient", "op": "quantize", "rows": 1000, "cols": 1100, "dtype": "fp32",
         "square": False, "fmt": "e5m2"},
        # one token times a square projection
        {"name": "matmul 1 token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "fa": "e4m3", "fb": "e4m3",
         "out": "bf16", "add": False},
        # an odd, small product
        {"name": "matmul ragged", "op": "matmul", "m": 777, "n": 1100, "k": 1000, "fa": "e4m3", "fb": "e4m3",
         "out": "fp16", "add": False},
        # the up projection of 8192 tokens
        {"name": "matmul forward", "op": "matmul", "m": 8192, "n": 14336, "k": 4096, "fa": "e4m3", "fb": "e4m3",
         "out": "bf16", "add": False},
        # the gradient of a square projection over 8192 tokens, added to the gradient so far
        {"name": "matmul weight gradient", "op": "matmul", "m": 4096, "n": 4096, "k": 8192, "fa": "e5m2",
         "fb": "e4m3", "out": "fp32", "add": True},
    ]


def _log(rng, lo, hi):
    """A whole number, even over the logarithm; odd as often as not."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["clip", "norm", "norm_grad", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "clip":
        count, size = rng.randint(1, 48), _log(rng, 1 << 15, 4096 * 14336 * 2)
        rows = _log(rng, 1, 4096)
        return {"op": op, "count": count, "rows": rows, "cols": max(1, size // (rows * count)), "dtype": dtype,
                "std": 1e-2, "max_norm": rng.choice([0.5, 1.0, 1e4])}
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        case = {"op": op, "rows": _log(rng, 1, min(32768, 8192 * 4096 // cols)), "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.7}
        return dict(case, fmt=rng.choice(["e4m3", "e5m2"])) if op == "norm" else case
    if op == "quantize":
        cols = _log(rng, 1, 16384)
        return {"op": op, "rows": _log(rng, 1, min(32768, 4096 * 14336 // cols)), "cols": cols, "dtype": dtype,
                "square": rng.random() < 0.4, "fmt": rng.choice(["e4m3", "e5m2"])}
    n, k = _log(rng, 64, 14336), _log(rng, 64, 14336)
    return {"op": op, "m": _log(rng, 1, 8192), "n": n, "k": k, "fa": rng.choice(["e4m3", "e5m2"]),
            "fb": rng.choice(["e4m3", "e5m2"]), "out": dtype, "add": rng.random() < 0.3}


# ---------------------------------------------------------------- the 8-bit layout, in plain operations

def _pow2(e):
    """2^e of whole numbers in [-127, 127], exactly, in 32 bits (2^-127 is subnormal)."""
    n = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return n.to(torch.int32).view(torch.float32)


def _exponent(amax, fmt):
    """The smallest e with 2^e * (largest value of fmt) >= amax, of finite amax >= 0 in 32 bits; 0 for amax = 0."""
    bits = amax.view(torch.int32)
    e = ((bits + 0x1FFFFF) >> 23) - 127 - (8 if fmt == "e4m3" else 15)
    return torch.where(bits == 0, torch.zeros_like(e), e.clamp(-127, 127))


def _store_scales(e):
    """Exponents [rows, blocks] -> the scales as they are kept."""
    rows, blocks = e.shape
    rp, bp = -(-rows // 4) * 4, -(-blocks // 4) * 4
    full = torch.full((rp, bp), 127, dtype=torch.uint8, device=e.device)
    full[:rows, :blocks] = (e + 127).to(torch.uint8)
    return full.view(rp, bp // 4, 4).permute(1, 0, 2).contiguous().view(torch.float8_e8m0fnu)


def _pad_cols(x, to):
    return torch.nn.functional.pad(x, (0, -(-x.shape[1] // to) * to - x.shape[1])) if x.shape[1] % to else x


def _quantize_rows(x, fmt, e=None):
    """x [rows, cols] in 32 bits -> 8-bit data and scales, blocks of 128 columns; `e`: exponents already known."""
    rows, cols = x.shape
    xb = _pad_cols(x, BLOCK).view(rows, -1, BLOCK)
    if e is None:
        e = _exponent(xb.abs().amax(dim=2), fmt)
    q = (xb * _pow2(-e)[:, :, None]).to(FP8[fmt])
    data = _pad_cols(q.view(torch.uint8).view(rows, -1)[:, :cols], 16).view(FP8[fmt])
    return data[:, :cols], _store_scales(e)


def _square_exponents(x, fmt):
    """Exponents of the 128 x 128 blocks of x [rows, cols], one for each row and column block."""
    rows, cols = x.shape
    xp = torch.nn.functional.pad(x.abs(), (0, -cols % BLOCK, 0, -rows % BLOCK))
    t = xp.view(xp.shape[0] // BLOCK, BLOCK, xp.shape[1] // BLOCK, BLOCK).amax(dim=(1, 3))
    return _exponent(t, fmt)


def _values(data, scale):
    """What 8-bit data and scales stand for, in 32 bits."""
    rows, cols = data.shape
    s = scale.view(torch.uint8).to(torch.int32) - 127
    s = s.permute(1, 0, 2).reshape(s.shape[1], -1)[:rows, : -(-cols // BLOCK)]
    return data.to(torch.float32) * _pow2(s).repeat_interleave(BLOCK, dim=1)[:, :cols]


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=g) * std


def _operand(g, rows, cols, fmt):
    """Activations with outlying columns, or (e5m2) gradients whose rows differ in size, as 8-bit operands."""
    x = _normal(g, rows, cols)
    x *= torch.exp(_normal(g, 1, cols)) if fmt == "e4m3" else 1e-4 * torch.exp(2 * _normal(g, rows, 1))
    return _quantize_rows(x, fmt)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "clip":
        dt = DTYPES[case["dtype"]]
        s["grads"] = [_normal(g, case["rows"], case["cols"], std=case["std"]).to(dt) for _ in range(case["count"])]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
    elif op in ("norm", "norm_grad"):
        dt, rows, cols = DTYPES[case["dtype"]], case["rows"], case["cols"]
        s["weight"] = 1 + _normal(g, cols, std=0.1)
        s["residual"] = _normal(g, rows, cols).to(dt) if case["residual"] else None
        if op == "norm":
            s["x"] = (_normal(g, rows, cols) * torch.exp(_normal(g, 1, cols))).to(dt)
        else:
            s["dy"] = _normal(g, rows, cols, std=1e-3).to(dt)
            s["h"] = _normal(g, rows, cols).to(dt)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + 1e-6)
    elif op == "quantize":
        x = _normal(g, case["rows"], case["cols"], std=0.02)
        s["x"] = (x * torch.exp(2 * _normal(g, case["rows"], 1))).to(DTYPES[case["dtype"]])
    else:
        s["a"] = _operand(g, case["m"], case["k"], case["fa"])
        s["b"] = _operand(g, case["n"], case["k"], case["fb"])
        size = (30.0, 0.1, 1e-5)[(case["fa"] == "e5m2") + (case["fb"] == "e5m2")]  # about the product's own
        s["add"] = _normal(g, case["m"], case["n"], std=size).to(DTYPES[case["out"]]) if case["add"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _plain_clip(s):
    square = [g.float().square().sum() for g in s["grads"]]
    norm = torch.stack(square).sum().sqrt()
    coef = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    return [norm] + [(g.float() * coef).to(g.dtype) for g in s["grads"]]


def _plain_norm(s):
    x = s["x"].float()
    h = x if s["residual"] is None else x + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(dim=1) + 1e-6)
    y = h * rstd[:, None] * s["weight"]
    data, scale = _quantize_rows(y, s["case"]["fmt"])
    return {"y": y.to(s["x"].dtype), "h": h.to(s["x"].dtype), "rstd": rstd, "data": data, "scale": scale}


def _plain_norm_grad(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["weight"]
    xhat = h * rstd
    dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(s["dy"].dtype), "dweight": (dy * xhat).sum(dim=0)}


def _plain_quantize(s):
    x, fmt = s["x"].float(), s["case"]["fmt"]
    if s["case"]["square"]:
        e = _square_exponents(x, fmt)
        by_row = e.repeat_interleave(BLOCK, dim=0)[: x.shape[0]]
        by_col = e.t().repeat_interleave(BLOCK, dim=0)[: x.shape[1]]
    else:
        by_row = by_col = None
    rows, cols = _quantize_rows(x, fmt, by_row), _quantize_rows(x.t().contiguous(), fmt, by_col)
    return {"data": rows[0], "scale": rows[1], "data_t": cols[0], "scale_t": cols[1]}


def _plain_matmul(s):
    c = _values(*s["a"]) @ _values(*s["b"]).t()
    if s["add"] is not None:
        c = c + s["add"].float()
    return c.to(DTYPES[s["case"]["out"]])


def _package():
    import newton_schulz_04_gb300
    return newton_schulz_04_gb300


def _own_clip(s):
    return [_package().clip_grads(s["grads"], s["case"]["max_norm"], out=s["out"])] + s["out"]


def _own_norm(s):
    r = _package().rms_norm(s["x"], s["weight"], residual=s["residual"], fp8=s["case"]["fmt"])
    return {"y": r.y, "h": r.h, "rstd": r.rstd, "data": r.q.data, "scale": r.q.scale}


def _own_norm_grad(s):
    dx, dweight = _package().rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dresidual=s["residual"])
    return {"dx": dx, "dweight": dweight}


def _own_quantize(s):
    q, qt = _package().fp8_quantize(s["x"], fmt=s["case"]["fmt"], square=s["case"]["square"], rows=True, cols=True)
    return {"data": q.data, "scale": q.scale, "data_t": qt.data, "scale_t": qt.scale}


def _own_matmul(s):
    p = _package()
    return p.fp8_matmul(p.Fp8Tensor(*s["a"]), p.Fp8Tensor(*s["b"]), out_dtype=DTYPES[s["case"]["out"]], add=s["add"])


_plain = {"clip": _plain_clip, "norm": _plain_norm, "norm_grad": _plain_norm_grad, "quantize": _plain_quantize,
          "matmul": _plain_matmul}
_own = {"clip": _own_clip, "norm": _own_norm, "norm_grad": _own_norm_grad, "quantize": _own_quantize,
        "matmul": _own_matmul}


# ---------------------------------------------------------------- what a pass cannot do without

def _fp8_bytes(rows, cols):
    return rows * cols + rows * -(-cols // BLOCK)


def work(case):
    op = case["op"]
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        out = m * n * BYTES[case["out"]] * (2 if case["add"] else 1)
        return {"bytes": _fp8_bytes(m, k) + _fp8_bytes(n, k) + out, "flops": 2 * m * n * k}
    rows, cols, size = case["rows"], case["cols"], BYTES[case["dtype"]]
    n = rows * cols
    if op == "clip":
        return {"bytes": 2 * case["count"] * n * size + 4, "flops": 3 * case["count"] * n}
    if op == "norm":  # x in, y and the 8-bit copy out; with a residual that in and the sum out
        return {"bytes": n * size * (4 if case["residual"] else 2) + _fp8_bytes(rows, cols) + 4 * rows + 4 * cols,
                "flops": 8 * n}
    if op == "norm_grad":
        return {"bytes": n * size * (4 if case["residual"] else 3) + 4 * rows + 8 * cols, "flops": 12 * n}
    return {"bytes": n * size + _fp8_bytes(rows, cols) + _fp8_bytes(cols, rows), "flops": 6 * n}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _two64(e):
    """2^e, exactly, from the bits of a 64-bit number."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round8(v, fmt):
    """v rounded to the nearest value of fmt, ties to even: 3 bits after the point down to 2^-6, or 2 to 2^-14."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, p = torch.frexp(v)
    step = _two64(torch.clamp(p - 1, min=low) - bits)
    return torch.round(v / step) * step


def _scale64(amax, fmt):
    m, p = torch.frexp(amax / TOP[fmt])
    e = torch.where(m == 0.5, p - 1, p).clamp(-127, 127)
    return _two64(torch.where(amax == 0, torch.zeros_like(e), e))


def _kept64(scale):
    """Scales [rows, blocks] in the order in which they are kept, the gaps filled with 1."""
    rows, blocks = scale.shape
    out = torch.ones(-(-blocks // 4), -(-rows // 4) * 4, 4, dtype=torch.float64, device=scale.device)
    kb = torch.arange(blocks, device=scale.device)
    out[kb // 4, :rows, kb % 4] = scale.t()
    return out


def _blocks64(x, down):
    """The largest magnitude of each block of `down` rows x 128 columns."""
    return torch.nn.functional.max_pool2d(x.abs()[None], (down, BLOCK), ceil_mode=True)[0]


def _quantized64(x, fmt, down):
    scale = _scale64(_blocks64(x, down), fmt)
    scale = scale.repeat_interleave(down, dim=0)[: x.shape[0]]
    wide = scale.repeat_interleave(BLOCK, dim=1)[:, : x.shape[1]]
    return _round8(x / wide, fmt), _kept64(scale)


def _value64(data, scale):
    rows, cols = data.shape
    kb = torch.arange(cols, device=data.device) // BLOCK
    return data.to(torch.float32).double() * scale.to(torch.float32).double()[kb // 4, :rows, kb % 4].t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.dot(g.double().view(-1), g.double().view(-1))) for g in s["grads"]))
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        return [torch.tensor(norm, dtype=torch.float64)] + [g.double() * coef for g in s["grads"]]
    if op == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        rstd = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"] + 1e-6) ** -0.5
        y = h * (rstd[:, None] * s["weight"].double())
        data, scale = _quantized64(y, case["fmt"], 1)
        return {"y": y, "h": h, "rstd": rstd, "data": data, "scale": scale}
    if op == "norm_grad":
        # y = r(h) h w with dr/dh = -r^3 h / cols
        dy, h, r = s["dy"].double(), s["h"].double(), s["rstd"].double()[:, None]
        along = torch.einsum("ij,ij,j->i", dy, h, s["weight"].double())[:, None]
        dx = dy * s["weight"].double() * r - h * r ** 3 * along / case["cols"]
        if s["residual"] is not None:
            dx = dx + s["residual"].double()
        return {"dx": dx, "dweight": torch.einsum("ij,ij,i->j", dy, h, r[:, 0])}
    if op == "quantize":
        x, down = s["x"].double(), BLOCK if case["square"] else 1
        q, qt = _quantized64(x, case["fmt"], down), _quantized64(x.t().contiguous(), case["fmt"], down)
        return {"data": q[0], "scale": q[1], "data_t": qt[0], "scale_t": qt[1]}
    c = torch.einsum("mk,nk->mn", _value64(*s["a"]), _value64(*s["b"]))
    return c if s["add"] is None else c + s["add"].double()
