"""The operators around a block of a residual network trained with 8-bit checkpoints, as measurable cases.

A block reads the normalised residual stream and its output joins the stream through a norm, a gate and a scale of its own;
the next block's norm follows in the same pass (block_norm, block_norm_backward).  Within the block stands the product of
an activation and a linear branch (gated_activation, gated_activation_backward).  What the backward pass needs of the
forward one is kept in 8 bits: both forward operators write such copies, both gradients read them, and fp8_transpose lays
one out as the operand of a weight gradient, which is summed over the tokens.  `run` computes a case in plain torch
operations, or with `own` set through the package's entry points.

An 8-bit matrix [rows, cols] is a float8 tensor whose rows are padded to a multiple of 16 bytes, with its scales as
[ceil(cols / 512), rows rounded up to 4, 4] powers of two (float8_e8m0fnu): the scale of block kb of row r is at
[kb // 4, r, kb % 4].  Scales of no row or block are 1.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}  # largest finite values: both 1.75 * 2^k
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one generated token past a block of the d = 4096 model: 8-bit input of the next product, nothing kept
        {"name": "block norm 1 token", "op": "norm", "rows": 1, "cols": 4096, "dtype": "bf16", "gate": "element",
         "scale": True, "alpha": 1.0, "fmt": "e4m3", "y": False, "kept": "none"},
        # the tokens and width of the package's example of a training step, with a gate for each token
        {"name": "block norm 2048 x 512", "op": "norm", "rows": 2048, "cols": 512, "dtype": "bf16", "gate": "token",
         "scale": False, "alpha": 1.0, "fmt": "e4m3", "y": True, "kept": "e4m3"},
        # a training batch of 8192 tokens with its checkpoints
        {"name": "block norm 8192 tokens", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "gate": "element",
         "scale": True, "alpha": 1.0, "fmt": "e4m3", "y": False, "kept": "e4m3"},
        # a ragged fp32 stream without gate, scaled down, its gradient from what was kept in 32 bits
        {"name": "block norm gradient ragged", "op": "norm_grad", "rows": 1000, "cols": 1100, "dtype": "fp32",
         "gate": "none", "scale": True, "alpha": 0.5, "kept": "none", "dh": True},
        # the gradient of the training batch, at an odd number of tokens, from 8-bit checkpoints
        {"name": "block norm gradient 8191", "op": "norm_grad", "rows": 8191, "cols": 4096, "dtype": "bf16",
         "gate": "element", "scale": True, "alpha": 1.0, "kept": "e4m3", "dh": True},
        # one generated token between the block's products
        {"name": "gated 1 token", "op": "gated", "rows": 1, "cols": 14336, "dtype": "bf16", "act": "silu",
         "fmt": "e4m3", "y": False, "kept": "none"},
        # the training batch between the block's products: an 8-bit operand and the checkpoints of both branches
        {"name": "gated 8192 tokens", "op": "gated", "rows": 8192, "cols": 14336, "dtype": "bf16", "act": "silu",
         "fmt": "e4m3", "y": False, "kept": "e4m3"},
        # an odd, small gradient kept and returned in 16 bits
        {"name": "gated gradient ragged", "op": "gated_grad", "rows": 777, "cols": 1101, "dtype": "fp16", "act": "gelu",
         "kept": "none", "dense": True, "fmt": "none", "y_fmt": "none"},
        # the training batch's gradient from the checkpoints: 8-bit operands of the four products that follow, and the
        # activation again as the operand of the down projection's weight gradient
        {"name": "gated gradient 8192 tokens", "op": "gated_grad", "rows": 8192, "cols": 14336, "dtype": "bf16",
         "act": "silu", "kept": "e4m3", "dense": False, "fmt": "e5m2", "y_fmt": "e4m3"},
        # a checkpoint of the training batch as a weight gradient's operand
        {"name": "transpose 8192 x 4096", "op": "transpose", "rows": 8192, "cols": 4096, "kept": "e4m3"},
        # a ragged one, small
        {"name": "transpose ragged", "op": "transpose", "rows": 1001, "cols": 1100, "kept": "e5m2"},
    ]


def _log(rng, lo, hi):
    """A whole number, even over the logarithm; odd as often as not."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated_grad", "transpose"])
    dtype, kept = rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice(["none", "e4m3", "e4m3", "e5m2"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        case = {"op": op, "rows": _log(rng, 1, min(32768, 8192 * 4096 // cols)), "cols": cols, "dtype": dtype,
                "gate": rng.choice(["none", "token", "element", "element"]), "scale": rng.random() < 0.7,
                "alpha": rng.choice([1.0, 1.0, 0.5]), "kept": kept}
        if op == "norm":
            fmt = rng.choice(["none", "e4m3", "e5m2"])
            return dict(case, fmt=fmt, y=fmt == "none" or rng.random() < 0.5)
        return dict(case, dh=rng.random() < 0.8)
    cols = _log(rng, 64, 16384)
    rows = _log(rng, 1, min(32768, 8192 * 4096 // cols))
    if op == "transpose":
        return {"op": op, "rows": rows, "cols": cols, "kept": rng.choice(["e4m3", "e5m2"])}
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "act": rng.choice(["silu", "silu", "gelu"]),
            "kept": kept}
    if op == "gated":
        fmt = rng.choice(["none", "e4m3", "e5m2"])
        return dict(case, fmt=fmt, y=fmt == "none" or rng.random() < 0.5)
    fmt = rng.choice(["none", "e4m3", "e5m2"])
    return dict(case, dense=fmt == "none" or rng.random() < 0.3, fmt=fmt, y_fmt=rng.choice(["none", "e4m3"]))


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


def _quantize(x, fmt):
    """x [rows, cols] in 32 bits -> 8-bit data and scales, blocks of 128 columns."""
    rows, cols = x.shape
    xb = _pad_cols(x, BLOCK).view(rows, -1, BLOCK)
    e = _exponent(xb.abs().amax(dim=2), fmt)
    q = (xb * _pow2(-e)[:, :, None]).to(FP8[fmt])
    data = _pad_cols(q.view(torch.uint8).view(rows, -1)[:, :cols], 16).view(FP8[fmt])
    return data[:, :cols], _store_scales(e)


def _values(data, scale):
    """What 8-bit data and scales stand for, in 32 bits."""
    rows, cols = data.shape
    s = scale.view(torch.uint8).to(torch.int32) - 127
    s = s.permute(1, 0, 2).reshape(s.shape[1], -1)[:rows, : -(-cols // BLOCK)]
    return data.to(torch.float32) * _pow2(s).repeat_interleave(BLOCK, dim=1)[:, :cols]


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=g) * std


def _keep(x, case):
    """What a forward pass left for the backward pass: 8-bit data with scales, or the tensor in its type."""
    return x.to(DTYPES[case["dtype"]]) if case["kept"] == "none" else _quantize(x, case["kept"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, op, rows, cols = {"case": case}, case["op"], case["rows"], case["cols"]
    if op == "transpose":  # activations with outlying columns, or gradients whose rows differ in size
        x = _normal(g, rows, cols)
        x *= torch.exp(_normal(g, 1, cols)) if case["kept"] == "e4m3" else 1e-4 * torch.exp(2 * _normal(g, rows, 1))
        s["q"] = _quantize(x, case["kept"])
        return s
    dt = DTYPES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        s["post"], s["pre"] = 1 + _normal(g, cols, std=0.1), 1 + _normal(g, cols, std=0.1)
        s["scale"] = 0.5 + _normal(g, cols, std=0.1) if case["scale"] else None
        x = _normal(g, rows, cols) * torch.exp(_normal(g, 1, cols))
        gate = None
        if case["gate"] != "none":
            gate = _normal(g, rows, 1 if case["gate"] == "token" else cols, std=2.0)
    if op == "norm":
        s["x"], s["residual"] = x.to(dt), _normal(g, rows, cols).to(dt)
        s["gate"] = None if gate is None else gate.to(dt)
    elif op == "norm_grad":
        h = _normal(g, rows, cols)
        s["rx"], s["rh"] = (torch.rsqrt(v.square().mean(dim=1) + EPS) for v in (x, h))
        s["x"], s["h"] = _keep(x, case), _keep(h, case)
        s["gate"] = None if gate is None else gate.to(dt) if case["gate"] == "token" else _keep(gate, case)
        s["dy"] = _normal(g, rows, cols, std=1e-3).to(dt)
        s["dh"] = _normal(g, rows, cols, std=1e-3).to(dt) if case["dh"] else None
    elif op == "gated":
        s["gate"], s["up"] = (2 * _normal(g, rows, cols)).to(dt), _normal(g, rows, cols).to(dt)
    else:
        s["gate"], s["up"] = _keep(2 * _normal(g, rows, cols), case), _keep(_normal(g, rows, cols), case)
        s["dy"] = (1e-3 * _normal(g, rows, cols) * torch.exp(_normal(g, rows, 1))).to(dt)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _read(kept):
    return _values(*kept) if isinstance(kept, tuple) else kept.float()


def _put(out, name, x, fmt):
    out[name], out[name + "_scale"] = _quantize(x, fmt)


def _sigmoid(g):
    return 1 / (1 + torch.exp(-g))


def _plain_norm(s):
    case, dt, out = s["case"], DTYPES[s["case"]["dtype"]], {}
    x, r = s["x"].float(), s["residual"].float()
    rx = torch.rsqrt(x.square().mean(dim=1) + EPS)
    v = x * rx[:, None] * s["post"]
    if s["scale"] is not None:
        v = v * s["scale"]
    if s["gate"] is not None:
        v = v * _sigmoid(s["gate"].float())
    h = case["alpha"] * r + v
    rh = torch.rsqrt(h.square().mean(dim=1) + EPS)
    y = h * rh[:, None] * s["pre"]
    out["h"], out["rstd_x"], out["rstd_h"] = h.to(dt), rx, rh
    if case["y"]:
        out["y"] = y.to(dt)
    if case["fmt"] != "none":
        _put(out, "q", y, case["fmt"])
    if case["kept"] != "none":
        _put(out, "kept_x", x, case["kept"])
        _put(out, "kept_h", h, case["kept"])
        if case["gate"] == "element":
            _put(out, "kept_gate", s["gate"].float(), case["kept"])
    return out


def _plain_norm_grad(s):
    case, dt, out = s["case"], DTYPES[s["case"]["dtype"]], {}
    dy, x, h = s["dy"].float(), _read(s["x"]) * s["rx"][:, None], _read(s["h"]) * s["rh"][:, None]
    a = dy * s["pre"]
    d = s["rh"][:, None] * (a - h * (a * h).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        d = d + s["dh"].float()
    out["dresidual"] = (case["alpha"] * d).to(dt)
    sig = None if s["gate"] is None else _sigmoid(_read(s["gate"]))
    t = d if sig is None else d * sig
    weight = s["post"] if s["scale"] is None else s["post"] * s["scale"]
    b = t * weight
    along = b * x
    out["dx"] = (s["rx"][:, None] * (b - x * along.mean(dim=1, keepdim=True))).to(dt)
    if sig is not None:
        out["dgate"] = ((1 - sig) * (along.sum(dim=1, keepdim=True) if case["gate"] == "token" else along)).to(dt)
    per_column = (t * x).sum(dim=0)
    out["dpost"] = per_column if s["scale"] is None else per_column * s["scale"]
    out["dpre"] = (dy * h).sum(dim=0)
    if s["scale"] is not None:
        out["dscale"] = per_column * s["post"]
    return out


def _phi(g):
    """The normal distribution's function, exact in its lower tail too."""
    return 0.5 * torch.erfc(g * -math.sqrt(0.5))


def _plain_gated(s):
    case, out = s["case"], {}
    g, u = s["gate"].float(), s["up"].float()
    y = (g * _sigmoid(g) if case["act"] == "silu" else g * _phi(g)) * u
    if case["y"]:
        out["y"] = y.to(DTYPES[case["dtype"]])
    if case["fmt"] != "none":
        _put(out, "q", y, case["fmt"])
    if case["kept"] != "none":
        _put(out, "kept_gate", g, case["kept"])
        _put(out, "kept_up", u, case["kept"])
    return out


def _plain_gated_grad(s):
    case, dt, out = s["case"], DTYPES[s["case"]["dtype"]], {}
    dy, g, u = s["dy"].float(), _read(s["gate"]), _read(s["up"])
    if case["act"] == "silu":
        sig = _sigmoid(g)
        act = g * sig
        slope = sig * (1 + g * (1 - sig))
    else:
        phi = _phi(g)
        act = g * phi
        slope = phi + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    dgate, dup = dy * u * slope, dy * act
    if case["dense"]:
        out["dgate"], out["dup"] = dgate.to(dt), dup.to(dt)
    if case["fmt"] != "none":
        _put(out, "dgate_rows", dgate, case["fmt"])
        _put(out, "dgate_cols", dgate.t().contiguous(), case["fmt"])
        _put(out, "dup_rows", dup, case["fmt"])
        _put(out, "dup_cols", dup.t().contiguous(), case["fmt"])
    if case["y_fmt"] != "none":
        _put(out, "y_cols", (act * u).t().contiguous(), case["y_fmt"])
    return out


def _plain_transpose(s):
    data, scale = _quantize(_values(*s["q"]).t().contiguous(), s["case"]["kept"])
    return {"data": data, "scale": scale}


def _package():
    import newton_schulz_04_gb300
    return newton_schulz_04_gb300


def _own_kept(p, kept):
    return p.Fp8Tensor(*kept) if isinstance(kept, tuple) else kept


def _own_put(out, name, q):
    if q is not None:
        out[name], out[name + "_scale"] = q.data, q.scale


def _fmt(name):
    return None if name == "none" else name


def _own_norm(s):
    case = s["case"]
    r = _package().block_norm(s["x"], s["residual"], s["post"], s["pre"], gate=s["gate"], scale=s["scale"],
                              alpha=case["alpha"], eps=EPS, fp8=_fmt(case["fmt"]), y=case["y"],
                              checkpoint=_fmt(case["kept"]))
    out = {"h": r.h, "rstd_x": r.kept.rstd_x, "rstd_h": r.kept.rstd_h}
    if case["y"]:
        out["y"] = r.y
    _own_put(out, "q", r.q)
    if case["kept"] != "none":
        _own_put(out, "kept_x", r.kept.x)
        _own_put(out, "kept_h", r.kept.h)
        if case["gate"] == "element":
            _own_put(out, "kept_gate", r.kept.gate)
    return out


def _own_norm_grad(s):
    p, case = _package(), s["case"]
    kept = p.BlockNormKept(_own_kept(p, s["x"]), _own_kept(p, s["h"]), _own_kept(p, s["gate"]), s["rx"], s["rh"])
    r = p.block_norm_backward(s["dy"], kept, s["post"], s["pre"], scale=s["scale"], alpha=case["alpha"], dh=s["dh"])
    out = {"dx": r.dx, "dresidual": r.dresidual, "dpost": r.dpost_weight, "dpre": r.dpre_weight}
    if s["gate"] is not None:
        out["dgate"] = r.dgate
    if s["scale"] is not None:
        out["dscale"] = r.dscale
    return out


def _own_gated(s):
    case, out = s["case"], {}
    r = _package().gated_activation(s["gate"], s["up"], activation=case["act"], fp8=_fmt(case["fmt"]), y=case["y"],
                                    checkpoint=_fmt(case["kept"]))
    if case["y"]:
        out["y"] = r.y
    _own_put(out, "q", r.q)
    if case["kept"] != "none":
        _own_put(out, "kept_gate", r.kept.gate)
        _own_put(out, "kept_up", r.kept.up)
    return out


def _own_gated_grad(s):
    p, case, out = _package(), s["case"], {}
    kept = p.GatedKept(_own_kept(p, s["gate"]), _own_kept(p, s["up"]))
    r = p.gated_activation_backward(s["dy"], kept, activation=case["act"], dense=case["dense"], fp8=_fmt(case["fmt"]),
                                    y_fp8=_fmt(case["y_fmt"]))
    if case["dense"]:
        out["dgate"], out["dup"] = r.dgate, r.dup
    if case["fmt"] != "none":
        _own_put(out, "dgate_rows", r.dgate_rows)
        _own_put(out, "dgate_cols", r.dgate_cols)
        _own_put(out, "dup_rows", r.dup_rows)
        _own_put(out, "dup_cols", r.dup_cols)
    _own_put(out, "y_cols", r.y_cols)
    return out


def _own_transpose(s):
    p = _package()
    r = p.fp8_transpose(p.Fp8Tensor(*s["q"]))
    return {"data": r.data, "scale": r.scale}


_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "gated": _plain_gated, "gated_grad": _plain_gated_grad,
          "transpose": _plain_transpose}
_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "gated": _own_gated, "gated_grad": _own_gated_grad,
        "transpose": _own_transpose}


# ---------------------------------------------------------------- what a pass cannot do without

def _fp8_bytes(rows, cols):
    return rows * cols + rows * -(-cols // BLOCK)


def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    n, by_rows, by_cols = rows * cols, _fp8_bytes(rows, cols), _fp8_bytes(cols, rows)
    if op == "transpose":
        return {"bytes": by_rows + by_cols, "flops": 3 * n}
    size = BYTES[case["dtype"]]
    eight = case["kept"] != "none"
    if op in ("norm", "norm_grad"):
        vectors, token = 4 * cols * (3 if case["scale"] else 2), rows * size if case["gate"] == "token" else 0
        element = case["gate"] == "element"
        if op == "norm":  # x, the stream and the gate in, the stream out, then what was asked for
            moved = n * size * (3 + element + case["y"]) + (by_rows if case["fmt"] != "none" else 0)
            moved += by_rows * (2 + element) if eight else 0
            return {"bytes": moved + token + 8 * rows + vectors, "flops": 24 * n}
        kept = (2 + element) * (by_rows if eight else n * size)
        moved = kept + n * size * (3 + case["dh"] + element)
        return {"bytes": moved + 2 * token + 8 * rows + 2 * vectors, "flops": 32 * n}
    if op == "gated":
        moved = n * size * (2 + case["y"]) + (by_rows if case["fmt"] != "none" else 0) + (2 * by_rows if eight else 0)
        return {"bytes": moved, "flops": 16 * n}
    moved = n * size * (1 + 2 * case["dense"]) + 2 * (by_rows if eight else n * size)
    moved += 2 * (by_rows + by_cols) if case["fmt"] != "none" else 0
    return {"bytes": moved + (by_cols if case["y_fmt"] != "none" else 0), "flops": 24 * n}


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


def _put64(out, name, x, fmt):
    """x in 8 bits: the scales from each block's largest magnitude, and the rounded quotients."""
    rows, cols = x.shape
    amax = torch.nn.functional.max_pool2d(x.abs()[None], (1, BLOCK), ceil_mode=True)[0]
    m, p = torch.frexp(amax / TOP[fmt])
    e = torch.where(m == 0.5, p - 1, p).clamp(-127, 127)
    scale = _two64(torch.where(amax == 0, torch.zeros_like(e), e))
    kept = torch.ones(-(-scale.shape[1] // 4), -(-rows // 4) * 4, 4, dtype=torch.float64, device=x.device)
    kb = torch.arange(scale.shape[1], device=x.device)
    kept[kb // 4, :rows, kb % 4] = scale.t()
    out[name], out[name + "_scale"] = _round8(x / scale.repeat_interleave(BLOCK, dim=1)[:, :cols], fmt), kept


def _read64(kept):
    if not isinstance(kept, tuple):
        return kept.double()
    data, scale = kept
    rows, cols = data.shape
    kb = torch.arange(cols, device=data.device) // BLOCK
    return data.to(torch.float32).double() * scale.to(torch.float32).double()[kb // 4, :rows, kb % 4].t()


def _exact_norm(s, case):
    out, n = {}, case["cols"]
    x = s["x"].double()
    rx = (torch.linalg.vector_norm(x, dim=1) ** 2 / n + EPS) ** -0.5
    weight = s["post"].double() * (1 if s["scale"] is None else s["scale"].double())
    v = torch.einsum("ij,i,j->ij", x, rx, weight)
    if s["gate"] is not None:
        v = v / (1 + torch.exp(-s["gate"].double()))
    h = v + s["residual"].double() * case["alpha"]
    rh = (torch.linalg.vector_norm(h, dim=1) ** 2 / n + EPS) ** -0.5
    y = torch.einsum("ij,i,j->ij", h, rh, s["pre"].double())
    out["h"], out["rstd_x"], out["rstd_h"] = h, rx, rh
    if case["y"]:
        out["y"] = y
    if case["fmt"] != "none":
        _put64(out, "q", y, case["fmt"])
    if case["kept"] != "none":
        _put64(out, "kept_x", x, case["kept"])
        _put64(out, "kept_h", h, case["kept"])
        if case["gate"] == "element":
            _put64(out, "kept_gate", s["gate"].double(), case["kept"])
    return out


def _exact_norm_grad(s, case):
    # y = rh(h) h pre with drh/dh = -rh^3 h / n;  h = alpha residual + sig(gate) scale post rx(x) x, drx/dx alike
    out, n = {}, case["cols"]
    dy, x, h, pre, post = s["dy"].double(), _read64(s["x"]), _read64(s["h"]), s["pre"].double(), s["post"].double()
    rx, rh = s["rx"].double()[:, None], s["rh"].double()[:, None]
    scale = torch.ones_like(post) if s["scale"] is None else s["scale"].double()
    stream = dy * pre * rh - h * rh ** 3 * torch.einsum("ij,ij,j->i", dy, h, pre)[:, None] / n
    if s["dh"] is not None:
        stream = stream + s["dh"].double()
    out["dresidual"] = stream * case["alpha"]
    sig = torch.ones_like(x) if s["gate"] is None else torch.sigmoid(_read64(s["gate"])).expand_as(x)
    branch = stream * sig
    along = torch.einsum("ij,ij,j->i", branch, x, post * scale)[:, None]
    out["dx"] = branch * (post * scale) * rx - x * rx ** 3 * along / n
    if s["gate"] is not None:  # d sig = sig (1 - sig)
        full = stream * (sig * (1 - sig)) * (x * rx) * (post * scale)
        out["dgate"] = full.sum(dim=1, keepdim=True) if case["gate"] == "token" else full
    sums = torch.einsum("ij,ij,i->j", branch, x, rx[:, 0])
    out["dpost"] = sums * scale
    out["dpre"] = torch.einsum("ij,ij,i->j", dy, h, rh[:, 0])
    if s["scale"] is not None:
        out["dscale"] = sums * post
    return out


def _exact_act(g, act):
    """(value, slope) of the activation."""
    if act == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig + g * sig * torch.sigmoid(-g)
    phi = torch.special.ndtr(g)
    return g * phi, phi + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    op, out = case["op"], {}
    if op == "norm":
        return _exact_norm(s, case)
    if op == "norm_grad":
        return _exact_norm_grad(s, case)
    if op == "transpose":
        _put64(out, "data", _read64(s["q"]).t().contiguous(), case["kept"])
        return {"data": out["data"], "scale": out["data_scale"]}
    g, u = _read64(s["gate"]), _read64(s["up"])
    value, slope = _exact_act(g, case["act"])
    if op == "gated":
        if case["y"]:
            out["y"] = value * u
        if case["fmt"] != "none":
            _put64(out, "q", value * u, case["fmt"])
        if case["kept"] != "none":
            _put64(out, "kept_gate", g, case["kept"])
            _put64(out, "kept_up", u, case["kept"])
        return out
    dy = s["dy"].double()
    if case["dense"]:
        out["dgate"], out["dup"] = dy * u * slope, dy * value
    if case["fmt"] != "none":
        for name, v in (("dgate", dy * u * slope), ("dup", dy * value)):
            _put64(out, name + "_rows", v, case["fmt"])
            _put64(out, name + "_cols", v.t().contiguous(), case["fmt"])
    if case["y_fmt"] != "none":
        _put64(out, "y_cols", (value * u).t().contiguous(), case["y_fmt"])
    return out
