"""Gradient clipping, the RMS norm and its gradient, 8-bit quantisation and the 8-bit product: pins of the 64-bit
oracle and the refusals (CPU), and the kernels against the oracle (GPU).

Tolerances.  An output of type T carries one rounding, U[T] of its value.  A sum of n terms in fp32 is off by at most
n 2^-24 of the sum of the terms' magnitudes (2^-23 where the tensor core truncates); n is the longest chain that the
kernel can have, not the one that it has at that size.  8-bit data and scales of a quantised matrix are exact."""
import ctypes
import math

import pytest
import torch

import oracle.training as ref

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # bf16: 8 significant bits
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
F24 = 2.0 ** -24
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm():
    from newton_schulz_04_gb300 import build as b
    b.build()
    import newton_schulz_04_gb300 as m
    m.load()
    return m


def gen(seed, *shape, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32) * std


def close(got, want, tol):
    got, want = got.cpu().double(), want.double()
    bad = (got - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() - tol).max()):.3g}"


# ---------------------------------------------------------------- pins of the oracle

def test_round8_keeps_the_types_own_values():
    for fmt, dt in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        v = torch.arange(256, dtype=torch.uint8).view(dt).float().double()
        v = v[torch.isfinite(v)]
        assert torch.equal(ref.round8(v, fmt), v)
        assert float(v.max()) == ref.TOP[fmt]
        # midpoints go to the even neighbour, as torch's own conversion says
        s = torch.unique(v)
        mid = (s[1:] + s[:-1]) / 2
        assert torch.equal(ref.round8(mid, fmt), mid.float().to(dt).float().double())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_exponent_is_the_smallest_that_fits(fmt):
    top = ref.TOP[fmt]
    a = torch.tensor([top, top * (1 + 2.0 ** -40), top * 8, 1.0, 1e-30, 0.0, top * 2.0 ** -5, 3e38], dtype=torch.float64)
    e = ref.exponent8(a, fmt)
    assert e.tolist()[:3] == [0, 1, 3] and int(e[5]) == 0 and int(e[6]) == -5
    nz = a > 0
    assert bool((a[nz] <= top * 2.0 ** e[nz].double()).all())
    assert bool((a[nz] > top * 2.0 ** (e[nz].double() - 1)).all())


def test_oracle_gradient_matches_differences():
    x, w, v, t = gen(1, 3, 17).double(), gen(2, 17).double(), gen(3, 3, 17).double(), gen(4, 3, 17).double()
    loss = lambda x, w: float((ref.rms_norm(x, w)[0] * v).sum() + (x * t).sum())  # noqa: E731
    _, h, rstd = ref.rms_norm(x, w)
    dx, dw = ref.rms_norm_backward(v, h, w, rstd, t)
    eps = 1e-6
    for i in (0, 7, 16):
        d = torch.zeros_like(x)
        d[1, i] = eps
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * eps) - float(dx[1, i])) < 1e-7
        d = torch.zeros_like(w)
        d[i] = eps
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * eps) - float(dw[i])) < 1e-7


def test_oracle_clip_reaches_the_norm():
    g = [gen(5, 10, 3), gen(6, 4)]
    norm, out = ref.clip_grads(g, 0.25, eps=0.0)
    assert abs(sum(float((o ** 2).sum()) for o in out) ** 0.5 - 0.25) < 1e-14
    assert ref.clip_grads(g, 2 * norm)[1][0].equal(g[0].double())


# ---------------------------------------------------------------- refusals (no GPU)

A, B_, C_, D_, E_ = (1 << 30, 1 << 31, 1 << 32, 1 << 33, 1 << 34)  # far apart, never read


def _clip_call(mm, **kw):
    P, n = ctypes.c_void_p * 1, ctypes.c_int64 * 1
    g, o = kw.get("g", A), kw.get("o", B_)
    return mm.load().muon_clip_grads(
        None if g is None else P(g), None if o is None else P(o), n(kw.get("n", 64)),
        (ctypes.c_int32 * 1)(kw.get("dt", 1)), kw.get("count", 1), kw.get("max", 1.0), kw.get("eps", 1e-6),
        kw.get("norm", C_), kw.get("ws", D_), kw.get("bytes", 1 << 20), None)


def test_clip_refuses(mm):
    assert _clip_call(mm, count=-1) == 1
    assert _clip_call(mm, g=None) == 1
    assert _clip_call(mm, g=0) == 1                              # NULL gradient of a non-empty tensor
    assert _clip_call(mm, o=0) == 1
    assert _clip_call(mm, o=None, norm=None) == 1                # nothing to do
    assert _clip_call(mm, dt=3) == 1
    assert _clip_call(mm, max=-1.0) == 1
    assert _clip_call(mm, max=math.nan) == 1
    assert _clip_call(mm, eps=-1.0) == 1
    assert _clip_call(mm, eps=math.inf) == 1
    assert _clip_call(mm, ws=None) == 1
    assert _clip_call(mm, o=A + 128) == 1                        # partly overlapping
    assert _clip_call(mm, o=D_) == 1                             # the workspace
    assert _clip_call(mm, n=-1) == 2
    assert _clip_call(mm, g=A + 2) == 3
    assert _clip_call(mm, norm=C_ + 1) == 3
    assert _clip_call(mm, ws=D_ + 4) == 3
    assert _clip_call(mm, bytes=64) == 4
    assert "workspace" in mm.load().muon_last_error().decode()


def _norm_call(mm, **kw):
    g = lambda k, d: kw.get(k, d)  # noqa: E731
    return mm.load().muon_rms_norm(g("x", A), g("ldx", 64), g("r", None), g("ldr", 64), g("w", None), g("wdt", 1),
                                   g("rows", 4), g("cols", 64), g("eps", 1e-6), g("y", B_), g("ldy", 64), g("h", None), 64,
                                   None, g("q", None), g("ldq", 64), g("qs", None), g("fmt", 0), g("dt", 0), None)


def test_rms_norm_refuses(mm):
    for kw in (dict(x=None), dict(y=None), dict(dt=5), dict(w=C_, wdt=9), dict(eps=-1.0), dict(eps=math.nan),
               dict(q=C_), dict(qs=C_), dict(q=C_, qs=D_, fmt=2), dict(y=A + 64), dict(y=B_, h=B_ + 128)):
        assert _norm_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=65537), dict(rows=4194305), dict(ldx=63), dict(ldy=10),
               dict(q=C_, qs=D_, ldq=48)):
        assert _norm_call(mm, **kw) == 2, kw
    for kw in (dict(x=A + 1), dict(y=B_ + 1), dict(w=C_ + 2), dict(q=C_ + 8, qs=D_), dict(q=C_, qs=D_, ldq=72)):
        assert _norm_call(mm, **kw) == 3, kw
    assert _norm_call(mm, rows=0) == 0


def _back_call(mm, **kw):
    g = lambda k, d: kw.get(k, d)  # noqa: E731
    return mm.load().muon_rms_norm_backward(g("dy", A), g("lddy", 64), g("h", B_), 64, None, 0, g("rstd", C_), g("dres", None),
                                            64, g("rows", 4), g("cols", 64), g("dx", D_), 64, g("dw", None), g("ws", None),
                                            g("bytes", 0), g("dt", 0), None)


def test_rms_norm_backward_refuses(mm):
    for kw in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None), dict(dw=E_), dict(dx=A + 32), dict(dt=7)):
        assert _back_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=0), dict(lddy=63)):
        assert _back_call(mm, **kw) == 2, kw
    for kw in (dict(rstd=C_ + 2), dict(dx=D_ + 1), dict(dw=E_ + 2), dict(dw=E_, ws=B_ + 8, bytes=1 << 20)):
        assert _back_call(mm, **kw) == 3, kw
    assert _back_call(mm, dw=E_, ws=B_, bytes=16) == 4


def _quant_call(mm, **kw):
    g = lambda k, d: kw.get(k, d)  # noqa: E731
    return mm.load().muon_fp8_quantize(g("x", A), g("ldx", 100), g("rows", 40), g("cols", 100), g("dt", 0), g("fmt", 0),
                                       g("sq", 0), g("q", B_), g("ldq", 112), g("qs", C_), g("qt", D_), g("ldqt", 48),
                                       g("qts", E_), None)


def test_quantize_refuses(mm):
    for kw in (dict(x=None), dict(dt=4), dict(fmt=2), dict(sq=2), dict(q=None), dict(qs=None), dict(qts=None),
               dict(q=None, qs=None, qt=None, qts=None), dict(q=A + 16), dict(qt=B_ + 160)):
        assert _quant_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=4194305), dict(ldx=99), dict(ldq=96), dict(ldqt=32)):
        assert _quant_call(mm, **kw) == 2, kw
    for kw in (dict(x=A + 1), dict(q=B_ + 8), dict(ldq=120), dict(qs=C_ + 1)):
        assert _quant_call(mm, **kw) == 3, kw
    assert _quant_call(mm, rows=0) == 0 and _quant_call(mm, cols=0) == 0


def _mm_call(mm, **kw):
    g = lambda k, d: kw.get(k, d)  # noqa: E731
    return mm.load().muon_fp8_matmul(g("a", A), g("lda", 128), g("sa", A + (1 << 20)), g("fa", 0), g("b", B_), g("ldb", 128),
                                     g("sb", B_ + (1 << 20)), 0, g("m", 8), g("n", 16), g("k", 128), g("add", None),
                                     g("ldadd", 16), g("out", C_), g("ldc", 16), g("dt", 0), None)


def test_matmul_refuses(mm):
    for kw in (dict(a=None), dict(sb=None), dict(out=None), dict(fa=2), dict(dt=3), dict(out=A + 64), dict(out=B_ + (1 << 20)),
               dict(add=C_ + 2), dict(add=C_, ldadd=24)):
        assert _mm_call(mm, **kw) == 1, kw
    for kw in (dict(m=-1), dict(n=4194305), dict(k=-5), dict(lda=112), dict(ldc=15)):
        assert _mm_call(mm, **kw) == 2, kw
    for kw in (dict(a=A + 8), dict(lda=136), dict(out=C_ + 1), dict(sa=A + (1 << 20) + 2)):
        assert _mm_call(mm, **kw) == 3, kw
    assert _mm_call(mm, m=0) == 0 and _mm_call(mm, n=0) == 0


def test_python_refuses(mm):
    data = torch.zeros(4, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(1, 4, 4, dtype=torch.uint8)
    t = mm.Fp8Tensor(data, scale)
    assert t.fmt == "e4m3" and t.shape == (4, 32)
    with pytest.raises(TypeError):
        mm.Fp8Tensor(data.float(), scale)
    with pytest.raises(ValueError):
        mm.Fp8Tensor(data, scale[:, :3].contiguous())
    with pytest.raises(ValueError):
        mm.Fp8Tensor(data[:, :24].contiguous(), scale)           # row stride 24
    with pytest.raises(ValueError):
        mm.fp8_matmul(t, t)                                      # not on a GPU
    with pytest.raises(ValueError):
        mm.fp8_matmul(t, mm.Fp8Tensor(data[:, :16], scale))      # another k
    with pytest.raises(TypeError):
        mm.fp8_matmul(data, t)
    with pytest.raises(ValueError):
        mm.rms_norm(torch.zeros(2, 8), None)
    with pytest.raises(ValueError):
        mm.fp8_quantize(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        mm.fp8_quantize(torch.zeros(2, 8), fmt="e3m4")
    with pytest.raises(ValueError):
        mm.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        mm.clip_grads([torch.zeros(3)], 1.0)


# ---------------------------------------------------------------- clipping

def _clip_case(mm, grads, max_norm, eps=1e-6):
    want_n, want = ref.clip_grads(grads, max_norm, eps)
    dev = [g.cuda() for g in grads]
    out = [torch.full_like(g, 7.0) for g in dev]
    norm = mm.clip_grads(dev, max_norm, out=out, eps=eps)
    alone = mm.grad_norm(dev)
    again = [g.clone() for g in dev]
    norm2 = mm.clip_grads(again, max_norm, eps=eps)
    torch.cuda.synchronize()
    # a thread sums at most 8192 elements of each of a few chunks in four chains; 2^-24 each, halved by the root
    tol = 4096 * F24
    assert abs(float(norm) - want_n) <= tol * want_n + 1e-44
    assert float(norm2) == float(norm) == float(alone)
    for g, o, w, i in zip(grads, out, want, again):
        close(o, w, (U[g.dtype] + tol + 4 * F24) * w.abs() + TINY[g.dtype])
        assert torch.equal(o, i)
    return float(norm), out


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1], [7], [8191, 1, 8193, 64], [100_003, 0, 5, 65_536], [3] * 65, [2_000_001]])
def test_clip_matches_oracle(mm, dtype, sizes):
    grads = [gen(10 + i, n).to(dtype) for i, n in enumerate(sizes)]
    _clip_case(mm, grads, 0.5)
    _clip_case(mm, grads, 1e6)  # below the limit


@gpu
def test_clip_mixed_types_shapes_and_alignment(mm):
    grads = [gen(1, 33, 65).bfloat16(), gen(2, 1000), gen(3, 7, 3, 5).half(), gen(4, 1).bfloat16()]
    norm, _ = _clip_case(mm, grads, 1.0)
    buf = torch.zeros(5000, device="cuda", dtype=torch.bfloat16)
    buf[1:2146] = grads[0].flatten().cuda()                       # 2 bytes off 16
    out = [torch.empty_like(g, device="cuda") for g in grads]
    n2 = mm.clip_grads([buf[1:2146]] + [g.cuda() for g in grads[1:]], 1.0, out=[out[0].view(-1)] + out[1:])
    assert abs(float(n2) - norm) <= 1e-6 * norm
    assert float(buf[0]) == 0 and float(buf[2146:].abs().sum()) == 0


@gpu
def test_clip_more_tensors_than_one_launch_takes(mm):
    grads = [gen(i, 1 + i % 37).to(DTYPES[i % 3]) for i in range(2500)]
    _clip_case(mm, grads, 1.0)


@gpu
@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-15, 1e18, 1e25, 1e37])
def test_clip_norm_outside_the_range_of_squares(mm, size):
    grads = [gen(1, 5000, std=size / 10), gen(2, 300, std=size / 10).bfloat16()]
    _clip_case(mm, grads, size, eps=0.0)


@gpu
def test_clip_special_values(mm):
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(mm.clip_grads(z, 1.0)) == 0.0 and float(z[0].abs().sum()) == 0.0
    g = [torch.ones(100, device="cuda"), torch.ones(9, device="cuda").bfloat16()]
    g[0][3] = math.inf
    assert float(mm.clip_grads(g, 1.0)) == math.inf
    assert math.isnan(float(g[0][3])) and float(g[0][4]) == 0.0 and float(g[1][0]) == 0.0
    g = [torch.ones(100, device="cuda")]
    g[0][50] = math.nan
    assert math.isnan(float(mm.clip_grads(g, 1.0))) and bool(torch.isnan(g[0]).all())
    g = [torch.full((64,), 3.0, device="cuda")]
    assert float(mm.clip_grads(g, math.inf)) == 24.0 and float(g[0][0]) == 3.0
    assert float(mm.clip_grads(g, 0.0)) == 24.0 and float(g[0].abs().sum()) == 0.0


# ---------------------------------------------------------------- quantisation

def _kept(exps):
    rows, blocks = exps.shape
    out = torch.full((-(-blocks // 4), -(-rows // 4) * 4, 4), 127, dtype=torch.uint8)
    for kb in range(blocks):
        out[kb // 4, :rows, kb % 4] = (exps[:, kb] + 127).to(torch.uint8)
    return out


def _check_quantized(q, x, fmt, square):
    data, exps = ref.quantize(x, fmt, square)
    assert q.shape == x.shape and q.fmt == fmt
    assert torch.equal(q.data.float().cpu().double(), data)
    assert torch.equal(q.scale.view(torch.uint8).cpu(), _kept(exps))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (1, 640), (130, 7), (129, 385), (5, 1030), (256, 512)])
def test_quantize_is_exact(mm, dtype, fmt, square, shape):
    x = (gen(3, *shape) * torch.exp(3 * gen(4, shape[0], 1))).to(dtype)
    q, qt = mm.fp8_quantize(x.cuda(), fmt, square=square, rows=True, cols=True)
    _check_quantized(q, x, fmt, square)
    _check_quantized(qt, x.t(), fmt, square)
    only, none = mm.fp8_quantize(x.cuda(), fmt, square=square)
    assert none is None and torch.equal(only.data.view(torch.uint8), q.data.view(torch.uint8))
    none, only = mm.fp8_quantize(x.cuda(), fmt, square=square, rows=False, cols=True)
    assert none is None and torch.equal(only.data.view(torch.uint8), qt.data.view(torch.uint8))
    assert torch.equal(only.scale.view(torch.uint8), qt.scale.view(torch.uint8))


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_boundaries(mm, fmt):
    """Block maxima on and next to a power of two times the largest value, zeros, subnormals, fp32's extremes."""
    top = ref.TOP[fmt]
    ones = torch.tensor([top, top * (1 + 2.0 ** -23), top * (1 - 2.0 ** -24), top * 2.0 ** -130, 2.0 ** -149, 1e-40, 0.0,
                         3.4e38, top * 2.0 ** 100, 2.0 ** -126])
    x = gen(1, len(ones), 256).clamp(-1, 1) * ones[:, None]
    x[:, 0] = ones
    q, qt = mm.fp8_quantize(x.cuda(), fmt, rows=True, cols=True)
    _check_quantized(q, x, fmt, False)
    _check_quantized(qt, x.t(), fmt, False)


@gpu
def test_quantize_strides_and_padding(mm):
    big = gen(9, 300, 400).bfloat16().cuda()
    for x in (big[3:200, 5:205], big[:, :393], big.view(600, 200)[::2]):
        q, qt = mm.fp8_quantize(x, rows=True, cols=True)
        _check_quantized(q, x.cpu(), "e4m3", False)
        _check_quantized(qt, x.cpu().t(), "e4m3", False)
    with pytest.raises(ValueError):
        mm.fp8_quantize(big.t())
    q, qt = mm.fp8_quantize(big[:0], rows=True, cols=True)
    assert q.shape == (0, 400) and qt.shape == (400, 0)


@gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_quantize_marks_what_is_not_finite(mm, value):
    x = gen(2, 200, 300)
    x[10, 140] = value
    q, qt = mm.fp8_quantize(x.cuda(), rows=True, cols=True)
    v, vt = q.dequantize().cpu(), qt.dequantize().cpu()
    assert bool(torch.isnan(v[10, 128:256]).all()) and int(torch.isnan(v).sum()) == 128
    assert bool(torch.isnan(vt[140, :128]).all()) and int(torch.isnan(vt).sum()) == 128
    assert int(q.scale.view(torch.uint8)[0, 10, 1]) == 255
    s, _ = mm.fp8_quantize(x.cuda(), square=True)
    assert int(torch.isnan(s.dequantize()).sum()) == 128 * 128
    # and the product of a marked row is NaN, the others are not
    w, _ = mm.fp8_quantize(gen(3, 40, 300).cuda())
    c = mm.fp8_matmul(q, w, torch.float32).cpu()
    assert bool(torch.isnan(c[10]).all()) and int(torch.isnan(c).sum()) == 40


# ---------------------------------------------------------------- RMS norm

def _check_norm(mm, x, w, res, eps=1e-6, fp8=None, dtype=None):
    r = mm.rms_norm(x.cuda(), None if w is None else w.cuda(), None if res is None else res.cuda(), eps=eps, fp8=fp8)
    torch.cuda.synchronize()
    y, h, rstd = ref.rms_norm(x, w, res, eps)
    cols, u = x.shape[-1], U[x.dtype]
    # chains of at most 128 terms and nine joins; the root halves it; division, root and mean add 4
    rel = (137 / 2 + 4) * F24
    close(r.rstd, rstd.flatten(), rel * rstd.flatten())
    close(r.h, h, u * h.abs() + TINY[x.dtype])
    add = 0 if res is None else 2.0 ** -24 * h.abs() * 1.0  # the fp32 sum of x and residual
    yt = (u + rel + 3 * F24) * y.abs() + TINY[x.dtype]
    if res is not None:
        yt = yt + add * rstd[..., None] * (1 if w is None else w.double().abs())
    close(r.y, y, yt)
    if fp8:
        assert r.q.shape == (x.numel() // cols, cols)
        half, sub = (2.0 ** -4, 2.0 ** -10) if fp8 == "e4m3" else (2.0 ** -3, 2.0 ** -17)
        v, s = r.q.dequantize().cpu().double(), r.q.scales().cpu().double().repeat_interleave(128, dim=1)[:, :cols]
        y2 = y.reshape(-1, cols)
        assert bool(((v - y2).abs() <= (half + 2 * rel) * y2.abs() + sub * s).all())
        if x.dtype == torch.float32:  # y is the unrounded value that was quantised
            data, exps = ref.quantize(r.y.cpu().reshape(-1, cols), fp8)
            assert torch.equal(r.q.data.float().cpu().double(), data)
            assert torch.equal(r.q.scale.view(torch.uint8).cpu(), _kept(exps))
        else:
            assert int((r.q.scale.view(torch.uint8) == 255).sum()) == 0
    return r


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(1, 1), (3, 8), (5, 127), (9, 256), (2, 513), (7, 1000), (4, 2048), (3, 4100), (2, 8192),
                                   (1, 16384), (2, 20001)])
def test_rms_norm_matches_oracle(mm, dtype, residual, shape):
    x = (gen(1, *shape) * torch.exp(gen(2, 1, shape[1]))).to(dtype)
    res = gen(3, *shape).to(dtype) if residual else None
    _check_norm(mm, x, 1 + gen(4, shape[1], std=0.1), res, fp8="e4m3")
    _check_norm(mm, x, None, res, fp8="e5m2" if shape[1] % 2 else None)


@gpu
@pytest.mark.parametrize("wdt", DTYPES)
def test_rms_norm_weight_types_dimensions_and_zero_rows(mm, wdt):
    x = gen(1, 2, 5, 384).bfloat16()
    x[1, 2] = 0
    r = _check_norm(mm, x, gen(2, 384).to(wdt), None, fp8="e4m3")
    assert r.y.shape == x.shape and r.h.data_ptr() != 0
    assert float(r.y[1, 2].abs().sum()) == 0 and abs(float(r.rstd[7]) - 1e3) < 1e-2
    r = mm.rms_norm(x.cuda(), None, y=False, fp8="e5m2")
    assert r.y is None and r.q.fmt == "e5m2"
    e = mm.rms_norm(x[:0].cuda(), None, fp8="e4m3")
    assert e.y.shape == (0, 5, 384) and e.q.shape == (0, 384)


@gpu
def test_rms_norm_strides_alignment_and_not_finite_rows(mm):
    big = gen(5, 40, 700).bfloat16()
    dev = big.cuda()
    for sl in ((slice(None), slice(3, 260)), (slice(2, 30), slice(0, 512)), (slice(0, 40, 3), slice(8, 700))):
        x = dev[sl]
        r = mm.rms_norm(x, None, x, fp8="e4m3")
        y, h, _ = ref.rms_norm(big[sl], None, big[sl])
        close(r.y, y, (U[torch.bfloat16] + 100 * F24) * y.abs())
        close(r.h, h, U[torch.bfloat16] * h.abs())
        data, exps = ref.quantize(y, "e4m3")
        assert (r.q.data.float().cpu().double() - data).abs().max() <= 32  # one step of the largest values
    with pytest.raises(ValueError):
        mm.rms_norm(dev.t(), None)
    x = gen(6, 3, 500)
    x[1, 200] = math.inf
    r = mm.rms_norm(x.cuda(), None, fp8="e4m3")
    assert math.isnan(float(r.y[1, 200])) and bool(torch.isfinite(r.y[[0, 2]]).all())
    assert int(torch.isnan(r.q.dequantize()).sum()) == 128
    x[1, 200] = math.nan
    r = mm.rms_norm(x.cuda(), None, fp8="e4m3")
    assert bool(torch.isnan(r.y[1]).all()) and bool(torch.isfinite(r.y[[0, 2]]).all())
    assert int(torch.isnan(r.q.dequantize()).sum()) == 500


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (3, 8), (700, 130), (9, 257), (33, 512), (2, 1000), (1500, 1024), (5, 2048),
                                   (641, 4100), (3, 8192), (2, 9001), (610, 16500)])
def test_rms_norm_backward_matches_oracle(mm, dtype, shape):
    rows, cols = shape
    h, dy = gen(1, *shape).to(dtype), gen(2, *shape).to(dtype)
    w, res = 1 + gen(3, cols, std=0.2), gen(4, *shape).to(dtype)
    rstd = ref.rms_norm(h)[2].float()
    for dres, weight in ((None, w), (res, w), (res, None)):
        dx, dw = mm.rms_norm_backward(dy.cuda(), h.cuda(), None if weight is None else weight.cuda(), rstd.cuda(),
                                      None if dres is None else dres.cuda())
        want, want_w = ref.rms_norm_backward(dy, h, weight, rstd, dres)
        g = dy.double() * (1 if weight is None else weight.double())
        r = rstd.double()[:, None]
        mean = (g * h.double()).abs().mean(dim=1, keepdim=True)
        # the mean's chain as in the norm; four more operations on each term
        tol = (140 * F24) * h.double().abs() * r ** 3 * mean + 6 * F24 * ((r * g).abs() + want.abs())
        close(dx, want, tol + U[dtype] * want.abs() + TINY[dtype])
        # a column's chain: the rows of one CTA, then the CTAs
        n = rows + 16
        close(dw, want_w, (n + 4) * F24 * (dy.double() * h.double() * r).abs().sum(dim=0))
    again = mm.rms_norm_backward(dy.cuda(), h.cuda(), None, rstd.cuda(), res.cuda())
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    dx2, none = mm.rms_norm_backward(dy.cuda(), h.cuda(), None, rstd.cuda(), res.cuda(), dweight=False)
    assert none is None and torch.equal(dx2, dx)


@gpu
def test_rms_norm_backward_against_differences(mm):
    x, w, v = gen(1, 3, 40), 1 + gen(2, 40, std=0.3), gen(3, 3, 40)
    r = mm.rms_norm(x.cuda(), w.cuda())
    dx, dw = mm.rms_norm_backward(v.cuda(), r.h, w.cuda(), r.rstd)
    loss = lambda x, w: float((ref.rms_norm(x, w)[0] * v.double()).sum())  # noqa: E731
    step = 1e-5
    for i in range(0, 40, 7):
        d = torch.zeros(3, 40, dtype=torch.float64)
        d[2, i] = step
        want = (loss(x.double() + d, w) - loss(x.double() - d, w)) / (2 * step)
        assert abs(float(dx[2, i]) - want) < 1e-5  # fp32 arithmetic on terms of about 1, plus the difference's step^2
        e = torch.zeros(40, dtype=torch.float64)
        e[i] = step
        want = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * step)
        assert abs(float(dw[i]) - want) < 1e-5


@gpu
def test_rms_norm_backward_no_rows(mm):
    dx, dw = mm.rms_norm_backward(torch.zeros(0, 64, device="cuda"), torch.zeros(0, 64, device="cuda"), None,
                                  torch.zeros(0, device="cuda"))
    assert dx.shape == (0, 64) and float(dw.abs().sum()) == 0


# ---------------------------------------------------------------- product

def _operand(mm, seed, rows, cols, fmt, std=1.0):
    x = (gen(seed, rows, cols) * torch.exp(gen(seed + 1, rows, 1)) * std)
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    return q, ref.values(q.data.cpu(), q.scale.view(torch.uint8).cpu())


def _mm_tol(a, b, want, dtype, k):
    # fp32 over k / 32 steps that may truncate (2^-23), 32 products inside a step, and up to 16 parts
    return U[dtype] * want.abs() + (k / 32 + 48) * 2.0 ** -23 * (a.abs() @ b.abs().t()) + TINY[dtype]


@gpu
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 300, 129), (3, 256, 640), (33, 100, 31), (225, 257, 513), (64, 513, 1152),
                                   (500, 40, 2049)])
def test_matmul_matches_oracle(mm, out, fa, fb, m, n, k):
    a, av = _operand(mm, 1, m, k, fa)
    b, bv = _operand(mm, 3, n, k, fb, std=0.1)
    add = gen(9, m, n).to(out)
    want = ref.matmul(av, bv)
    close(mm.fp8_matmul(a, b, out), want, _mm_tol(av, bv, want, out, k))
    want = want + add.double()
    acc = add.cuda()
    c = mm.fp8_matmul(a, b, add=acc, out=acc)
    assert c is acc
    close(c, want, _mm_tol(av, bv, want, out, k) + F24 * want.abs())
    assert mm.fp8_status() == 0


@gpu
@pytest.mark.parametrize("m,n,k", [(1, 2048, 8192), (7, 512, 20000), (2, 4100, 4096), (33, 700, 1500), (64, 256, 6000),
                                   (100, 300, 9000), (5, 9000, 1030), (40, 64, 513)])
@pytest.mark.parametrize("out", DTYPES)
def test_matmul_few_tiles(mm, m, n, k, out):
    """k is split over the pairs of a cluster and joined; the same bits every time."""
    a, av = _operand(mm, 1, m, k, "e4m3")
    b, bv = _operand(mm, 3, n, k, "e4m3")
    want = ref.matmul(av, bv)
    add = gen(5, m, n).to(out)
    c = mm.fp8_matmul(a, b, out)
    close(c, want, _mm_tol(av, bv, want, out, k))
    for _ in range(3):
        assert torch.equal(mm.fp8_matmul(a, b, out), c)
    d = mm.fp8_matmul(a, b, out, add=add.cuda())
    want = want + add.double()
    close(d, want, _mm_tol(av, bv, want, out, k) + F24 * want.abs())
    assert mm.fp8_status() == 0


@gpu
@pytest.mark.parametrize("m,n,k", [(1000, 3000, 700), (2100, 1500, 1024), (4000, 2000, 300)])
def test_matmul_many_tiles(mm, m, n, k):
    a, av = _operand(mm, 1, m, k, "e4m3")
    b, bv = _operand(mm, 3, n, k, "e4m3")
    want = ref.matmul(av, bv)
    c = mm.fp8_matmul(a, b)
    close(c, want, _mm_tol(av, bv, want, torch.bfloat16, k))
    assert torch.equal(mm.fp8_matmul(a, b), c)


@gpu
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (8, 17, 48), (4, 15, 127), (8, 33, 2500), (9, 33, 2500), (1, 2500, 1000),
                                   (6, 50, 4144), (3, 4870, 600), (2, 1, 9000), (8, 700, 513)])
def test_matmul_few_rows(mm, out, fa, fb, m, n, k):
    """At most 8 rows of a: the kernel for single tokens, on both sides of its limits."""
    a, av = _operand(mm, 11, m, k, fa)
    b, bv = _operand(mm, 13, n, k, fb, std=0.1)
    want = ref.matmul(av, bv)
    buf = torch.full((m, n + 5), 3.0, device="cuda", dtype=out)
    c = mm.fp8_matmul(a, b, out=buf[:, 2:n + 2])
    close(c, want, _mm_tol(av, bv, want, out, k))
    assert bool((buf[:, :2] == 3).all()) and bool((buf[:, n + 2:] == 3).all())
    add = gen(9, m, n).to(out)
    acc = add.cuda()
    want = want + add.double()
    close(mm.fp8_matmul(a, b, add=acc, out=acc), want, _mm_tol(av, bv, want, out, k) + F24 * want.abs())
    for _ in range(3):
        assert torch.equal(mm.fp8_matmul(a, b, out), c)


@gpu
@pytest.mark.parametrize("m", [1, 8, 9])
@pytest.mark.parametrize("ea,eb", [(60, 60), (-60, -60), (120, -115), (-115, 125)])
def test_matmul_few_rows_extreme_scales(mm, m, ea, eb):
    """The product of two scales may leave fp32's range where the result does not."""
    n, k = 40, 700
    a, _ = _operand(mm, 1, m, k, "e4m3", std=0.01)
    b, _ = _operand(mm, 3, n, k, "e4m3", std=0.01)
    a = mm.Fp8Tensor(a.data, a.scale.view(torch.uint8) + ea)  # a few bytes wrap round, so that large meets large too
    b = mm.Fp8Tensor(b.data, b.scale.view(torch.uint8) + eb)
    av, bv = (ref.values(q.data.cpu(), q.scale.cpu()) for q in (a, b))
    want, most = ref.matmul(av, bv), av.abs() @ bv.abs().t()
    got = mm.fp8_matmul(a, b, torch.float32).cpu()
    assert bool(got[want.isnan() | (want.abs() >= 2.0 ** 128)].isfinite().logical_not().all())
    fits = most < 2.0 ** 127  # none of the last case's
    close(got[fits], want[fits], (_mm_tol(av, bv, want, torch.float32, k) + 2.0 ** -140)[fits])


@gpu
@pytest.mark.parametrize("m", [1, 2, 8, 9])
@pytest.mark.parametrize("fmt,nan", [("e4m3", 0x7f), ("e4m3", 0xff), ("e5m2", 0x7e)])
def test_matmul_few_rows_nan(mm, m, fmt, nan):
    """A NaN among the values or the scales reaches its row and column and nothing else."""
    n, k = 37, 1300
    a, _ = _operand(mm, 1, m, k, fmt)
    b, _ = _operand(mm, 3, n, k, fmt)
    c = mm.fp8_matmul(a, b, torch.float32)
    a.data.view(torch.uint8)[m - 1, 1298] = nan
    d = mm.fp8_matmul(a, b, torch.float32)
    assert bool(d[m - 1].isnan().all()) and torch.equal(d[:m - 1], c[:m - 1])
    x = (gen(3, n, k) * torch.exp(gen(4, n, 1))).cuda()
    x[20, 130] = float("inf")
    b, _ = mm.fp8_quantize(x, fmt)
    d = mm.fp8_matmul(a, b, torch.float32)
    assert bool(d[:, 20].isnan().all()) and bool(d[m - 1].isnan().all())
    rest = [j for j in range(n) if j != 20]
    assert torch.equal(d[:m - 1][:, rest], c[:m - 1][:, rest])


@gpu
@pytest.mark.parametrize("m,n,k", [(4096, 4096, 4096), (2048, 2500, 2048), (300, 4096, 6000), (64, 8000, 3000)])
def test_matmul_add_keeps_its_bits(mm, m, n, k):
    """An epilogue that reads as well as writes holds the MMAs up and the scales wait for them: still the plain
    product plus the addend, one rounding in fp32, call after call."""
    a, av = _operand(mm, 1, m, k, "e4m3")
    b, bv = _operand(mm, 3, n, k, "e4m3")
    plain = mm.fp8_matmul(a, b, torch.float32)
    rows = torch.arange(0, m, max(1, m // 32))
    want = ref.matmul(av[rows], bv)
    close(plain[rows.cuda()], want, _mm_tol(av[rows], bv, want, torch.float32, k))
    add = gen(7, m, n).cuda()
    want = plain + add
    outs = [mm.fp8_matmul(a, b, torch.float32, add=add) for _ in range(12)]
    assert [torch.equal(c, want) for c in outs] == [True] * 12
    low = add.bfloat16()
    want = (plain + low.float()).bfloat16()
    outs = [mm.fp8_matmul(a, b, torch.bfloat16, add=low) for _ in range(12)]
    assert [torch.equal(c, want) for c in outs] == [True] * 12
    assert mm.fp8_status() == 0


@gpu
def test_matmul_strided_output_and_extreme_scales(mm):
    a, av = _operand(mm, 1, 50, 300, "e4m3")
    b, bv = _operand(mm, 3, 70, 300, "e4m3")
    want = ref.matmul(av, bv)
    buf = torch.full((50, 201), 5.0, device="cuda")
    mm.fp8_matmul(a, b, out=buf[:, 3:73])
    close(buf[:, 3:73], want, _mm_tol(av, bv, want, torch.float32, 300))
    assert bool((buf[:, :3] == 5).all()) and bool((buf[:, 73:] == 5).all())
    # scales far from 1 on both sides: exact powers of two, so the product only moves by their product
    big, small = mm.Fp8Tensor(a.data, (a.scale.view(torch.uint8) + 60)), mm.Fp8Tensor(b.data, b.scale.view(torch.uint8) - 70)
    close(mm.fp8_matmul(big, small, torch.float32), want * 2.0 ** -10, _mm_tol(av, bv, want, torch.float32, 300) * 2.0 ** -10)


@gpu
def test_matmul_empty(mm):
    z = mm.Fp8Tensor.empty(5, 0)
    w = mm.Fp8Tensor.empty(7, 0)
    assert torch.equal(mm.fp8_matmul(z, w, torch.float32), torch.zeros(5, 7, device="cuda"))
    add = gen(1, 5, 7).cuda()
    assert torch.equal(mm.fp8_matmul(z, w, torch.float32, add=add), add)
    e, _ = mm.fp8_quantize(torch.zeros(0, 64, device="cuda"))
    f, _ = mm.fp8_quantize(torch.ones(3, 64, device="cuda"))
    assert mm.fp8_matmul(e, f).shape == (0, 3) and mm.fp8_matmul(f, e).shape == (3, 0)


# ---------------------------------------------------------------- together

@gpu
def test_operators_on_another_stream(mm):
    """Everything on a side stream gives what it gives on the current one."""
    x, w = gen(1, 300, 512).bfloat16().cuda(), gen(2, 256, 512).bfloat16().cuda()
    g = [gen(3, 5000).cuda(), gen(4, 77).bfloat16().cuda()]

    def once(stream):
        gg = [t.clone() for t in g]
        torch.cuda.synchronize()
        r = mm.rms_norm(x, None, x, fp8="e4m3", stream=stream)
        wq, wt = mm.fp8_quantize(w, square=True, cols=True, stream=stream)
        c = mm.fp8_matmul(r.q, wq, stream=stream)
        dx, dw = mm.rms_norm_backward(r.y, r.h, None, r.rstd, stream=stream)
        n = mm.clip_grads(gg, 1.0, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        return [r.y, r.h, r.rstd, r.q.data.view(torch.uint8), wt.data.view(torch.uint8), c, dx, dw, n] + gg

    for a, b in zip(once(None), once(torch.cuda.Stream())):
        assert torch.equal(a, b)


@gpu
def test_operators_under_graph_capture(mm):
    x, w = gen(1, 64, 512).bfloat16().cuda(), gen(2, 256, 512).bfloat16().cuda()
    q, _ = mm.fp8_quantize(w)

    def step():
        r = mm.rms_norm(x, None, fp8="e4m3")
        c = mm.fp8_matmul(r.q, q)
        return c, mm.clip_grads([c], 1.0)

    want, n = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got, m = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and float(m) == float(n)


def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_training_step.py")
    spec = importlib.util.spec_from_file_location("fp8_training_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@gpu
def test_example_gradients_match_autograd(mm):
    """The example's 8-bit forward and backward pass against fp32 autograd of the same model, to 8-bit accuracy."""
    ex = _example()
    model = ex.Mlp(2, 256, 384, seed=3)
    x = gen(1, 300, 256).bfloat16().cuda()
    y, saved = model.forward(x)
    dy = gen(2, 300, 256).bfloat16().cuda()
    matrices, norms = model.backward(dy, saved)
    ws = [w.master.float().requires_grad_() for w in model.weights]
    ns = [n.clone().requires_grad_() for n in model.norms]
    s = x.float()
    for i in range(2):
        n = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * ns[i]
        s = s + torch.nn.functional.silu(n @ ws[2 * i].t()) @ ws[2 * i + 1].t()
    out = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * ns[2]
    (out * dy.float()).sum().backward()
    # an 8-bit operand is off by 2^-4 (e4m3) or 2^-3 (e5m2) of its value at most, a third of that in the mean square;
    # a gradient passes at most six such operands in a row
    far = lambda a, b: float((a.float() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    limit = 6 ** 0.5 * 2.0 ** -3 / 3 ** 0.5
    assert far(y, out) < limit
    for got, want in zip(matrices, ws):
        assert far(got, want.grad) < limit
    for got, want in zip(norms, ns):
        assert far(got, want.grad) < limit


@gpu
def test_example_learns(mm):
    losses, norms = _example().train(steps=12, tokens=1024, log=lambda *_: None)
    assert all(math.isfinite(v) for v in losses + norms)
    assert losses[-1] < 0.9 * losses[0]


@gpu
def test_fp8_status_reports_a_wait_that_ran_out(mm):
    assert mm.fp8_status() == 0
    mm.debug_bounded_wait_fp8(100_000)
    assert mm.fp8_status() == 6   # MUON_ERR_TIMEOUT, once
    assert mm.fp8_status() == 0
    with pytest.raises(mm.MuonError):
        mm.debug_bounded_wait_fp8(0)


@gpu
def test_rms_norm_weight_off_16_bytes(mm):
    """A weight at an odd address takes the kernels without 16-byte accesses; so do odd strides, with the same values."""
    x, w = gen(1, 37, 1200).bfloat16(), 1 + gen(2, 1201, std=0.1)
    a = mm.rms_norm(x.cuda(), w.cuda()[1:], fp8="e4m3")
    b = mm.rms_norm(x.cuda(), w[1:].clone().cuda(), fp8="e4m3")
    y, _, rstd = ref.rms_norm(x, w[1:])
    for r in (a, b):
        close(r.y, y, (U[torch.bfloat16] + 100 * F24) * y.abs())
        close(r.rstd, rstd, 80 * F24 * rstd)
    dy = gen(3, 37, 1200).bfloat16().cuda()
    want = ref.rms_norm_backward(dy.cpu(), x, w[1:], rstd)
    for weight in (w.cuda()[1:], w[1:].clone().cuda()):
        dx, dw = mm.rms_norm_backward(dy, x.cuda(), weight, rstd.float().cuda())
        assert float((dx.cpu().double() - want[0]).norm() / want[0].norm()) < U[torch.bfloat16]
        assert float((dw.cpu().double() - want[1]).norm() / want[1].norm()) < 64 * F24


@gpu
def test_offsets_past_32_bits(mm):
    """Matrices of more than 2^31 elements: their last rows and columns equal those of the same rows and columns alone."""
    rows, cols = 66_003, 33_000
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    q, qt = mm.fp8_quantize(x, rows=True, cols=True)
    tail, _ = mm.fp8_quantize(x[-7:].contiguous())
    assert torch.equal(raw(q.data[-7:]), raw(tail.data))
    assert torch.equal(q.scales()[-7:], tail.scales())
    _, side = mm.fp8_quantize(x[:, -9:].contiguous(), rows=False, cols=True)
    assert torch.equal(raw(qt.data[-9:]), raw(side.data)) and torch.equal(qt.scales()[-9:], side.scales())
    w, _ = mm.fp8_quantize(x[:300].contiguous())
    c = mm.fp8_matmul(q, w)                       # both operands' rows past 2^31 bytes
    assert torch.equal(c[-7:], mm.fp8_matmul(q, w)[-7:])
    few = mm.fp8_matmul(tail, w, torch.float32)
    assert float((c[-7:].float() - few).norm() / few.norm()) < U[torch.bfloat16]
    del q, qt, c
    r = mm.rms_norm(x, None, fp8="e4m3")
    s = mm.rms_norm(x[-7:].contiguous(), None, fp8="e4m3")
    assert torch.equal(r.y[-7:], s.y) and torch.equal(r.rstd[-7:], s.rstd) and torch.equal(raw(r.q.data[-7:]), raw(s.q.data))
    dx, _ = mm.rms_norm_backward(r.y, x, None, r.rstd)
    assert torch.equal(dx[-7:], mm.rms_norm_backward(s.y, x[-7:].contiguous(), None, s.rstd)[0])
    del r, s, dx
    last = x[-1, -300:].clone()
    norm = mm.clip_grads([x], 1000.0)
    want = sum(float(last_rows.double().square().sum()) for last_rows in x.split(2048)) ** 0.5
    assert abs(want - 1000.0) < 1000.0 * 1e-3     # in place; bf16 rounding of 2e9 values averages out
    assert torch.equal(x[-1, -300:], (last.float() * float(torch.tensor(1000.0) / (norm.cpu() + 1e-6))).bfloat16())
    small_k = mm.fp8_quantize(torch.ones(66_003, 128, device="cuda", dtype=torch.bfloat16))[0]
    wide = mm.fp8_quantize(torch.ones(33_000, 128, device="cuda", dtype=torch.bfloat16))[0]
    big = mm.fp8_matmul(small_k, wide)            # an output past 2^31 elements
    assert float(big[-1, -1]) == 128.0 and float(big[-5:].float().sum()) == 5 * 33_000 * 128.0
