"""The norms around a block, the gated activation and 8-bit checkpoints: pins of the 64-bit oracle and the refusals
(CPU), and the kernels against the oracle (GPU).

Tolerances.  An output of type T carries one rounding, U[T] of its value, or half a step of an 8-bit type.  A sum in fp32
is off by at most its longest chain times 2^-24 of the terms' magnitudes; chains have at most CHAIN terms and joins along a
row (128 in a thread at 65536 columns, 9 joins), and one for each row along a column.  sigmoid(g) is off by at most
(4 + 1.2 |g|) 2^-23 of itself: the exponential of 16-bit data by 2 + 1.17 |g| units in the last place, the sum and the
quotient by one each.  Errors of a product's factors add; `close` takes the sum of what each step allows."""
import math

import pytest
import torch

import oracle.blocks as ref
import oracle.training as ref8

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
HALF8 = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}  # of the value; of the scale (subnormals)
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
F24 = 2.0 ** -24
CHAIN = 140
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


def close(got, want, tol, what=""):
    got, want = got.cpu().double().reshape(want.shape), want.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() - tol).max()):.3g}"


def sig_err(g):
    return (4 + 1.2 * g.double().abs()) * 2 * F24


def kept_scales(exps):
    rows, blocks = exps.shape
    out = torch.full((-(-blocks // 4), -(-rows // 4) * 4, 4), 127, dtype=torch.uint8)
    for kb in range(blocks):
        out[kb // 4, :rows, kb % 4] = (exps[:, kb] + 127).to(torch.uint8)
    return out


def check8_exact(q, x, fmt):
    """q is x quantised, to the bit."""
    data, exps = ref8.quantize(x, fmt)
    assert q.shape == x.shape and q.fmt == fmt
    assert torch.equal(q.data.float().cpu().double(), data)
    assert torch.equal(q.scale.view(torch.uint8).cpu(), kept_scales(exps))


def check8(q, x, err, fmt, what=""):
    """q stands for x within half a step and `err`, with scales that fit the blocks' largest values as closely."""
    cols = x.shape[1]
    assert q.shape == x.shape and q.fmt == fmt
    s = q.scales().cpu().double()
    wide = s.repeat_interleave(128, dim=1)[:, :cols]
    half, sub = HALF8[fmt]
    close(q.dequantize(), x, half * x.abs() + (1 + half) * err + sub * wide, what)
    low = torch.nn.functional.max_pool2d((x.abs() - err)[None], (1, 128), ceil_mode=True)[0]
    high = torch.nn.functional.max_pool2d((x.abs() + err)[None], (1, 128), ceil_mode=True)[0]
    top = ref8.TOP[fmt]
    assert bool((low <= top * s).all()) and bool(((high > top * s / 2) | (high == err.max()) | (s == 1)).all()), what


# ---------------------------------------------------------------- pins of the oracle

@pytest.mark.parametrize("gate", [None, "row", "element"])
def test_oracle_block_norm_gradient_is_that_of_differences(gate):
    x, r, v, t = (gen(i, 3, 19).double() for i in range(4))
    post, pre, scale = (1 + 0.3 * gen(i, 19).double() for i in (5, 6, 7))
    g = None if gate is None else gen(8, 3, 1 if gate == "row" else 19).double()
    args = [x, r, post, pre, scale] + ([] if g is None else [g])

    def loss(x, r, post, pre, scale, g=None):
        y, h, _, _ = ref.block_norm(x, r, post, pre, g, scale, 0.5)
        return float((y * v).sum() + (h * t).sum())

    _, h, rx, rh = ref.block_norm(x, r, post, pre, g, scale, 0.5)
    dx, dr, dg, dpost, dpre, dscale = ref.block_norm_backward(v, x, h, rx, rh, post, pre, g, scale, 0.5, t)
    for i, d in enumerate([dx, dr, dpost, dpre, dscale] + ([] if g is None else [dg])):
        for at in (0, args[i].numel() // 2, args[i].numel() - 1):
            step = torch.zeros_like(args[i]).flatten()
            step[at] = 1e-6
            step = step.view(args[i].shape)
            up = loss(*(a + step if k == i else a for k, a in enumerate(args)))
            down = loss(*(a - step if k == i else a for k, a in enumerate(args)))
            assert abs((up - down) / 2e-6 - float(d.flatten()[at])) < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_gated_gradient_is_that_of_differences(kind):
    g, u, v = (gen(i, 40, std=2.0).double() for i in range(3))
    dg, du, y = ref.gated_backward(v, g, u, kind)
    fn = torch.nn.functional.silu if kind == "silu" else torch.nn.functional.gelu
    assert torch.allclose(y, fn(g) * u, rtol=1e-13, atol=1e-15)
    for d, one in ((dg, lambda e: ref.gated(g + e, u, kind)), (du, lambda e: ref.gated(g, u + e, kind))):
        assert float(((one(1e-6) - one(-1e-6)) / 2e-6 * v - d).abs().max()) < 1e-7


# ---------------------------------------------------------------- refusals (no GPU)

P = [(1 << 30) + (k << 34) for k in range(40)]  # far apart, never read


def norm_call(mm, **kw):
    from newton_schulz_04_gb300.blocks import _BLOCK_NORM
    v = dict(x=P[0], ldx=64, r=P[1], ldr=64, gate=None, ldg=64, post=P[2], scale=None, pre=P[3], y=P[4], ldy=64, h=P[5], ldh=64,
             rx=P[6], rh=P[7], q=None, qs=None, ldq=64, x8=None, x8s=None, ldx8=64, h8=None, h8s=None, ldh8=64, g8=None, g8s=None,
             ldg8=64, rows=4, cols=64, dt=0, wdt=1, per_row=0, fmt=0, kfmt=0, alpha=1.0, eps=1e-6)
    assert not kw.keys() - v.keys()
    v.update(kw)
    return mm.load().muon_block_norm(_BLOCK_NORM(*(0 if a is None else a for a in v.values())), None)


def test_block_norm_refuses(mm):
    for kw in (dict(x=None), dict(r=None), dict(post=None), dict(pre=None), dict(dt=5), dict(wdt=9), dict(eps=-1.0),
               dict(eps=math.nan), dict(alpha=math.inf), dict(per_row=2), dict(q=P[8]), dict(qs=P[8]),
               dict(q=P[8], qs=P[9], fmt=2), dict(x8=P[8], x8s=P[9], kfmt=-1), dict(g8=P[8], g8s=P[9]),
               dict(gate=P[10], per_row=1, g8=P[8], g8s=P[9]), dict(y=P[0]), dict(h=P[1] + 64), dict(y=P[5] + 128), dict(rx=P[7] + 8),
               dict(x8=P[8], x8s=P[8] + 64), dict(h=P[2]),
               dict(y=None, h=None, rx=None, rh=None)):
        assert norm_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=65537), dict(rows=4194305), dict(ldx=63), dict(ldy=10), dict(gate=P[10], ldg=63),
               dict(q=P[8], qs=P[9], ldq=48)):
        assert norm_call(mm, **kw) == 2, kw
    for kw in (dict(x=P[0] + 1), dict(post=P[2] + 2), dict(rx=P[6] + 2), dict(h8=P[8] + 8, h8s=P[9]), dict(q=P[8], qs=P[9], ldq=72),
               dict(gate=P[10] + 1)):
        assert norm_call(mm, **kw) == 3, kw
    assert norm_call(mm, rows=0) == 0
    assert mm.load().muon_block_norm(None, None) == 1


def norm_grad_call(mm, **kw):
    from newton_schulz_04_gb300.blocks import _BLOCK_NORM_GRAD
    v = dict(dy=P[0], lddy=64, dh=None, lddh=64, x=P[1], xs=None, ldx=64, h=P[2], hs=None, ldh=64, gate=None, gs=None, ldg=64,
             rx=P[3], rh=P[4], post=P[5], scale=None, pre=P[6], dx=P[7], lddx=64, dr=P[8], lddr=64, dgate=None, lddg=64, dpost=None,
             dpre=None, dscale=None, ws=None, bytes=0, rows=4, cols=64, dt=0, wdt=1, per_row=0, kfmt=0, alpha=1.0)
    assert not kw.keys() - v.keys()
    v.update(kw)
    return mm.load().muon_block_norm_backward(_BLOCK_NORM_GRAD(*(0 if a is None else a for a in v.values())), None)


def test_block_norm_backward_refuses(mm):
    for kw in (dict(dy=None), dict(x=None), dict(h=None), dict(rx=None), dict(post=None), dict(dt=7), dict(alpha=math.nan),
               dict(dx=None, dr=None), dict(dgate=P[10]), dict(dscale=P[10]), dict(xs=P[10]), dict(hs=P[10]),
               dict(xs=P[10], hs=P[11], kfmt=2), dict(gate=P[12], xs=P[10], hs=P[11]), dict(gate=P[12], gs=P[10]),
               dict(gate=P[12], gs=P[13], per_row=1, xs=P[10], hs=P[11]), dict(dx=P[0]), dict(dr=P[1] + 32), dict(dpre=P[10]),
               dict(dpre=P[7] + 4, ws=P[11], bytes=1 << 30), dict(dpre=P[10], ws=P[10], bytes=1 << 30)):
        assert norm_grad_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=65537), dict(lddy=63), dict(xs=P[10], hs=P[11], ldx=48)):
        assert norm_grad_call(mm, **kw) == 2, kw
    for kw in (dict(rh=P[4] + 2), dict(dx=P[7] + 1), dict(dpre=P[10] + 2), dict(xs=P[10], hs=P[11], ldh=72), dict(xs=P[10] + 4, hs=P[11]),
               dict(dpre=P[10], ws=P[11] + 8, bytes=1 << 30)):
        assert norm_grad_call(mm, **kw) == 3, kw
    assert norm_grad_call(mm, dpre=P[10], ws=P[11], bytes=16) == 4
    assert norm_grad_call(mm, dpre=P[10], ws=P[11], bytes=-1) == 4
    assert mm.load().muon_block_norm_backward(None, None) == 1


def gated_call(mm, **kw):
    from newton_schulz_04_gb300.blocks import _GATED
    v = dict(gate=P[0], ldg=64, up=P[1], ldu=64, y=P[2], ldy=64, q=None, qs=None, ldq=64, g8=None, g8s=None, ldg8=64, u8=None,
             u8s=None, ldu8=64, rows=4, cols=64, dt=0, act=0, fmt=0, kfmt=0)
    assert not kw.keys() - v.keys()
    v.update(kw)
    return mm.load().muon_gated_activation(_GATED(*(0 if a is None else a for a in v.values())), None)


def test_gated_activation_refuses(mm):
    for kw in (dict(gate=None), dict(up=None), dict(y=None), dict(dt=3), dict(act=2), dict(act=-1), dict(q=P[3]), dict(u8s=P[3]),
               dict(q=P[3], qs=P[4], fmt=2), dict(g8=P[3], g8s=P[4], kfmt=2), dict(y=P[0]), dict(y=P[1] + 64),
               dict(g8=P[3], g8s=P[4], u8=P[3] + 128, u8s=P[5])):
        assert gated_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=-1), dict(cols=4194305), dict(ldg=60), dict(ldu=1), dict(q=P[3], qs=P[4], ldq=32)):
        assert gated_call(mm, **kw) == 2, kw
    for kw in (dict(gate=P[0] + 1), dict(q=P[3] + 4, qs=P[4]), dict(q=P[3], qs=P[4], ldq=65)):
        assert gated_call(mm, **kw) == 3, kw
    assert gated_call(mm, rows=0) == 0 and gated_call(mm, cols=0) == 0
    assert mm.load().muon_gated_activation(None, None) == 1


def gated_grad_call(mm, **kw):
    from newton_schulz_04_gb300.blocks import _GATED_GRAD
    v = dict(dy=P[0], lddy=64, gate=P[1], gs=None, ldg=64, up=P[2], us=None, ldu=64, dg=P[3], lddg=64, du=P[4], lddu=64)
    for n in ("gr", "gc", "ur", "uc", "yc"):
        v |= {n: None, n + "s": None, "ld" + n: 64}
    v |= dict(rows=4, cols=64, dt=0, act=0, kfmt=0, fmt=0, yfmt=0)
    assert not kw.keys() - v.keys()
    v.update(kw)
    return mm.load().muon_gated_activation_backward(_GATED_GRAD(*(0 if a is None else a for a in v.values())), None)


def test_gated_activation_backward_refuses(mm):
    for kw in (dict(dy=None), dict(gate=None), dict(up=None), dict(dg=None, du=None), dict(dt=3), dict(act=2), dict(gs=P[5]), dict(us=P[5]),
               dict(gs=P[5], us=P[6], kfmt=7), dict(gr=P[5]), dict(gr=P[5], grs=P[6], fmt=2), dict(yc=P[5], ycs=P[6], yfmt=2),
               dict(dg=P[0]), dict(dg=P[4] + 8), dict(uc=P[5], ucs=P[6], gc=P[5] + 16, gcs=P[7])):
        assert gated_grad_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=4194305), dict(lddy=63), dict(gs=P[5], us=P[6], ldg=48), dict(gr=P[5], grs=P[6], ldgr=48),
               dict(gc=P[5], gcs=P[6], ldgc=0)):
        assert gated_grad_call(mm, **kw) == 2, kw
    for kw in (dict(dy=P[0] + 1), dict(gs=P[5] + 8, us=P[6]), dict(yc=P[5] + 1, ycs=P[6])):
        assert gated_grad_call(mm, **kw) == 3, kw
    assert gated_grad_call(mm, rows=0) == 0 and gated_grad_call(mm, cols=0) == 0


def transpose_call(mm, **kw):
    v = dict(q=P[0], ldq=112, qs=P[1], rows=40, cols=100, fmt=0, qt=P[2], ldqt=48, qts=P[3])
    assert not kw.keys() - v.keys()
    v.update(kw)
    return mm.load().muon_fp8_transpose(*v.values(), None)


def test_transpose_refuses(mm):
    for kw in (dict(q=None), dict(qs=None), dict(qt=None), dict(qts=None), dict(fmt=2), dict(qt=P[0] + 160), dict(qts=P[1])):
        assert transpose_call(mm, **kw) == 1, kw
    for kw in (dict(rows=-1), dict(cols=4194305), dict(ldq=96), dict(ldqt=32)):
        assert transpose_call(mm, **kw) == 2, kw
    for kw in (dict(q=P[0] + 8), dict(ldq=104), dict(qs=P[1] + 4), dict(qt=P[2] + 8), dict(ldqt=56)):
        assert transpose_call(mm, **kw) == 3, kw
    assert transpose_call(mm, rows=0) == 0 and transpose_call(mm, cols=0) == 0


def test_python_refuses(mm):
    x, w = torch.zeros(2, 8), torch.ones(8)
    q = mm.Fp8Tensor(torch.zeros(2, 16, dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :8], torch.zeros(1, 4, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w, w)                                # not on a GPU
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w, w, y=False)
    with pytest.raises(TypeError):
        mm.block_norm(x, None, w, w)
    with pytest.raises(TypeError):
        mm.block_norm(x, x, None, w)
    with pytest.raises(ValueError):
        mm.gated_activation(x, x)
    with pytest.raises(ValueError):
        mm.gated_activation(x, x, activation="tanh")
    with pytest.raises(ValueError):
        mm.gated_activation(x, x, y=False)
    with pytest.raises(TypeError):
        mm.gated_activation(x, None)
    with pytest.raises(ValueError):
        mm.gated_activation_backward(x, mm.GatedKept(x, x), dense=False)
    with pytest.raises(TypeError):
        mm.fp8_transpose(x)
    with pytest.raises(ValueError):
        mm.fp8_transpose(q)


@gpu
def test_python_refuses_mixtures(mm):
    x = gen(1, 6, 256).cuda().bfloat16()
    w = torch.ones(256, device="cuda")
    q, _ = mm.fp8_quantize(x)
    q5, _ = mm.fp8_quantize(x, "e5m2")
    r = torch.ones(6, device="cuda")
    with pytest.raises(ValueError):
        mm.block_norm(x, x[:5], w, w)
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w[:255], w)
    with pytest.raises(TypeError):
        mm.block_norm(x, x, w, w.half())
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w, w, gate=x[:, :2])
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w, w, gate=x.float())
    with pytest.raises(ValueError):
        mm.block_norm(x, x, w, w, checkpoint="e3m4")
    for kept in ((q, x, None, r, r), (q, q5, None, r, r), (q, q, x, r, r), (x, x, q, r, r), (q, q, None, r[:5], r),
                 (q, q, None, r, r.double()), (x.float(), x, None, r, r)):
        with pytest.raises(ValueError):
            mm.block_norm_backward(x, mm.BlockNormKept(*kept), w, w)
    for kept in ((q, x), (q, q5), (x.float(), x)):
        with pytest.raises(ValueError):
            mm.gated_activation_backward(x, mm.GatedKept(*kept))
    with pytest.raises(ValueError):
        mm.gated_activation_backward(x, mm.GatedKept(q, q), stream=torch.cuda.Stream(), fp8="e9")


# ---------------------------------------------------------------- norms around a block

def norm_inputs(seed, rows, cols, dtype, gate, scale, wdt=torch.float32):
    x = (gen(seed, rows, cols) * torch.exp(gen(seed + 1, 1, cols))).to(dtype)
    r = gen(seed + 2, rows, cols).to(dtype)
    g = None if gate == "none" else gen(seed + 3, rows, 1 if gate == "row" else cols, std=2.0).to(dtype)
    post, pre = (1 + gen(seed + 4, cols, std=0.2)).to(wdt), (1 + gen(seed + 5, cols, std=0.2)).to(wdt)
    return x, r, g, post, pre, (0.5 + gen(seed + 6, cols, std=0.2)).to(wdt) if scale else None



def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_norm(mm, ins, alpha=1.0, eps=1e-6, fp8=None, checkpoint=None, y=True, run=None):
    x, r, g, post, pre, scale = ins
    dx, dr, dg, dpost, dpre, dscale = run or dev(*ins)
    got = mm.block_norm(dx, dr, dpost, dpre, gate=dg, scale=dscale, alpha=alpha, eps=eps, fp8=fp8, y=y, checkpoint=checkpoint)
    torch.cuda.synchronize()
    cols, dt = x.shape[1], x.dtype
    wy, wh, wrx, wrh = ref.block_norm(x, r, post, pre, g, scale, alpha, eps)
    rel = (CHAIN / 2 + 4) * F24
    close(got.kept.rstd_x, wrx, rel * wrx, "rstd_x")
    branch = (wh - alpha * r.double()).abs()
    eh = branch * (rel + 5 * F24 + (0 if g is None else sig_err(g))) + 2 * F24 * (wh.abs() + abs(alpha) * r.double().abs())
    close(got.h, wh, U[dt] * wh.abs() + eh + TINY[dt], "h")
    rel_h = rel + (eh.norm(dim=1) / wh.norm(dim=1).clamp_min(1e-300))[:, None]
    close(got.kept.rstd_h[:, None], wrh[:, None], rel_h * wrh[:, None], "rstd_h")
    ey = wy.abs() * (rel_h + 3 * F24) + eh * wrh[:, None] * pre.double().abs()
    assert (got.y is not None) == y and (got.q is not None) == (fp8 is not None)
    if y:
        close(got.y, wy, U[dt] * wy.abs() + ey + TINY[dt], "y")
    if fp8:
        check8(got.q, wy, ey, fp8, "q")
        if y and dt == torch.float32:  # y is the unrounded value that was quantised
            check8_exact(got.q, got.y.reshape(-1, cols).cpu(), fp8)
    if checkpoint:
        check8_exact(got.kept.x, x, checkpoint)
        check8(got.kept.h, wh, eh, checkpoint, "kept h")
        if dt == torch.float32:
            check8_exact(got.kept.h, got.h.reshape(-1, cols).cpu(), checkpoint)
        if g is not None and g.shape == x.shape:
            check8_exact(got.kept.gate, g, checkpoint)
        else:
            assert got.kept.gate is dg
    else:
        assert got.kept.x is dx and got.kept.gate is dg and got.kept.h is got.h
    return got


SHAPES = [(1, 1), (3, 8), (5, 127), (9, 256), (2, 513), (7, 1000), (4, 2048), (3, 4100), (5, 4096), (2, 8192), (1, 16384),
          (2, 16385), (2, 20001)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_block_norm_matches_oracle(mm, dtype, shape):
    check_norm(mm, norm_inputs(1, *shape, dtype, "element", True), fp8="e4m3", checkpoint="e4m3")
    check_norm(mm, norm_inputs(2, *shape, dtype, "row", False), alpha=0.5, fp8="e5m2", checkpoint="e5m2", y=False)
    check_norm(mm, norm_inputs(3, *shape, dtype, "none", True), alpha=-2.0, eps=1e-3)


@gpu
@pytest.mark.parametrize("cols", [64, 100, 512, 1024, 1500, 4096, 6000, 16384])
def test_block_norm_many_rows(mm, cols):
    """More rows than CTAs, so that a CTA's second and later rows are looked at too."""
    rows = 1300 if cols <= 1500 else 700
    check_norm(mm, norm_inputs(4, rows, cols, torch.bfloat16, "element", True), fp8="e4m3", checkpoint="e4m3")


# rows of one CTA's widest ring, of clusters, and those that no cluster's rings hold
WIDE = [(torch.bfloat16, 12_000), (torch.bfloat16, 16_392), (torch.bfloat16, 32_768), (torch.bfloat16, 32_769), (torch.bfloat16, 40_960),
        (torch.bfloat16, 65_536), (torch.float16, 65_535), (torch.float32, 8_192), (torch.float32, 16_384), (torch.float32, 16_385),
        (torch.float32, 32_768), (torch.float32, 40_000), (torch.float32, 65_536)]


@gpu
@pytest.mark.parametrize("dtype,cols", WIDE)
def test_block_norm_wide_rows(mm, dtype, cols):
    check_norm(mm, norm_inputs(16, 3, cols, dtype, "element", True), fp8="e4m3", checkpoint="e4m3")
    check_norm(mm, norm_inputs(17, 2, cols, dtype, "row", False), fp8="e5m2", checkpoint="e4m3", y=False)
    for kept in ("e4m3", None, "e5m2"):
        check_norm_grad(mm, 18, 3, cols, dtype, "element", True, kept=kept)
        check_norm_grad(mm, 19, 2, cols, dtype, "row", False, kept=kept, dh=False)


@gpu
@pytest.mark.parametrize("cols", [8_200, 16_392, 33_000])
@pytest.mark.parametrize("kept", [None, "e4m3"])
def test_block_norm_wide_rows_more_than_clusters(mm, cols, kept):
    check_norm(mm, norm_inputs(20, 170, cols, torch.bfloat16, "element", True), fp8="e4m3", checkpoint=kept)
    check_norm_grad(mm, 21, 170, cols, torch.bfloat16, "element", True, kept=kept)


# two rows at a time in a cluster: several turns, of which some end in one row or none, from aligned rows and others
@gpu
@pytest.mark.parametrize("dtype,cols,kept", [(torch.bfloat16, 8_192, None), (torch.float16, 16_390, None), (torch.float32, 4_096, None),
                                             (torch.float32, 4_104, "e4m3"), (torch.float32, 8_192, "e5m2"), (torch.float32, 16_384, None)])
@pytest.mark.parametrize("rows", [1, 39, 331])
def test_block_norm_backward_of_pairs_of_rows(mm, dtype, cols, kept, rows):
    check_norm_grad(mm, 22, rows, cols, dtype, "element", True, kept=kept)
    check_norm_grad(mm, 23, rows, cols, dtype, "row", False, kept=kept, pad=3, offset=1)


def strided(t, pad, offset=0):
    """t's values on the GPU in rows with `pad` more elements, `offset` elements into the allocation."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[offset:].as_strided((rows, cols), (cols + pad, 1))
    v.copy_(t)
    return v


@gpu
@pytest.mark.parametrize("wdt", DTYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (8, 8), (0, 1), (5, 3)])
def test_block_norm_strides_alignment_and_weight_types(mm, wdt, pad, offset):
    for gate in ("element", "row"):
        ins = norm_inputs(5, 11, 520, torch.bfloat16, gate, True, wdt)
        run = [strided(t, pad, offset) for t in ins[:3]] + dev(*ins[3:])
        got = check_norm(mm, ins, fp8="e4m3", checkpoint="e5m2", run=run)
        again = mm.block_norm(*run[:2], *run[3:5], gate=run[2], scale=run[5], fp8="e4m3", checkpoint="e5m2")
        assert torch.equal(got.y, again.y) and torch.equal(got.h, again.h)
        check_norm_grad(mm, 6, 11, 520, torch.bfloat16, gate, True, wdt=wdt, pad=pad, offset=offset)


@gpu
@pytest.mark.parametrize("cols,pad", [(4, 4), (12, 4), (100, 4), (123, 5), (130, 6), (1_020, 4), (4_093, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_block_norm_ragged_rows_on_16_bytes(mm, dtype, cols, pad):
    """Rows that start on 16 bytes and end off them."""
    ins = norm_inputs(22, 37, cols, dtype, "element", True)
    check_norm(mm, ins, fp8="e4m3", checkpoint="e4m3", run=[strided(t, pad) for t in ins[:3]] + dev(*ins[3:]))
    check_norm_grad(mm, 23, 37, cols, dtype, "element", True, pad=pad)
    check_norm_grad(mm, 24, 37, cols, dtype, "row", True, pad=pad, kept="e4m3")


@gpu
def test_block_norm_more_dimensions_and_no_rows(mm):
    x, r, g, post, pre, scale = dev(*norm_inputs(7, 12, 264, torch.bfloat16, "row", True))
    a = mm.block_norm(x, r, post, pre, gate=g, scale=scale, fp8="e4m3")
    b = mm.block_norm(x.view(3, 4, 264), r.view(3, 4, 264), post, pre, gate=g.view(3, 4, 1), scale=scale, fp8="e4m3")
    assert b.y.shape == b.h.shape == (3, 4, 264) and b.q.shape == (12, 264) and b.kept.rstd_x.shape == (12,)
    assert torch.equal(a.y, b.y.view(12, 264)) and torch.equal(a.q.data.view(torch.uint8), b.q.data.view(torch.uint8))
    ga = mm.block_norm_backward(x, a.kept, post, pre, scale=scale, dh=r)
    gb = mm.block_norm_backward(x.view(3, 4, 264), b.kept, post, pre, scale=scale, dh=r.view(3, 4, 264))
    assert gb.dgate.shape == (3, 4, 1) and torch.equal(ga.dgate, gb.dgate.view(12, 1)) and torch.equal(ga.dscale, gb.dscale)
    e = mm.block_norm(x[:0], r[:0], post, pre, gate=g[:0], scale=scale, fp8="e4m3", checkpoint="e4m3")
    assert e.y.shape == (0, 264) and e.q.shape == (0, 264)
    ge = mm.block_norm_backward(x[:0], e.kept, post, pre, scale=scale)
    assert ge.dx.shape == (0, 264) and float(ge.dpost_weight.abs().sum() + ge.dscale.abs().sum() + ge.dpre_weight.abs().sum()) == 0
    alone = mm.block_norm_backward(x, a.kept, post, pre, scale=scale, dh=r, dweights=False)
    assert alone.dpost_weight is None and alone.dscale is None and torch.equal(alone.dx, ga.dx)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [256, 300])
def test_block_norm_special_values(mm, dtype, cols):
    x, r, g, post, pre, _ = norm_inputs(8, 8, cols, dtype, "element", False)
    x[0] = 0
    r[0] = 0                                   # a row of zeros
    x[1] = 0                                   # a branch of zeros
    g[2] = -math.inf                           # a branch that is shut, and one that is wide open
    g[3] = math.inf
    x[4, 5] = math.nan
    r[5, 7] = math.inf
    g[6, 9] = math.nan
    got = mm.block_norm(*dev(x, r, post, pre), gate=g.cuda(), fp8="e4m3", checkpoint="e4m3")
    y, h = got.y.cpu().float(), got.h.cpu().float()
    assert float(y[0].abs().sum()) == 0 and float(h[0].abs().sum()) == 0
    assert torch.equal(h[1], r[1].float()) and torch.equal(h[2], r[2].float())
    wy, wh, _, _ = ref.block_norm(x[3:4], r[3:4], post, pre)
    close(got.h[3:4], wh, (U[dtype] + 160 * F24) * (wh.abs() + r[3:4].double().abs()) + TINY[dtype])
    assert bool(torch.isnan(y[4]).all())
    assert math.isinf(float(h[5, 7])) and bool(torch.isfinite(h[5, :7]).all()) and math.isnan(float(y[5, 7])) and float(y[5, 0]) == 0
    assert math.isnan(float(h[6, 9])) and bool(torch.isfinite(h[6, :9]).all()) and bool(torch.isnan(y[6]).all())
    assert bool(torch.isfinite(y[7]).all())
    v = got.kept.gate.dequantize().cpu()       # a block with an infinity or NaN is NaN as a whole
    assert bool(torch.isnan(v[2]).all()) and bool(torch.isnan(v[6, :128]).all()) and bool(torch.isfinite(v[6, 128:]).all())
    # the gradient of shut gates: the branch gets none, and no NaN
    kept = mm.BlockNormKept(*dev(x, h.to(dtype), g), got.kept.rstd_x, got.kept.rstd_h)
    d = mm.block_norm_backward(gen(9, 8, cols).to(dtype).cuda(), kept, *dev(post, pre))
    assert float(d.dx[2].abs().sum()) == 0 and float(d.dgate[2].abs().sum()) == 0 and bool(torch.isfinite(d.dresidual[2]).all())
    assert float(d.dgate[3].abs().sum()) == 0 and bool(torch.isfinite(d.dx[3]).all())


def sums_err(terms, chain):
    return (chain + 6) * F24 * terms.abs().sum(dim=1, keepdim=True)


def check_norm_grad(mm, seed, rows, cols, dtype, gate, scale, alpha=1.0, dh=True, kept=None, wdt=torch.float32, pad=0, offset=0):
    x, h, g, post, pre, scale = norm_inputs(seed, rows, cols, dtype, gate, scale, wdt)
    rx = ((x.double() ** 2).mean(dim=1) + 1e-6).rsqrt().float()
    rh = ((h.double() ** 2).mean(dim=1) + 1e-6).rsqrt().float()
    dy, up = gen(seed + 20, rows, cols).to(dtype), gen(seed + 21, rows, cols).to(dtype) if dh else None
    put = (lambda t: None if t is None else strided(t, pad, offset)) if pad or offset else (lambda t: None if t is None else t.cuda())
    if kept:
        qs = [None if t is None or t.shape[1] != cols else mm.fp8_quantize(t.cuda(), kept)[0] for t in (x, h, g)]
        kx, kh = qs[:2]
        kg = put(g) if qs[2] is None else qs[2]
        x, h = kx.dequantize().cpu(), kh.dequantize().cpu()
        if qs[2] is not None:
            g = qs[2].dequantize().cpu()
    else:
        kx, kh, kg = put(x), put(h), put(g)
    got = mm.block_norm_backward(put(dy), mm.BlockNormKept(kx, kh, kg, rx.cuda(), rh.cuda()), post.cuda(), pre.cuda(),
                                 scale=None if scale is None else scale.cuda(), alpha=alpha, dh=put(up))
    torch.cuda.synchronize()
    wdx, wdr, wdg, wdpost, wdpre, wdscale = ref.block_norm_backward(dy, x, h, rx, rh, post, pre, g, scale, alpha, up)
    # the steps of the kernel with their magnitudes
    u, n = U[dtype], cols
    per_row = g is not None and g.shape[1] != cols
    sig = torch.ones(rows, cols, dtype=torch.float64) if g is None else torch.sigmoid(g.double()).expand(rows, cols)
    se = torch.zeros_like(sig) if g is None else sig_err(g).expand(rows, cols)
    one = 1 - sig if g is None else torch.sigmoid(-g.double()).expand(rows, cols)
    c = post.double() * (1 if scale is None else scale.double())
    r1, r2 = rx.double()[:, None], rh.double()[:, None]
    X, H, a = x.double() * r1, h.double() * r2, dy.double() * pre.double()
    D = wdr / alpha
    mag = (0 if up is None else up.double().abs()) + r2 * a.abs()
    m1, e1 = (a * H).mean(dim=1, keepdim=True), sums_err(a * H, CHAIN) / n
    eD = 8 * F24 * (mag + r2 * (H * m1).abs()) + r2 * H.abs() * e1
    close(got.dresidual, wdr, u * wdr.abs() + abs(alpha) * eD + TINY[dtype], "dresidual")
    e = sig * c * X
    along_e = (sums_err(mag * e, CHAIN) + (mag * e.abs() * se).sum(dim=1, keepdim=True)
               + r2 * m1.abs() * (sums_err(H * e, CHAIN) + (H * e * se).abs().sum(dim=1, keepdim=True))
               + r2 * (e1 + 4 * F24 * m1.abs()) * (H * e).abs().sum(dim=1, keepdim=True))
    b = D * sig * c
    eb = eD * (sig * c).abs() + b.abs() * (4 * F24 + se)
    m2 = (b * X).mean(dim=1, keepdim=True)
    edx = r1 * (eb + X.abs() * along_e / n + 4 * F24 * (b.abs() + (X * m2).abs()))
    close(got.dx, wdx, u * wdx.abs() + edx + TINY[dtype], "dx")
    if g is not None:
        eo = one * 0 + 2 * F24 + se * sig       # of 1 - sigmoid
        if per_row:
            along = (b * X).sum(dim=1, keepdim=True)
            tol = u * wdg.abs() + along.abs() * eo[:, :1] + one[:, :1] * (along_e + 3 * F24 * along.abs()) + TINY[dtype]
        else:
            tol = u * wdg.abs() + (b * X).abs() * (eo + 3 * F24) + one * eb * X.abs() + TINY[dtype]
        close(got.dgate, wdg, tol, "dgate")
        assert got.dgate.shape == g.shape
    else:
        assert got.dgate is None
    t = D * sig
    et = ((eD * sig + t.abs() * (3 * F24 + se)) * X.abs()).sum(dim=0) + (rows + 50) * F24 * (t * X).abs().sum(dim=0)
    close(got.dpost_weight, wdpost, et * (1 if scale is None else scale.double().abs()) + 2 * F24 * wdpost.abs(), "dpost")
    close(got.dpre_weight, wdpre, (rows + 50) * F24 * (dy.double() * H).abs().sum(dim=0), "dpre")
    if scale is not None:
        close(got.dscale, wdscale, et * post.double().abs() + 2 * F24 * wdscale.abs(), "dscale")
    else:
        assert got.dscale is None
    return got


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_block_norm_backward_matches_oracle(mm, dtype, shape):
    check_norm_grad(mm, 10, *shape, dtype, "element", True)
    check_norm_grad(mm, 11, *shape, dtype, "element", True, kept="e4m3")
    check_norm_grad(mm, 12, *shape, dtype, "row", False, alpha=0.5, kept="e5m2")
    check_norm_grad(mm, 13, *shape, dtype, "none", True, alpha=-2.0, dh=False)


@gpu
@pytest.mark.parametrize("kept", [None, "e4m3"])
@pytest.mark.parametrize("cols", [64, 100, 512, 1024, 1500, 4096, 6000, 16384, 16400])
def test_block_norm_backward_many_rows(mm, cols, kept):
    rows = 1300 if cols <= 1500 else 700
    check_norm_grad(mm, 14, rows, cols, torch.bfloat16, "element", True, kept=kept)


@gpu
def test_block_norm_backward_matches_differences(mm):
    """fp32, against central differences of the forward kernel's own outputs."""
    rows, cols = 4, 96
    x, r, g, post, pre, scale = dev(*norm_inputs(15, rows, cols, torch.float32, "element", True))
    v, t = gen(30, rows, cols).cuda(), gen(31, rows, cols).cuda()
    out = mm.block_norm(x, r, post, pre, gate=g, scale=scale, alpha=0.5)
    d = mm.block_norm_backward(v, out.kept, post, pre, scale=scale, alpha=0.5, dh=t)

    def loss(x, r, post, pre, scale, g):
        o = mm.block_norm(x, r, post, pre, gate=g, scale=scale, alpha=0.5)
        return float((o.y.double() * v.double()).sum() + (o.h.double() * t.double()).sum())

    args = [x, r, post, pre, scale, g]
    for i, grad in enumerate((d.dx, d.dresidual, d.dpost_weight, d.dpre_weight, d.dscale, d.dgate)):
        way = gen(40 + i, *args[i].shape).cuda()
        eps = 1e-2
        up = loss(*(a + eps * way if k == i else a for k, a in enumerate(args)))
        down = loss(*(a - eps * way if k == i else a for k, a in enumerate(args)))
        want = float((grad.double() * way.double()).sum())
        # the cubic term of the differences: eps^2 times a third derivative of the size of the loss's terms, which sum to
        # at most the gradient's and the direction's lengths; rounding adds 2^-24 of 400 terms over eps
        assert abs((up - down) / (2 * eps) - want) < 1e-3 * float(grad.double().norm() * way.double().norm()) + 1e-2


# ---------------------------------------------------------------- gated activation

GATED_SHAPES = [(1, 1), (3, 8), (129, 127), (2, 513), (130, 256), (7, 1000), (257, 640), (1, 14336), (3, 20001)]


def act_err(g, kind, dtype):
    """(error of f, error of f') for gate values g of data of `dtype`."""
    g = g.double()
    f, slope = ref.activation(g, kind)
    if kind == "silu":
        # where 1 + exp(-g) is above 2^126 (g below -87.3) its reciprocal leaves fp32's normal range and may count as 0:
        # the sigmoid is then off by at most 2^-126, f by |g| and f' by 1 + |g| times that
        s, low = torch.sigmoid(g), 2.0 ** -126
        return (f.abs() * (sig_err(g) + 2 * F24) + g.abs() * low,
                s * sig_err(g) * (1 + g.abs()) + 4 * F24 * (f.abs() + s) + (1 + g.abs()) * low)
    if dtype != torch.float32:
        # Phi = t R(t) exp(-g^2 / 2) / 2 in its lower tail: R fitted to 2.7 2^-24 and evaluated with 10 roundings (6), t off by
        # 3 (a reciprocal and a sum), which counts twice in t R(t), three products (3); the exponential by 2 units (4) and
        # the three roundings of its argument, 1.5 g^2 in all.  Below 2^-126 it may count as 0
        phi, low = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), 2.0 ** -126
        bell = g.abs() * torch.exp(-0.5 * g * g) * 0.4
        return (f.abs() * (24 + 1.6 * g * g) * F24 + g.abs() * low,
                phi * (22 + 1.5 * g * g) * F24 + bell * (8 + 1.5 * g * g) * F24 + F24 * slope.abs() + (1 + g.abs()) * low)
    # Phi: 5 units in the last place, below fp32's normal range 2^-149 of its own and f |g| times that;
    # exp(-g^2 / 2): 2 + 1.17 g^2 / 2 units, and two roundings of its argument, g^2 / 2 2^-24 each
    phi = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
    bell = g.abs() * torch.exp(-0.5 * g * g) * 0.4
    tiny = TINY[torch.float32]
    return f.abs() * 12 * F24 + (1 + g.abs()) * tiny, phi * 12 * F24 + bell * (10 + 2.2 * g * g) * F24 + F24 * slope.abs() + tiny


def gated_inputs(seed, rows, cols, dtype):
    return gen(seed, rows, cols, std=2.0).to(dtype), gen(seed + 1, rows, cols).to(dtype)


def check_gated(mm, g, u, kind, fp8=None, checkpoint=None, y=True, run=None):
    dg, du = run or dev(g, u)
    got = mm.gated_activation(dg, du, activation=kind, fp8=fp8, y=y, checkpoint=checkpoint)
    torch.cuda.synchronize()
    want = ref.gated(g, u, kind)
    err = act_err(g, kind, g.dtype)[0] * u.double().abs() + 2 * F24 * want.abs()
    assert (got.y is not None) == y and (got.q is not None) == (fp8 is not None)
    if y:
        close(got.y, want, U[g.dtype] * want.abs() + err + TINY[g.dtype], "y")
    if fp8:
        check8(got.q, want, err, fp8, "q")
        if y and g.dtype == torch.float32:
            check8_exact(got.q, got.y.cpu(), fp8)
    if checkpoint:
        check8_exact(got.kept.gate, g, checkpoint)
        check8_exact(got.kept.up, u, checkpoint)
    else:
        assert got.kept.gate is dg and got.kept.up is du


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("shape", GATED_SHAPES)
def test_gated_activation_matches_oracle(mm, dtype, kind, shape):
    g, u = gated_inputs(50, *shape, dtype)
    check_gated(mm, g, u, kind, fp8="e4m3", checkpoint="e4m3")
    check_gated(mm, g, u, kind, fp8="e5m2", checkpoint="e5m2", y=False)
    check_gated(mm, g, u, kind)


def check_gated_grad(mm, seed, rows, cols, dtype, kind, kept=None, fp8="e5m2", y_fp8="e4m3", dense=True, put=None):
    put = put or (lambda t: t.cuda())
    g, u = gated_inputs(seed, rows, cols, dtype)
    dy = (gen(seed + 2, rows, cols) * torch.exp(gen(seed + 3, rows, 1))).to(dtype)
    if kept:
        kg, ku = mm.fp8_quantize(g.cuda(), kept)[0], mm.fp8_quantize(u.cuda(), kept)[0]
        g, u = kg.dequantize().cpu(), ku.dequantize().cpu()
    else:
        kg, ku = put(g), put(u)
    got = mm.gated_activation_backward(put(dy), mm.GatedKept(kg, ku), activation=kind, dense=dense, fp8=fp8, y_fp8=y_fp8)
    torch.cuda.synchronize()
    wg, wu, wy = ref.gated_backward(dy, g, u, kind)
    ef, es = act_err(g, kind, dtype)
    d, ua = dy.double().abs(), u.double().abs()
    eg, eu, ey = d * ua * es + 3 * F24 * wg.abs(), d * ef + 2 * F24 * wu.abs(), ef * ua + 2 * F24 * wy.abs()
    lost = TINY[torch.float32]
    eg, eu, ey = eg + lost, eu + lost, ey + lost
    if dense:
        close(got.dgate, wg, U[dtype] * wg.abs() + eg + TINY[dtype], "dgate")
        close(got.dup, wu, U[dtype] * wu.abs() + eu + TINY[dtype], "dup")
    else:
        assert got.dgate is None and got.dup is None
    if fp8:
        for q, w, e in ((got.dgate_rows, wg, eg), (got.dup_rows, wu, eu)):
            check8(q, w, e, fp8, "rows")
        for q, w, e in ((got.dgate_cols, wg, eg), (got.dup_cols, wu, eu)):
            check8(q, w.t().contiguous(), e.t().contiguous(), fp8, "cols")
        if dense and dtype == torch.float32:  # the dense ones are the unrounded values that were quantised
            check8_exact(got.dgate_rows, got.dgate.cpu(), fp8)
            check8_exact(got.dup_cols, got.dup.cpu().t(), fp8)
    else:
        assert got.dgate_rows is got.dgate_cols is got.dup_rows is got.dup_cols is None
    if y_fp8:
        check8(got.y_cols, wy.t().contiguous(), ey.t().contiguous(), y_fp8, "y")
    else:
        assert got.y_cols is None
    return got


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("shape", GATED_SHAPES)
def test_gated_activation_backward_matches_oracle(mm, dtype, kind, shape):
    check_gated_grad(mm, 60, *shape, dtype, kind)
    check_gated_grad(mm, 61, *shape, dtype, kind, kept="e4m3", dense=False)
    check_gated_grad(mm, 62, *shape, dtype, kind, kept="e5m2", fp8="e4m3", y_fp8="e5m2")
    check_gated_grad(mm, 63, *shape, dtype, kind, fp8=None, y_fp8=None)
    check_gated_grad(mm, 64, *shape, dtype, kind, kept="e4m3", fp8=None, dense=False)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
def test_gated_strides_and_alignment(mm, dtype, pad, offset):
    g, u = gated_inputs(70, 150, 264, dtype)
    check_gated(mm, g, u, "silu", fp8="e4m3", checkpoint="e4m3", run=[strided(g, pad, offset), strided(u, pad, offset)])
    check_gated_grad(mm, 71, 150, 264, dtype, "silu", put=lambda t: strided(t, pad, offset))
    both = torch.cat([g, u], dim=1).cuda()    # the halves of one product, and more dimensions
    a = mm.gated_activation(both[:, :264], both[:, 264:], fp8="e4m3")
    b = mm.gated_activation(g.cuda(), u.cuda(), fp8="e4m3")
    assert torch.equal(a.y, b.y)
    c = mm.gated_activation(g.cuda().view(3, 50, 264), u.cuda().view(3, 50, 264), fp8="e4m3")
    assert c.y.shape == (3, 50, 264) and c.q.shape == (150, 264) and torch.equal(c.y.view(150, 264), b.y)
    e = mm.gated_activation(both[:0, :264], both[:0, 264:], fp8="e4m3", checkpoint="e4m3")
    assert e.y.shape == (0, 264)
    ge = mm.gated_activation_backward(both[:0, :264], e.kept, fp8="e5m2", y_fp8="e4m3")
    assert ge.dgate.shape == (0, 264) and ge.dgate_cols.shape == (264, 0)


@gpu
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_special_values(mm, kind):
    g, u = gated_inputs(80, 140, 300, torch.float32)
    g[:4] = 0
    u[4] = 0
    g[5] = torch.linspace(-100, 100, 300)
    got = mm.gated_activation(*dev(g, u), activation=kind)
    assert float(got.y[:5].abs().sum()) == 0
    check_gated(mm, g, u, kind, fp8="e4m3", checkpoint="e4m3")
    g[6, 140], u[7, 3], g[8, 299] = math.nan, math.inf, math.nan
    got = mm.gated_activation(*dev(g, u), activation=kind, fp8="e4m3", checkpoint="e4m3")
    bad = torch.isnan(got.q.dequantize().cpu())
    assert bool(bad[6, 128:256].all()) and bool(bad[7, :128].all()) and bool(bad[8, 256:].all()) and int(bad.sum()) == 128 * 2 + 44
    dy = torch.ones(140, 300, device="cuda")
    d = mm.gated_activation_backward(dy, got.kept, activation=kind, dense=False, fp8="e5m2", y_fp8="e4m3")
    v = torch.isnan(d.dup_rows.dequantize().cpu())
    assert bool(v[6, 128:256].all()) and bool(v[8, 256:].all()) and int(v.sum()) == 128 + 44    # dup reads the gate alone
    w = torch.isnan(d.dup_cols.dequantize().cpu())
    assert bool(w[128:256, :128].all()) and bool(w[256:, :128].all()) and int(w.sum()) == 128 * (128 + 44)


# ---------------------------------------------------------------- transposition

def transposed_exactly(q):
    """(data, scale bytes) of the definition: q's values transposed and quantised."""
    v = ref8.values(q.data.cpu(), q.scale.view(torch.uint8).cpu())
    data, exps = ref8.quantize(v.t(), q.fmt)
    return data, kept_scales(exps)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 640), (130, 7), (129, 385), (5, 1030), (256, 512), (777, 100), (16, 20001)])
def test_transpose_is_exact(mm, fmt, shape):
    x = gen(90, *shape) * torch.exp(3 * gen(91, shape[0], 1)) * torch.exp(2 * gen(92, 1, shape[1]))
    x[:, ::7] *= 2.0 ** -20                    # values that end up below the normal range
    x[::5] = 0
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    t = mm.fp8_transpose(q)
    data, scale = transposed_exactly(q)
    assert t.shape == shape[::-1] and t.fmt == fmt
    assert torch.equal(t.data.float().cpu().double(), data) and torch.equal(t.scale.view(torch.uint8).cpu(), scale)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("spread", [0, 8, 13, 14, 15, 99, 100, 101])
@pytest.mark.parametrize("low", [1.0, 2.0 ** -14, 2.0 ** -16, 2.0 ** -73, 2.0 ** -78])
def test_transpose_at_the_limits_of_16_bits(mm, fmt, spread, low):
    """Rows whose scales are as far apart as the two-at-a-time way takes, and a little more; columns that are small
    everywhere; the type's smallest values."""
    rows = torch.linspace(0, spread, 200).round()
    rows[128:] -= torch.where(torch.arange(72) % 3 == 0, spread // 2 + 1, 0)    # some rows above the tile's first, too
    x = gen(98, 200, 256) * 2.0 ** -rows[:, None]
    x[130], x[150:] = 0.0, x[150:] * (torch.arange(50) % 4 > 0)[:, None]        # rows of zeros, whose scale is 1
    x[:, 1::3] *= low
    x[7, 9], x[:, 200] = 0.0, -0.0
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    t = mm.fp8_transpose(q)
    data, scale = transposed_exactly(q)
    assert torch.equal(t.data.float().cpu().double(), data) and torch.equal(t.scale.view(torch.uint8).cpu(), scale)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_transpose_over_the_whole_range(mm, fmt):
    """Every byte under every scale, far apart within a column."""
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    b = torch.randint(0, 256, (700, 300), generator=torch.Generator().manual_seed(1)).to(torch.uint8)
    b[~torch.isfinite(b.view(dt).float())] = 0x12
    pitch = 304
    data = torch.zeros(700, pitch, dtype=torch.uint8, device="cuda")
    data[:, :300] = b.cuda()
    scale = torch.randint(0, 246 if fmt == "e4m3" else 239, (1, 700, 4), generator=torch.Generator().manual_seed(2)).to(torch.uint8)
    scale[:, 128:256] = 0
    scale[:, 256:384] //= 8
    q = mm.Fp8Tensor(data.view(dt)[:, :300], scale.cuda())
    t = mm.fp8_transpose(q)
    want, exps = transposed_exactly(q)
    assert torch.equal(t.scale.view(torch.uint8).cpu(), exps)
    assert torch.equal(t.data.float().cpu().double(), want)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_transpose_marks_what_is_not_finite(mm, fmt):
    x = gen(93, 300, 400)
    x[10, 140] = math.nan
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    t = torch.isnan(mm.fp8_transpose(q).dequantize().cpu())
    assert bool(t[128:256, :128].all()) and int(t.sum()) == 128 * 128
    q, _ = mm.fp8_quantize(gen(94, 300, 400).cuda(), fmt)   # a NaN byte, and an infinity, under ordinary scales
    q.data.view(torch.uint8)[200, 33] = 0x7f
    if fmt == "e5m2":
        q.data.view(torch.uint8)[299, 34] = 0xfc
    t = torch.isnan(mm.fp8_transpose(q).dequantize().cpu())
    assert bool(t[33, 128:256].all()) and int(t.sum()) == 128 + (44 if fmt == "e5m2" else 0)


@gpu
def test_transpose_shapes_at_the_end_of_an_allocation(mm):
    """A single row whose data is not padded, and no rows or columns."""
    x = gen(95, 1, 100).cuda()
    q, _ = mm.fp8_quantize(x)
    tight = mm.Fp8Tensor(q.data[0, :100].clone().view(1, 100), q.scale)
    a, b = mm.fp8_transpose(q), mm.fp8_transpose(tight)
    assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8))
    e = mm.fp8_transpose(mm.Fp8Tensor.empty(0, 300))
    assert e.shape == (300, 0)


# ---------------------------------------------------------------- streams, graphs, repeated calls

@gpu
def test_calls_on_another_stream_and_in_a_graph(mm):
    ins = norm_inputs(100, 300, 1032, torch.bfloat16, "element", True)
    x, r, g, post, pre, scale = dev(*ins)

    def step(stream=None):
        o = mm.block_norm(x, r, post, pre, gate=g, scale=scale, fp8="e4m3", checkpoint="e4m3", stream=stream)
        d = mm.block_norm_backward(r, o.kept, post, pre, scale=scale, dh=x, stream=stream)
        a = mm.gated_activation(x, g, fp8="e4m3", checkpoint="e4m3", stream=stream)
        b = mm.gated_activation_backward(r, a.kept, fp8="e5m2", y_fp8="e4m3", stream=stream)
        t = mm.fp8_transpose(o.q, stream=stream)
        return [o.y, o.h, d.dx, d.dresidual, d.dgate, d.dpost_weight, d.dpre_weight, d.dscale, a.y, b.dgate, b.dup,
                t.data.view(torch.uint8), b.y_cols.data.view(torch.uint8), b.dgate_cols.data.view(torch.uint8)]

    first = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, b in zip(first, step(side)):
        side.synchronize()
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- together, as a training step runs them

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_checkpoint_step.py")
    spec = importlib.util.spec_from_file_location("fp8_checkpoint_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@gpu
def test_example_gradients_match_autograd(mm):
    """The example's forward and backward pass from 8-bit checkpoints against fp32 autograd of the same model."""
    ex = _example()
    model = ex.Network(2, 256, 384, seed=3)
    for i, v in enumerate(model.vectors):
        v += 0.2 * gen(200 + i, 256).cuda()
    x, dy = gen(1, 300, 256).bfloat16().cuda(), gen(2, 300, 256).bfloat16().cuda()
    y, saved = model.forward(x)
    matrices, vectors = model.backward(dy, saved)
    ws = [w.master.float().requires_grad_() for w in model.weights]
    vs = [v.clone().requires_grad_() for v in model.vectors]
    norm = lambda t, w: t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    s, n = x.float(), norm(x.float(), vs[0])
    for i in range(2):
        branch, up, down, gate = ws[4 * i:4 * i + 4]
        post, pre, scale = vs[1 + 3 * i:4 + 3 * i]
        o = (torch.nn.functional.silu(n @ branch.t()) * (n @ up.t())) @ down.t()
        s = s + torch.sigmoid(n @ gate.t()) * scale * norm(o, post)
        n = norm(s, pre)
    (n * dy.float()).sum().backward()
    # an 8-bit matrix is off by 2^-4 (e4m3) or 2^-3 (e5m2) of its values at most, a third of that in the mean square; a
    # gradient of the first block has passed at most 17 of them (in each block three checkpoints of the norms, two of
    # the branches, two operands of gradients and two weights, less one weight)
    far = lambda a, b: float((a.float() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    limit = 17 ** 0.5 * 2.0 ** -3 / 3 ** 0.5
    assert far(y, n) < limit
    for got, want in zip(matrices + vectors, ws + vs):
        assert got.shape == want.shape and far(got, want.grad) < limit
    # 5 matrices of `width` columns' size in 8 bits and 2 of `hidden`: at most 8 / 7 of their bytes with scales and factors
    assert ex.kept_bytes(saved) < 2 * 300 * (4 * 256 + 2 * 384) * 8 / 7


@gpu
def test_example_runs(mm):
    losses, norms = _example().train(steps=4, tokens=1024, log=lambda *_: None)
    assert all(math.isfinite(v) for v in losses + norms) and min(norms) > 0


@gpu
def test_backward_captured_while_an_eager_graph_of_the_same_leaves_lives(mm):
    """The calls take no part in autograd: they are captured into a graph beside one that autograd holds."""
    x = gen(1, 64, 256).cuda().requires_grad_()
    loss = (x * x).sum()
    w = torch.ones(256, device="cuda")
    o = mm.block_norm(x.detach(), x.detach(), w, w)
    d = mm.block_norm_backward(x.detach(), o.kept, w, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2 = mm.block_norm(x, x, w, w)
        d2 = mm.block_norm_backward(x, o2.kept, w, w)
    graph.replay()
    torch.cuda.synchronize()
    assert not o2.y.requires_grad and torch.equal(d.dx, d2.dx)
    loss.backward()
    assert torch.equal(x.grad, 2 * x.detach())


@gpu
def test_offsets_past_32_bits(mm):
    """Matrices of more than 2^31 elements and bytes: their last rows equal those of the same rows alone."""
    rows, cols = 66_003, 33_000
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    raw = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    end = x[-7:].contiguous()
    a, b = mm.gated_activation(x, x, fp8="e4m3", checkpoint="e4m3"), mm.gated_activation(end, end, fp8="e4m3", checkpoint="e4m3")
    assert torch.equal(a.y[-7:], b.y) and torch.equal(raw(a.q.data[-7:]), raw(b.q.data)) and torch.equal(a.q.scales()[-7:], b.q.scales())
    assert torch.equal(raw(a.kept.up.data[-7:]), raw(b.kept.up.data))
    d = mm.gated_activation_backward(x, a.kept, fp8="e5m2", dense=False)
    e = mm.gated_activation_backward(end, b.kept, fp8="e5m2", dense=False)
    assert torch.equal(raw(d.dup_rows.data[-7:]), raw(e.dup_rows.data)) and torch.equal(d.dgate_rows.scales()[-7:], e.dgate_rows.scales())
    del d, e
    t = mm.fp8_transpose(a.q)
    last = a.q.dequantize()[-83:, -3:]          # the last block of rows: 66003 = 515 * 128 + 83
    assert torch.allclose(t.dequantize()[-3:, -83:].t(), last, rtol=2.0 ** -4, atol=float(last.abs().max()) * 2.0 ** -18)
    del t, a, b
    w = torch.ones(cols, device="cuda")
    m, n = mm.block_norm(x, x, w, w, gate=x, checkpoint="e4m3"), mm.block_norm(end, end, w, w, gate=end, checkpoint="e4m3")
    assert torch.equal(m.y[-7:], n.y) and torch.equal(m.h[-7:], n.h) and torch.equal(raw(m.kept.gate.data[-7:]), raw(n.kept.gate.data))
    g, h = mm.block_norm_backward(x, m.kept, w, w, dh=x, dweights=False), mm.block_norm_backward(end, n.kept, w, w, dh=end, dweights=False)
    assert torch.equal(g.dx[-7:], h.dx) and torch.equal(g.dgate[-7:], h.dgate) and torch.equal(g.dresidual[-7:], h.dresidual)


@gpu
@pytest.mark.parametrize("cols", [9, 120, 515, 1300])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (1, 1), (5, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_with_strides_leave_what_lies_between_their_rows(mm, dtype, cols, pad, offset):
    """The C entry points with outputs of any stride and alignment: values as for contiguous ones, and nothing else written."""
    from newton_schulz_04_gb300 import blocks
    rows, lib, st = 21, mm.load(), torch.cuda.current_stream().cuda_stream
    code = {torch.bfloat16: 0, torch.float32: 1}[dtype]
    x, r, g, post, pre, scale = dev(*norm_inputs(110, rows, cols, dtype, "element", True))
    dy = gen(111, rows, cols).to(dtype).cuda()
    buffers = []

    def out():
        buf = torch.full((rows * (cols + pad) + offset + 16,), 5.0, dtype=dtype, device="cuda")
        v = buf[offset:].as_strided((rows, cols), (cols + pad, 1))
        buffers.append((buf, v))
        return v

    def same(v, want):
        assert torch.equal(v, want)
        v.fill_(5.0)

    ld = cols + pad
    want = mm.block_norm(x, r, post, pre, gate=g, scale=scale)
    y, h = out(), out()
    stats = torch.empty(2, rows, device="cuda")
    assert lib.muon_block_norm(blocks._BLOCK_NORM(
        x.data_ptr(), cols, r.data_ptr(), cols, g.data_ptr(), cols, post.data_ptr(), scale.data_ptr(), pre.data_ptr(), y.data_ptr(), ld,
        h.data_ptr(), ld, stats[0].data_ptr(), stats[1].data_ptr(), *([0] * 12), rows, cols, code, 1, 0, 0, 0, 1.0, 1e-6), st) == 0
    same(y, want.y), same(h, want.h)
    grads = mm.block_norm_backward(dy, want.kept, post, pre, scale=scale, dh=r)
    dx, dr, dg = out(), out(), out()
    assert lib.muon_block_norm_backward(blocks._BLOCK_NORM_GRAD(
        dy.data_ptr(), cols, r.data_ptr(), cols, x.data_ptr(), 0, cols, want.h.data_ptr(), 0, cols, g.data_ptr(), 0, cols,
        want.kept.rstd_x.data_ptr(), want.kept.rstd_h.data_ptr(), post.data_ptr(), scale.data_ptr(), pre.data_ptr(), dx.data_ptr(), ld,
        dr.data_ptr(), ld, dg.data_ptr(), ld, 0, 0, 0, 0, 0, rows, cols, code, 1, 0, 0, 1.0), st) == 0
    same(dx, grads.dx), same(dr, grads.dresidual), same(dg, grads.dgate)
    a = mm.gated_activation(g, x)
    y = out()
    assert lib.muon_gated_activation(blocks._GATED(g.data_ptr(), cols, x.data_ptr(), cols, y.data_ptr(), ld, *([0] * 9), rows, cols, code, 0, 0,
                                                   0), st) == 0
    same(y, a.y)
    for eight in (False, True):   # the two kernels
        b = mm.gated_activation_backward(dy, a.kept, y_fp8="e4m3" if eight else None)
        dg, du = out(), out()
        q = [b.y_cols.data.data_ptr(), b.y_cols.scale.data_ptr(), b.y_cols._ld()] if eight else [0, 0, 0]
        assert lib.muon_gated_activation_backward(blocks._GATED_GRAD(
            dy.data_ptr(), cols, g.data_ptr(), 0, cols, x.data_ptr(), 0, cols, dg.data_ptr(), ld, du.data_ptr(), ld, *([0] * 12), *q, rows, cols,
            code, 0, 0, 0, 0), st) == 0
        same(dg, b.dgate), same(du, b.dup)
    torch.cuda.synchronize()
    for buf, _ in buffers:
        assert bool((buf == 5.0).all())


@gpu
def test_calls_give_the_same_bits_again(mm):
    x, r, g, post, pre, scale = dev(*norm_inputs(120, 1000, 1100, torch.bfloat16, "element", True))
    a = mm.block_norm(x, r, post, pre, gate=g, scale=scale, checkpoint="e4m3")
    first = mm.block_norm_backward(x, a.kept, post, pre, scale=scale, dh=r)
    for _ in range(5):
        for one, two in zip(first, mm.block_norm_backward(x, a.kept, post, pre, scale=scale, dh=r)):
            assert torch.equal(one, two)
