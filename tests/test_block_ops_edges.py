"""Edges of the norms around a block, the gated activation and 8-bit checkpoints: the ends of the types' ranges, masked gates,
gates that are wide open, where memory lies."""
import math

import pytest
import torch

import oracle.blocks as ref
import test_block_ops as block_ops
from test_block_ops import (  # noqa: F401
    DTYPES, F24, check8_exact, close, dev, gen, gpu, mm, norm_inputs, transposed_exactly,
)

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


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("cols", [256, 300])
def test_gradient_from_checkpoints_of_the_largest_finite_values(mm, dtype, fmt, kind, cols):
    """Gates at both ends of the type's range, and linear branches: their 8-bit copies stand for +-2^128, of which the
    gradient's values are those of the largest finite number, within a rounding."""
    lim = torch.finfo(dtype)
    g, u, dy = (t.clone() for t in (torch.zeros(9, cols), torch.full((9, cols), 0.5), torch.full((9, cols), 0.5)))
    g[1, :] = lim.min                          # shut, open, and beside them gates that 8 bits round to 0 under such a scale
    g[2, ::3], g[3, 5], g[4, 130] = lim.min, lim.max, lim.max
    g[7], g[8] = 1.0, gen(2, cols)
    u[5], u[6, 1::2] = lim.max, lim.min
    a = mm.gated_activation(*dev(g.to(dtype), u.to(dtype)), activation=kind, checkpoint=fmt)
    kg, ku = (torch.where(t.abs() >= lim.max / 2, t.sign() * 2.0 ** 128, t.double()) for t in (g.double(), u.double()))
    for t in (kg, ku):                         # what the copies stand for, of the values as they are here
        block = torch.arange(cols) // 128
        for r in range(9):
            for b in range(int(block[-1]) + 1):
                if float(t[r, block == b].abs().max()) > 1e38:
                    t[r, (block == b) & (t[r].abs() < 1e38)] = 0.0
    kg[8] = mm.fp8_quantize(g[8:].to(dtype).cuda(), fmt)[0].dequantize().cpu().double()[0]
    wg, wu, _ = ref.gated_backward(dy, kg, ku, kind)
    for fp8 in (None, "e5m2"):                 # the two kernels
        d = mm.gated_activation_backward(dy.to(dtype).cuda(), a.kept, activation=kind, fp8=fp8)
        u_, tol = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype], 64 * F24
        close(d.dgate, wg, (u_ + tol) * wg.abs() + tol * 0.25 * ku.abs().clamp(max=1.0), "dgate")
        close(d.dup, wu, (u_ + tol) * wu.abs(), "dup")
        if fp8:
            for q, w in ((d.dgate_rows, wg), (d.dup_rows, wu), (d.dgate_cols, wg.t()), (d.dup_cols, wu.t())):
                assert not bool(torch.isnan(q.data.float()).any())


# ---------------------------------------------------------------- gates that are wide open

@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kept", [None, "e4m3"])
@pytest.mark.parametrize("cols", [5, 264, 1000, 8200, 40_000])
def test_gradient_of_open_gates(mm, dtype, kept, cols):
    """dgate = sigmoid(g) sigmoid(-g) ... of gates from 8 to 80, whose sigmoids are 1 but for 2^-12 to 2^-115 of it: relative to
    the value.  Without dy the stream's gradient is dh, so that nothing else of it cancels."""
    rows = 6
    x, h, _, post, pre, scale = norm_inputs(30, rows, cols, dtype, "none", True)
    dh = gen(31, rows, cols).to(dtype)
    rx, rh = ((t.double() ** 2).mean(dim=1).rsqrt().float() for t in (x, h))
    steps = torch.tensor([-80.0, -20.0, -8.0, 8.0, 10.0, 12.0, 16.0, 20.0, 40.0, 80.0])
    gate = steps[torch.arange(rows * cols) % 10].view(rows, cols).to(dtype)
    per_row = steps[3:3 + rows, None].to(dtype)
    X, c = x.double() * rx.double()[:, None], post.double() * scale.double()
    # an exponential (2 + 1.17 |g| units) counts twice, in exp(-g) and the sigmoid; two roundings each of theirs, six products'
    rel = lambda g: (2 * (4 + 1.2 * g.double().abs()) * 2 + 10) * F24  # noqa: E731
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: F24}[dtype]
    tiny = torch.finfo(dtype).smallest_normal * u * 2
    for g in (gate, per_row):
        if kept:
            qx, qh = (mm.fp8_quantize(t.cuda(), kept)[0] for t in (x, h))
            kg = mm.fp8_quantize(g.cuda(), kept)[0] if g is gate else g.cuda()
            state = mm.BlockNormKept(qx, qh, kg, rx.cuda(), rh.cuda())
            xs, gs = qx.dequantize().cpu().double() * rx.double()[:, None], kg.dequantize().cpu() if g is gate else g
        else:
            state, xs, gs = mm.BlockNormKept(*dev(x, h, g, rx, rh)), X, g
        d = mm.block_norm_backward(torch.zeros_like(dh).cuda(), state, *dev(post, pre), scale=scale.cuda(), dh=dh.cuda())
        s, shut = torch.sigmoid(gs.double()), torch.sigmoid(-gs.double())
        along = dh.double() * s * c * xs
        if g is gate:
            close(d.dgate, along * shut, ((u + rel(gs)) * along.abs() * shut + tiny), "dgate")
        else:                                  # a sum of at most 140 terms one after another, and those of its roundings
            total = along.abs().sum(dim=1, keepdim=True) * shut
            close(d.dgate, along.sum(dim=1, keepdim=True) * shut, (u + 150 * F24 + rel(gs)) * total + tiny, "dgate of rows")


# ---------------------------------------------------------------- transposition

@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scales", [(0, 1), (120, 136), (130, 131), (200, 239), (0, 239)])
def test_transpose_of_any_scales(mm, fmt, scales):
    """Rows whose scale bytes lie in a range, small and large, near one another and not; values of every size."""
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    g = torch.Generator().manual_seed(7)
    b = torch.randint(0, 256, (300, 208), generator=g).to(torch.uint8)
    b[~torch.isfinite(b.view(dt).float())] = 0x38
    scale = torch.randint(*scales, (1, 300, 4), generator=g).to(torch.uint8)
    q = mm.Fp8Tensor(b.cuda().view(dt), scale.cuda())
    t = mm.fp8_transpose(q)
    data, want = transposed_exactly(q)
    assert torch.equal(t.scale.view(torch.uint8).cpu(), want) and torch.equal(t.data.float().cpu().double(), data)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("size", [2.0 ** -120, 1e-6, 1.0, 300.0, 1e9, 2.0 ** 100])
@pytest.mark.parametrize("zeros", [1, 31, 33, 128, 200])
def test_transpose_of_rows_behind_zeros(mm, fmt, size, zeros):
    """Tiles that begin with rows of zeros, whose scales are 1 whatever the others' are."""
    x = gen(40, 270, 160) * size
    x[:zeros], x[256:256 + zeros % 14] = 0.0, 0.0
    x[250, :128] = 0.0
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    t = mm.fp8_transpose(q)
    data, want = transposed_exactly(q)
    assert torch.equal(t.scale.view(torch.uint8).cpu(), want) and torch.equal(t.data.float().cpu().double(), data)


# ---------------------------------------------------------------- the gradient's workspace

PARTS = [(256, 0, 608), (1024, 0, 608), (2048, 0, 304), (4096, 0, 152), (8192, 0, 76), (16384, 0, 38), (32768, 0, 19), (32769, 0, 304),
         (512, 1, 608), (1024, 1, 304), (2048, 1, 152), (4096, 1, 76), (16384, 1, 19), (16385, 1, 304)]


@pytest.mark.parametrize("cols,dt,parts", PARTS)
def test_workspace_of_the_norm_gradient(mm, cols, dt, parts):
    """Two fp32 rows for each CTA or cluster that can run, no more; a call asks for as much and no more."""
    from test_block_ops import P, norm_grad_call
    lib = mm.load()
    size = lib.muon_block_norm_backward_workspace_bytes_for(4_194_304, cols, dt)
    assert size == parts * 2 * cols * 4
    assert lib.muon_block_norm_backward_workspace_bytes_for(3, cols, dt) == min(3, parts) * 2 * cols * 4
    most = lib.muon_block_norm_backward_workspace_bytes(4_194_304, cols)
    assert most == max(lib.muon_block_norm_backward_workspace_bytes_for(4_194_304, cols, d) for d in (0, 1, 2))
    far = dict(rows=200_000, cols=cols, dt=dt, dpre=P[10], ws=P[11])
    far |= {k: cols for k in ("lddy", "lddh", "ldx", "ldh", "ldg", "lddx", "lddr", "lddg")}
    far |= {k: (1 << 40) * (i + 1) for i, k in enumerate(("dy", "x", "h", "rx", "rh", "dx", "dr"))}
    assert norm_grad_call(mm, **far, bytes=size - 1) == 4
    if not torch.cuda.is_available():          # enough: the next thing that is missing is the device
        assert norm_grad_call(mm, **far, bytes=size) not in (0, 1, 2, 3, 4)
    for bad in ((-1, 64, 0), (4, 0, 0), (4, 65537, 0), (4, 64, 7)):
        assert lib.muon_block_norm_backward_workspace_bytes_for(*bad) == 0


@gpu
@pytest.mark.parametrize("kept", [None, "e4m3"])
@pytest.mark.parametrize("cols,dtype", [(c, torch.float32 if d else torch.bfloat16) for c, d, _ in PARTS] + [(65_536, torch.float16)])
def test_norm_gradient_stays_within_its_workspace(mm, cols, dtype, kept):
    from newton_schulz_04_gb300 import blocks
    rows, lib, st = 900 if cols < 8192 else 340, mm.load(), torch.cuda.current_stream().cuda_stream
    x, r, g, post, pre, scale = dev(*norm_inputs(50, rows, cols, dtype, "element", True))
    o = mm.block_norm(x, r, post, pre, gate=g, scale=scale, checkpoint=kept)
    want = mm.block_norm_backward(r, o.kept, post, pre, scale=scale, dh=x)
    code = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}[dtype]
    size = lib.muon_block_norm_backward_workspace_bytes_for(rows, cols, code)
    ws = torch.full((size + 65_536,), 77, dtype=torch.uint8, device="cuda")
    sums = torch.empty(3, cols, device="cuda")
    k = [blocks._kept("k", t, r, rows, cols)[:3] for t in (o.kept.x, o.kept.h, o.kept.gate)]
    assert lib.muon_block_norm_backward(blocks._BLOCK_NORM_GRAD(
        r.data_ptr(), cols, x.data_ptr(), cols, *k[0], *k[1], *k[2], o.kept.rstd_x.data_ptr(), o.kept.rstd_h.data_ptr(), post.data_ptr(),
        scale.data_ptr(), pre.data_ptr(), 0, 0, 0, 0, 0, 0, sums[0].data_ptr(), sums[1].data_ptr(), sums[2].data_ptr(), ws.data_ptr(), size,
        rows, cols, code, 1, 0, 0, 1.0), st) == 0
    torch.cuda.synchronize()
    assert bool((ws[size:] == 77).all())
    for got, w in zip(sums, (want.dpost_weight, want.dpre_weight, want.dscale)):
        assert torch.equal(got, w)


# ---------------------------------------------------------------- where memory lies

def accepted(status):
    """Without a GPU a call whose arguments are right ends where it asks for the device."""
    return status not in (0, 1, 2, 3, 4)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
def test_outputs_between_the_rows_of_others(mm):
    from test_block_ops import P, gated_call, gated_grad_call, norm_call, norm_grad_call
    half = 128                                  # bytes of a row of 64 bf16 columns; all strides are 128 columns
    assert accepted(gated_grad_call(mm, lddg=128, lddu=128, du=P[3] + half))
    assert accepted(gated_grad_call(mm, ldg=128, ldu=128, up=P[1] + half, lddg=128, lddu=128, du=P[3] + half))
    assert accepted(norm_call(mm, ldy=128, ldh=128, y=P[5] + half))
    assert accepted(norm_call(mm, ldx=128, ldy=128, y=P[0] + half))
    assert accepted(norm_grad_call(mm, lddx=128, lddr=128, dr=P[7] + half))
    assert accepted(norm_call(mm, ldy=128, ldh=128, h=P[4] + 5 * 256 + half))    # further down, and the rows above
    assert accepted(norm_call(mm, ldy=128, ldh=128, y=P[5] + 256 + half))
    for clash in (gated_grad_call(mm, lddg=128, lddu=128, du=P[3] + half - 2), gated_grad_call(mm, lddg=128, lddu=128, du=P[3] + 256 - 16),
                  gated_grad_call(mm, lddg=128, lddu=136, du=P[3] + half), gated_grad_call(mm, lddg=64, lddu=64, du=P[3] + half),
                  norm_call(mm, ldy=128, ldh=128, y=P[5] + 256), norm_call(mm, ldx=128, ldy=128, y=P[0] + half - 16),
                  gated_call(mm, g8=P[3], g8s=P[4], u8=P[3] + 64, u8s=P[5], ldg8=128, ldu8=128)):     # 8-bit ones are not looked into
        assert clash == 1


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
def test_strides_of_single_rows_are_not_looked_at(mm):
    from test_block_ops import P, gated_call, gated_grad_call, norm_call, norm_grad_call, transpose_call
    for ld in (0, 1, 7, -16):
        assert accepted(norm_call(mm, rows=1, ldx=ld, ldr=ld, gate=P[20], ldg=ld, ldy=ld, ldh=ld, q=P[8], qs=P[9], ldq=ld, x8=P[10], x8s=P[11],
                                  ldx8=ld, h8=P[12], h8s=P[13], ldh8=ld, g8=P[14], g8s=P[15], ldg8=ld))
        assert accepted(norm_grad_call(mm, rows=1, lddy=ld, dh=P[20], lddh=ld, ldx=ld, ldh=ld, lddx=ld, lddr=ld, xs=P[10], hs=P[11]))
        assert accepted(gated_call(mm, rows=1, ldg=ld, ldu=ld, ldy=ld, q=P[3], qs=P[4], ldq=ld, g8=P[5], g8s=P[6], ldg8=ld, u8=P[7], u8s=P[8],
                                   ldu8=ld))
        assert accepted(gated_grad_call(mm, rows=1, lddy=ld, ldg=ld, ldu=ld, lddg=ld, lddu=ld, gr=P[5], grs=P[6], ldgr=ld, ur=P[7], urs=P[8],
                                        ldur=ld))
        assert accepted(gated_grad_call(mm, cols=1, gc=P[5], gcs=P[6], ldgc=ld, uc=P[7], ucs=P[8], lduc=ld, yc=P[9], ycs=P[10], ldyc=ld))
        assert accepted(transpose_call(mm, rows=1, ldq=ld, cols=100)) and accepted(transpose_call(mm, cols=1, ldqt=ld))
    assert gated_call(mm, rows=1, q=P[3] + 8, qs=P[4], ldq=0) == 3


@gpu
@pytest.mark.parametrize("ld", [0, 7, 1 << 40])
def test_single_rows_of_any_stride(mm, ld):
    from newton_schulz_04_gb300 import blocks
    lib, st, cols = mm.load(), torch.cuda.current_stream().cuda_stream, 300
    g, u = (gen(i, 1, cols).bfloat16().cuda() for i in (70, 71))
    want = mm.gated_activation(g, u, fp8="e4m3", checkpoint="e4m3")
    q = [mm.Fp8Tensor.empty(1, cols) for _ in range(3)]
    outs = [v for t in q for v in (t.data.data_ptr(), t.scale.data_ptr(), ld)]
    assert lib.muon_gated_activation(blocks._GATED(g.data_ptr(), ld, u.data_ptr(), ld, 0, ld, *outs, 1, cols, 0, 0, 0, 0), st) == 0
    for t, w in zip(q, (want.q, want.kept.gate, want.kept.up)):
        assert torch.equal(t.data.view(torch.uint8), w.data.view(torch.uint8))
        assert torch.equal(t.scale.view(torch.uint8), w.scale.view(torch.uint8))
    back = mm.gated_activation_backward(u, want.kept, fp8="e5m2", y_fp8="e4m3", dense=False)
    rows8 = [mm.Fp8Tensor.empty(1, cols, "e5m2") for _ in range(2)]
    cols8 = [mm.Fp8Tensor.empty(cols, 1, f) for f in ("e5m2", "e5m2", "e4m3")]
    a = lambda t, ld: (t.data.data_ptr(), t.scale.data_ptr(), ld)  # noqa: E731
    k = [(t.data.data_ptr(), t.scale.data_ptr(), ld) for t in (want.kept.gate, want.kept.up)]
    assert lib.muon_gated_activation_backward(blocks._GATED_GRAD(
        u.data_ptr(), ld, *k[0], *k[1], 0, 0, 0, 0, *a(rows8[0], ld), *a(cols8[0], 16), *a(rows8[1], ld), *a(cols8[1], 16), *a(cols8[2], 16),
        1, cols, 0, 0, 0, 1, 0), st) == 0
    for t, w in zip(rows8 + cols8, (back.dgate_rows, back.dup_rows, back.dgate_cols, back.dup_cols, back.y_cols)):
        assert torch.equal(t.data.view(torch.uint8), w.data.view(torch.uint8))
        assert torch.equal(t.scale.view(torch.uint8), w.scale.view(torch.uint8))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,gap", [(64, 0), (264, 0), (264, 8), (123, 0), (123, 2), (1_000, 3)])
def test_outputs_in_the_halves_of_a_matrix(mm, dtype, cols, gap):
    """The C entry points with outputs, and inputs, side by side in one matrix: as apart, and nothing between them is written."""
    from newton_schulz_04_gb300 import blocks
    rows, lib, st = 150, mm.load(), torch.cuda.current_stream().cuda_stream
    code, size, ld = {torch.bfloat16: 0, torch.float32: 1}[dtype], dtype.itemsize, 2 * (cols + gap)
    x, r, g, post, pre, scale = dev(*norm_inputs(60, rows, cols, dtype, "element", True))
    dy = gen(61, rows, cols).to(dtype).cuda()

    def wide():
        t = torch.full((rows, ld), 5.0, dtype=dtype, device="cuda")
        return t, t[:, :cols], t[:, cols + gap:2 * cols + gap]

    def between(t):
        return torch.cat([t[:, cols:cols + gap], t[:, 2 * cols + gap:]], dim=1)

    inputs, gate, up = wide()
    gate.copy_(g), up.copy_(x)
    grads, dgate, dup = wide()
    want = mm.gated_activation_backward(dy, mm.GatedKept(g, x))
    for q in (None, "e4m3"):                    # the two kernels
        y8 = mm.Fp8Tensor.empty(cols, rows, "e4m3")
        args = [0, 0, 0] if q is None else [y8.data.data_ptr(), y8.scale.data_ptr(), y8._ld()]
        assert lib.muon_gated_activation_backward(blocks._GATED_GRAD(
            dy.data_ptr(), cols, gate.data_ptr(), 0, ld, up.data_ptr(), 0, ld, dgate.data_ptr(), ld, dup.data_ptr(), ld, *([0] * 12), *args,
            rows, cols, code, 0, 0, 0, 0), st) == 0
        assert torch.equal(dgate, want.dgate) and torch.equal(dup, want.dup) and bool((between(grads) == 5.0).all())
        grads.fill_(5.0)
    out, h, y = wide()
    n = mm.block_norm(x, r, post, pre, gate=g, scale=scale)
    stats = torch.empty(2, rows, device="cuda")
    assert lib.muon_block_norm(blocks._BLOCK_NORM(
        up.data_ptr(), ld, r.data_ptr(), cols, gate.data_ptr(), ld, post.data_ptr(), scale.data_ptr(), pre.data_ptr(), y.data_ptr(), ld,
        h.data_ptr(), ld, stats[0].data_ptr(), stats[1].data_ptr(), *([0] * 12), rows, cols, code, 1, 0, 0, 0, 1.0, 1e-6), st) == 0
    assert torch.equal(y, n.y) and torch.equal(h, n.h) and bool((between(out) == 5.0).all())
    back, dx, dr = wide()
    dg = torch.empty_like(g)
    d = mm.block_norm_backward(dy, n.kept, post, pre, scale=scale, dh=r)
    assert lib.muon_block_norm_backward(blocks._BLOCK_NORM_GRAD(
        dy.data_ptr(), cols, r.data_ptr(), cols, up.data_ptr(), 0, ld, h.data_ptr(), 0, ld, gate.data_ptr(), 0, ld,
        n.kept.rstd_x.data_ptr(), n.kept.rstd_h.data_ptr(), post.data_ptr(), scale.data_ptr(), pre.data_ptr(), dx.data_ptr(), ld,
        dr.data_ptr(), ld, dg.data_ptr(), cols, 0, 0, 0, 0, 0, rows, cols, code, 1, 0, 0, 1.0), st) == 0
    assert torch.equal(dx, d.dx) and torch.equal(dr, d.dresidual) and torch.equal(dg, d.dgate) and bool((between(back) == 5.0).all())


# ---------------------------------------------------------------- 8-bit outputs, scale by scale

def check8_by_blocks(q, x, err, fmt, what=""):
    """q stands for x within half a step and `err`.  Each block's scale is the smallest power of two under which a largest magnitude
    within the block's own error fits, 1 only of a block that may be zero; scales of no row or block are 1."""
    cols = x.shape[1]
    x, err = x.double(), err.double().expand(x.shape)
    s = q.scales().cpu().double()
    half, sub = block_ops.HALF8[fmt]
    close(q.dequantize(), x, half * x.abs() + (1 + half) * err + sub * s.repeat_interleave(128, dim=1)[:, :cols], what)
    pool = lambda t: torch.nn.functional.max_pool2d(t[None], (1, 128), ceil_mode=True)[0]  # noqa: E731
    low, high, top = pool((x.abs() - err).clamp(min=0)), pool(x.abs() + err), block_ops.ref8.TOP[fmt]
    right = (low <= top * s) & ((high > top * s / 2) | ((low == 0) & (s == 1)) | (s == 2.0 ** -127))
    assert bool(right.all()), f"{what}: scales of {int((~right).sum())} blocks"
    rows, blocks = s.shape
    kept = q.scale.view(torch.uint8).cpu().permute(1, 0, 2).reshape(q.scale.shape[1], -1)
    assert bool((kept[rows:] == 127).all()) and bool((kept[:, blocks:] == 127).all()), what


@pytest.fixture
def by_blocks(monkeypatch):
    monkeypatch.setattr(block_ops, "check8", check8_by_blocks)


def test_a_wrong_scale_is_seen():
    """The check itself, on the CPU: scales of 1 throughout, and one that is a power too large or too small."""
    class Q:
        def __init__(self, data, exps, fmt):
            self.data, self.scale, self.fmt, self.shape = data, block_ops.kept_scales(exps), fmt, data.shape

        def scales(self):
            s = 2.0 ** (self.scale.double() - 127)
            return s.permute(1, 0, 2).reshape(s.shape[1], -1)[:self.shape[0], :-(-self.shape[1] // 128)]

        def dequantize(self):
            return self.data * self.scales().repeat_interleave(128, dim=1)[:, :self.shape[1]]

    x = gen(80, 5, 300).double()
    x[3] = 0
    for fmt in ("e4m3", "e5m2"):
        data, exps = block_ops.ref8.quantize(x, fmt)
        check8_by_blocks(Q(data, exps, fmt), x, x.abs() * 1e-6, fmt)
        some = (x[:, :1] != 0).int()
        for bad in (torch.zeros_like(exps), exps + (torch.arange(3) == 1) * some, exps - (torch.arange(3) == 2) * some):
            wide = 2.0 ** bad.repeat_interleave(128, dim=1)[:, :300].double()
            with pytest.raises(AssertionError):
                check8_by_blocks(Q(block_ops.ref8.round8(x / wide, fmt).clamp(-block_ops.ref8.TOP[fmt], block_ops.ref8.TOP[fmt]), bad, fmt), x,
                                 x.abs() * 1e-6, fmt)
        q = Q(data, exps, fmt)
        q.scale[0, 5, 0] = 0
        with pytest.raises(AssertionError):
            check8_by_blocks(q, x, x.abs() * 1e-6, fmt)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (5, 127), (130, 256), (7, 1_000), (37, 4_100), (3, 16_385), (2, 40_000)])
def test_norm_outputs_scale_by_scale(mm, by_blocks, dtype, shape):
    for fp8, kept in (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e5m2", "e5m2")):
        block_ops.check_norm(mm, norm_inputs(81, *shape, dtype, "element", True), fp8=fp8, checkpoint=kept)
        block_ops.check_norm(mm, norm_inputs(82, *shape, dtype, "row", False), alpha=0.5, fp8=fp8, checkpoint=kept, y=False)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("shape", [(1, 1), (5, 127), (129, 130), (130, 256), (7, 1_000), (257, 640), (3, 16_385)])
def test_gated_outputs_scale_by_scale(mm, by_blocks, dtype, kind, shape):
    g, u = block_ops.gated_inputs(83, *shape, dtype)
    for fp8, kept in (("e4m3", "e4m3"), ("e5m2", "e5m2"), ("e5m2", None)):
        block_ops.check_gated(mm, g, u, kind, fp8=fp8, checkpoint=kept)
        block_ops.check_gated_grad(mm, 84, *shape, dtype, kind, kept=kept, fp8=fp8, y_fp8="e4m3")
    if dtype == torch.float32:                  # every 8-bit output to the bit, from the dense ones
        y = mm.gated_activation(*dev(g, u), activation=kind).y.cpu()
        dy = gen(85, *shape)
        d = mm.gated_activation_backward(dy.cuda(), mm.GatedKept(*dev(g, u)), activation=kind, fp8="e5m2", y_fp8="e4m3")
        for q, t in ((d.dgate_rows, d.dgate), (d.dup_rows, d.dup), (d.dgate_cols, d.dgate.t()), (d.dup_cols, d.dup.t())):
            check8_exact(q, t.cpu(), "e5m2")
        check8_exact(d.y_cols, y.t(), "e4m3")


# ---------------------------------------------------------------- offsets past 32 bits, in the rings too

@gpu
@pytest.mark.parametrize("cols", [4_096, 8_192])
@pytest.mark.parametrize("kept", [None, "e4m3"])
def test_ring_offsets_past_32_bits(mm, cols, kept):
    """More than 2^31 elements in rows that CTAs (4096 columns) and clusters (8192) hold: the last rows equal those alone."""
    rows = 2 ** 31 // cols + 5
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    w, end = torch.ones(cols, device="cuda"), x[-7:].contiguous()
    m = mm.block_norm(x, x, w, w, gate=x, fp8="e4m3", y=False, checkpoint=kept)
    n = mm.block_norm(end, end, w, w, gate=end, fp8="e4m3", y=False, checkpoint=kept)
    assert torch.equal(m.h[-7:], n.h) and torch.equal(m.q.scales()[-7:], n.q.scales()) and torch.equal(m.kept.rstd_h[-7:], n.kept.rstd_h)
    assert torch.equal(m.q.data[-7:].contiguous().view(torch.uint8), n.q.data.view(torch.uint8))
    g = mm.block_norm_backward(x, m.kept, w, w, dh=x, dweights=False)
    h = mm.block_norm_backward(end, n.kept, w, w, dh=end, dweights=False)
    assert torch.equal(g.dx[-7:], h.dx) and torch.equal(g.dgate[-7:], h.dgate) and torch.equal(g.dresidual[-7:], h.dresidual)
