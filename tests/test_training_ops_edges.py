"""The operators around the update where the other tests do not reach: many turns of the persistent kernels, in-place
calls, streams, the failure report, extreme ranges.

Comparisons here fail on a NaN that the oracle does not have (`close` asks that every difference is within the
tolerance, not that none is beyond it)."""
import ctypes
import glob
import math
import os
import re

import pytest
import torch

import oracle.training as ref

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
F24 = 2.0 ** -24
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "newton_schulz_04_gb300", "csrc")
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
    got, want = got.cpu().double(), want.cpu().double()
    assert got.shape == want.shape
    fine = (got - want).abs() <= tol
    assert bool(fine.all()), f"{int((~fine).sum())} of {fine.numel()} off, worst {float(((got - want).abs() - tol).max()):.3g}"


def test_close_rejects_nan():
    one = torch.ones(3)
    close(one, one, 0.0)
    for bad in (torch.tensor([1.0, math.nan, 1.0]), torch.tensor([1.0, 1.0, math.inf])):
        with pytest.raises(AssertionError):
            close(bad, one, 1.0)


# ---------------------------------------------------------------- split products

def test_arrivals_on_other_ctas_barriers_have_cluster_scope():
    """An arrive that names no scope orders nothing for a waiter in another CTA of the cluster, whatever fence stands
    before it: the sums of a split product are published so."""
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        for ins in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", open(path).read()):
            seen += 1
            assert ".cluster." in ins.replace("shared::cluster", ""), (os.path.basename(path), ins)
    assert seen >= 2


def _operand(mm, seed, rows, cols, fmt="e4m3"):
    x = gen(seed, rows, cols) * torch.exp(gen(seed + 1, rows, 1))
    q, _ = mm.fp8_quantize(x.cuda(), fmt)
    return q, ref.values(q.data.cpu(), q.scale.view(torch.uint8).cpu())


def _product_tol(a, b, want, dtype, k):
    # fp32 over k / 32 steps that may truncate (2^-23), 32 products inside a step, and up to 16 parts
    return U[dtype] * want.abs() + (k / 32 + 48) * 2.0 ** -23 * (a.abs() @ b.abs().t()) + TINY[dtype]


@gpu
@pytest.mark.parametrize("m,n,k", [(9, 256, 8192), (12, 1024, 4096), (33, 700, 1500), (64, 513, 6000), (17, 4096, 2049),
                                   (225, 257, 513), (500, 40, 2049)])
def test_products_have_no_nan_and_the_same_bits(mm, m, n, k):
    """Split and whole products, written over NaN, call after call: a part that comes too late would change a sum."""
    a, av = _operand(mm, 1, m, k)
    b, bv = _operand(mm, 3, n, k)
    want = ref.matmul(av, bv)
    first = mm.fp8_matmul(a, b, torch.float32)
    close(first, want, _product_tol(av, bv, want, torch.float32, k))
    out = torch.empty_like(first)
    for _ in range(50):
        out.fill_(math.nan)
        mm.fp8_matmul(a, b, out=out)
        assert torch.equal(out, first)
    assert mm.fp8_status() == 0


# ---------------------------------------------------------------- streams and devices

class FakeStream:
    def __init__(self, index, pointer):
        self.device, self.cuda_stream = torch.device("cuda", index), pointer


@pytest.fixture
def two_devices(monkeypatch):
    """torch.cuda as on a host with two GPUs, cuda:0 current; returns the list of (device, stream pointer) entered."""
    now = [0, 100]

    class Enter:
        def __init__(self, at, value):
            self.at, self.value = at, value

        def __enter__(self):
            self.old = list(now)
            if self.value is not None:
                now[self.at] = self.value
                if self.at == 0:
                    now[1] = 100 + self.value  # that device's own current stream

        def __exit__(self, *exc):
            now[:] = self.old

    class Stream(Enter):
        def __init__(self, stream):
            super().__init__(1, None if stream is None else stream.cuda_stream)
            self.stream = stream

        def __enter__(self):
            super().__enter__()
            if self.stream is not None:
                now[0] = self.stream.device.index  # as torch does: a stream brings its device along

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", lambda d: Enter(0, torch.device(d).index))
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(*now))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    return now


def test_fp8_status_is_the_asked_devices(mm, monkeypatch, two_devices):
    """After a product on another device than the current one its status is asked of that device."""
    from newton_schulz_04_gb300 import binding
    asked = []

    class Lib:
        @staticmethod
        def muon_fp8_status(stream):
            asked.append((two_devices[0], int(getattr(stream, "value", stream))))
            return 6 if two_devices[0] == 1 else 0

        @staticmethod
        def muon_debug_bounded_wait_fp8(cycles, stream):
            asked.append((two_devices[0], int(getattr(stream, "value", stream)), cycles))
            return 0

    monkeypatch.setattr(binding, "load", lambda: Lib)
    assert mm.fp8_status(FakeStream(1, 7)) == 6 and asked.pop() == (1, 7)
    assert mm.fp8_status(FakeStream(0, 8)) == 0 and asked.pop() == (0, 8)
    assert mm.fp8_status() == 0 and asked.pop() == (0, 100)
    assert mm.fp8_status(device=1) == 6 and asked.pop() == (1, 101)
    assert mm.fp8_status(device="cuda:1") == 6 and asked.pop() == (1, 101)
    assert mm.fp8_status(device="cuda") == 0 and asked.pop() == (0, 100)
    mm.debug_bounded_wait_fp8(5, FakeStream(1, 7))
    assert asked.pop() == (1, 7, 5)


def test_stream_of_another_device_is_refused(mm, two_devices):
    """A stream of another device would make that device current and launch there with this device's pointers."""
    from newton_schulz_04_gb300 import training
    ran = []
    here = torch.device("cuda", 0)
    training._on(FakeStream(0, 7), here, (), lambda *a: ran.append(a), 1)
    training._on(None, torch.device("cuda", 1), (), lambda *a: ran.append(a), 2)
    assert ran == [(1, 7), (2, 101)]
    with pytest.raises(ValueError, match="stream"):
        training._on(FakeStream(1, 7), here, (), lambda *a: ran.append(a))
    with pytest.raises(ValueError, match="stream"):
        mm.fp8_status(FakeStream(1, 7), device=0)
    assert len(ran) == 2


@gpu
def test_inputs_outlive_the_stream_that_reads_them(mm):
    """Inputs that the caller lets go while the call still waits on another stream keep their memory until it has run."""
    side = torch.cuda.Stream()
    size = 1 << 20

    def filled(value, *shape, dtype=torch.float32):
        return torch.full(shape, value, dtype=dtype, device="cuda")

    def taken_again(call, *shapes):
        """Addresses that `call`'s inputs had and a new tensor of the same size gets while the call waits."""
        inputs = [filled(2.0, *s) for s in shapes]
        at = {t.data_ptr() for t in inputs}
        call(*inputs)  # loads the code, which may wait for the device
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)  # some 25 ms
        result = call(*inputs)
        del inputs
        again = [torch.empty(*s, device="cuda") for s in shapes for _ in range(2)]
        hit = at & {t.data_ptr() for t in again}
        side.synchronize()
        return hit, result

    rows = (1024, size // 1024)
    hit, r = taken_again(lambda x, res: mm.rms_norm(x, None, res, stream=side), rows, rows)
    assert not hit and bool((r.h == 4).all())
    hit, r = taken_again(lambda x: mm.fp8_quantize(x, stream=side), rows)
    assert not hit and bool((r[0].dequantize() == 2).all())
    hit, _ = taken_again(lambda dy, h: mm.rms_norm_backward(dy, h, None, filled(1.0, 1024), stream=side), rows, rows)
    assert not hit
    hit, norm = taken_again(lambda g: mm.grad_norm([g], stream=side), (size,))
    assert not hit and float(norm) == 2.0 * 1024
    # the product's operands and addend
    x = filled(2.0, *rows)
    a, b = mm.fp8_quantize(x)[0], mm.fp8_quantize(x)[0]
    add = filled(1.0, 1024, 1024)
    at = {t.data_ptr() for t in (a.data, b.data, add)}
    mm.fp8_matmul(a, b, torch.float32, add=add)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    c = mm.fp8_matmul(a, b, torch.float32, add=add, stream=side)
    del a, b, add
    again = [torch.empty(*rows, dtype=d, device="cuda") for d in (torch.uint8, torch.uint8, torch.float32, torch.float32)]
    assert not at & {t.data_ptr() for t in again}
    side.synchronize()
    assert bool((c == 4097).all())


@gpu
def test_fp8_status_loses_no_report(mm):
    """Reports made on one stream while another one's status is asked for again and again are each given once."""
    import threading
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    assert mm.fp8_status() == 0
    given, calls, stop = [], [0], threading.Event()

    def ask():
        while not stop.is_set():
            status = mm.fp8_status(other)
            if status != 0:
                given.append(status)
            calls[0] += 1

    thread = threading.Thread(target=ask)
    thread.start()
    try:
        for i in range(400):
            before = len(given)
            mm.debug_bounded_wait_fp8(1 + 97 * i, side)
            side.synchronize()
            n = calls[0]
            while calls[0] < n + 2 and thread.is_alive():  # a call begun after the report has returned
                pass
            assert given[before:] == [6], i
    finally:
        stop.set()
        thread.join()
    assert mm.fp8_status() == 0


# ---------------------------------------------------------------- clipping

def _clip(mm, grads, outs, numel, ws=1 << 40, dtype=1):
    """muon_clip_grads on addresses that are never read: of what is not refused, only the refusal is asked for."""
    count = len(grads)
    P, N, D = ctypes.c_void_p * count, ctypes.c_int64 * count, ctypes.c_int32 * count
    size = mm.load().muon_clip_workspace_bytes(count)
    return mm.load().muon_clip_grads(P(*grads), None if outs is None else P(*outs), N(*numel), D(*[dtype] * count), count,
                                     1.0, 1e-6, 1 << 41, ws, size, None)


@pytest.mark.parametrize("count", [2, 3, 65, 200])
def test_clip_refuses_outputs_that_share_memory(mm, count):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for hosts where nothing can be launched")
    step = 4096
    a = [(1 << 30) + step * ((7 * i) % count if count % 7 else i) for i in range(count)]  # in no order
    b = [p + (1 << 32) for p in a]
    n = [step // 4] * count
    fine = _clip(mm, a, a, n)
    assert fine not in (0, 1)                      # what the missing device says
    assert _clip(mm, a, b, n) == fine and _clip(mm, a, b, [0, *n[1:]]) == fine
    last = count - 1
    twice = [*a[:last], a[0]]
    assert _clip(mm, twice, twice, n) == 1         # one tensor listed twice, in place
    assert "overlaps another" in mm.load().muon_last_error().decode()
    assert _clip(mm, twice, None, n) == fine       # the norm alone may count it twice
    assert _clip(mm, twice, b, n) == fine          # and so may outputs of their own
    assert _clip(mm, a, [*b[:last], b[0]], n) == 1
    assert _clip(mm, a, [*b[:last], b[0] + step - 4], n) == 1
    assert _clip(mm, a, a[1:] + a[:1], n) == 1     # outputs in another order than the gradients
    assert _clip(mm, a, [*b[:last], a[0] + step - 4], n) == 1
    assert _clip(mm, twice, twice, [*n[:last], 0]) == fine
    assert _clip(mm, a, None, n, ws=a[last] + 8) == 1 and _clip(mm, a, b, n, ws=b[0] + 8) == 1


@gpu
def test_clip_refuses_a_tensor_listed_twice(mm):
    g, h = torch.ones(5000, device="cuda"), torch.ones(70, device="cuda")
    with pytest.raises(mm.MuonError, match="overlaps"):
        mm.clip_grads([g, h, g], 0.5)
    with pytest.raises(mm.MuonError, match="overlaps"):
        mm.clip_grads([g[:100], g[50:200]], 0.5)
    with pytest.raises(mm.MuonError, match="overlaps"):
        mm.clip_grads([g, h], 0.5, out=[g, g[:70]])
    assert bool((g == 1).all()) and float(mm.grad_norm([g, g])) == 100.0
    out = [torch.zeros_like(g), torch.zeros_like(g)]
    mm.clip_grads([g, g], 50.0, out=out)
    assert torch.equal(*out) and abs(float(out[0][0]) - 0.5) < 1e-6
    mm.clip_grads([g[2500:], g[:2500]], 10.0)      # neighbours, in any order
    assert abs(float(mm.grad_norm([g])) - 10.0) < 1e-5


def _kernels(text):
    """(name, body) of each kernel in a source."""
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\([^{;]*\) \{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at - 1]


def test_every_thread_waits_for_the_kernels_before():
    """A kernel that may start before the one ahead of it has ended waits for it in every thread, not in a branch or on
    some threads only: nothing else makes visible what earlier kernels wrote."""
    seen = []
    for name in ("clip.cu", "rms_norm.cu", "fp8_quant.cu", "fp8_gemm.cu", "fp8_few.cu"):
        for kernel, body in _kernels(open(os.path.join(CSRC, name)).read()):
            if kernel == "fp8_take_status_kernel":  # launched in stream order
                continue
            before = body[:body.index("pdl_wait();")]
            assert before.count("{") == before.count("}"), kernel
            seen.append(kernel)
    assert len(seen) >= 9 and "clip_scale_kernel" in seen


@gpu
def test_clip_right_after_the_kernels_that_write_its_gradients(mm):
    """Gradients rewritten by this package's kernels and clipped at once, again and again at the same addresses."""
    a = [mm.fp8_quantize(gen(i, 48, 256).cuda(), "e5m2")[0] for i in range(4)]
    b = [mm.fp8_quantize(gen(9 + i, 80, 256).cuda())[0] for i in range(4)]
    dy, h = gen(20, 300, 512).cuda(), gen(21, 300, 512).cuda()
    rstd = torch.ones(300, device="cuda")
    g = torch.empty(48, 80, device="cuda")
    want = []
    for i in range(4):
        dw = mm.rms_norm_backward(dy, h, None, rstd * (i + 1))[1]
        torch.cuda.synchronize()
        t = [mm.fp8_matmul(a[i], b[i], torch.float32), dw]
        torch.cuda.synchronize()
        n = mm.clip_grads(t, 1.0)
        torch.cuda.synchronize()
        want.append([n, *t])
    scaled = [rstd * (i + 1) for i in range(4)]
    for turn in range(200):
        i = turn % 4
        mm.fp8_matmul(a[i], b[i], out=g)
        dw = mm.rms_norm_backward(dy, h, None, scaled[i])[1]
        n = mm.clip_grads([g, dw], 1.0)
        got = [n.clone(), g.clone(), dw]
        assert all(torch.equal(x, y) for x, y in zip(got, want[i])), turn


# ---------------------------------------------------------------- RMS norm

@gpu
@pytest.mark.parametrize("cols", [256, 1000, 1001, 4096, 16384, 20001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rms_norm_range(mm, dtype, cols):
    """As stated: right while a row's sum of squares is below fp32's largest value, rho = 0 and y = 0 beyond."""
    large, small = 2.0 ** 63 / math.sqrt(cols), 1e-15
    x = gen(1, 4, cols).clamp(-3, 3)
    x = (x / 3 * torch.tensor([[large], [small], [1.0], [large]])).to(dtype)
    x[3] = 2.0 ** 66
    r = mm.rms_norm(x.cuda(), None, eps=0.0, fp8="e4m3")
    want, _, rstd = ref.rms_norm(x[:3], None, eps=0.0)
    rel = (137 / 2 + 4) * F24
    close(r.rstd[:3], rstd.flatten(), rel * rstd.flatten())
    close(r.y[:3], want, (U[dtype] + rel + 3 * F24) * want.abs() + TINY[dtype])
    assert float(r.rstd[3]) == 0 and float(r.y[3].abs().sum()) == 0
    assert float(r.q.dequantize()[3].abs().sum()) == 0 and bool(r.q.dequantize().isfinite().all())


RING = {  # columns that a ring takes, in 16-bit types (half of them in fp32): (rows ahead, rows per CTA, CTAs per SM)
    248: ((8, 4, 6), (4, 4, 6)), 504: ((4, 2, 8), (4, 4, 3)), 1000: ((4, 2, 4), (4, 2, 3)), 2040: ((4, 1, 3), (5, 1, 3)),
    4088: ((5, 1, 2), (4, 1, 2)), 8184: ((4, 1, 1), (4, 1, 1)), 16376: ((3, 1, 1), (2, 1, 1))}


def _many_rows(cols, dtype, which):
    """(rows, cols): more than enough for every CTA to refill its whole ring, and an odd rest; rows of one turn."""
    ahead, per, ctas = RING[cols][which]
    turn = per * ctas * torch.cuda.get_device_properties(0).multi_processor_count
    return (ahead + 2) * turn + 3, cols if dtype != torch.float32 else cols // 2, turn


def _raw(t):
    return t.contiguous().view(torch.uint8)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", list(RING))
def test_rms_norm_rings_many_turns(mm, cols, dtype):
    """The persistent kernel over many turns: near the oracle, and the bits that the same rows have in one turn."""
    rows, cols, turn = _many_rows(cols, dtype, 0)
    g = torch.Generator("cuda").manual_seed(5)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * torch.exp(torch.randn(rows, 1, device="cuda", generator=g)))
    x, res = x.to(dtype), torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    w = 1 + 0.1 * torch.randn(cols, device="cuda", generator=g)
    r = mm.rms_norm(x, w, res, fp8="e4m3")
    y, h, rstd = ref.rms_norm(x, w, res)
    rel = (137 / 2 + 4) * F24
    close(r.rstd, rstd.flatten(), rel * rstd.flatten().cpu())
    close(r.h, h, (U[dtype] * h.abs() + TINY[dtype]).cpu())
    tol = (U[dtype] + rel + 3 * F24) * y.abs() + TINY[dtype] + F24 * h.abs() * rstd[..., None] * w.double().abs()
    close(r.y, y, tol.cpu())
    data, scale, scales = _raw(r.q.data), r.q.scale.view(torch.uint8), r.q.scales()
    assert int((scale == 255).sum()) == 0
    for i in range(0, rows, turn):
        part = slice(i, min(rows, i + turn))
        s = mm.rms_norm(x[part], w, res[part], fp8="e4m3")
        assert torch.equal(s.y, r.y[part]) and torch.equal(s.h, r.h[part]) and torch.equal(s.rstd, r.rstd[part]), i
        assert torch.equal(_raw(s.q.data), data[part]) and torch.equal(s.q.scales(), scales[part]), i


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", list(RING))
def test_rms_norm_gradient_rings_many_turns(mm, cols, dtype):
    rows, cols, turn = _many_rows(cols, dtype, 1)
    g = torch.Generator("cuda").manual_seed(6)
    dy, h, res = (torch.randn(rows, cols, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = 1 + 0.2 * torch.randn(cols, device="cuda", generator=g)
    rstd = ref.rms_norm(h)[2].float()
    dx, dw = mm.rms_norm_backward(dy, h, w, rstd, res)
    want, want_w = ref.rms_norm_backward(dy, h, w, rstd, res)
    r, gw = rstd.double()[:, None], dy.double() * w.double()
    mean = (gw * h.double()).abs().mean(dim=1, keepdim=True)
    tol = (140 * F24) * h.double().abs() * r ** 3 * mean + 6 * F24 * ((r * gw).abs() + want.abs())
    close(dx, want, (tol + U[dtype] * want.abs() + TINY[dtype]).cpu())
    # a column's chain: 8 turns, 4 rows of a CTA, a 32nd of up to 912 CTAs, five joins; two products
    close(dw, want_w, (8 + 4 + 29 + 5 + 2) * F24 * (dy.double() * h.double() * r).abs().sum(dim=0).cpu())
    for i in range(0, rows, turn):
        part = slice(i, min(rows, i + turn))
        s = mm.rms_norm_backward(dy[part], h[part], w, rstd[part], res[part], dweight=False)[0]
        assert torch.equal(s, dx[part]), i


def _norm_in_place(mm, x, res, w, y, h, ld):
    """muon_rms_norm on [rows, cols] views of row stride ld; y, h or res may be None."""
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rows, cols = x.shape
    dt = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}[x.dtype]
    rstd = torch.empty(rows, device="cuda")
    assert mm.load().muon_rms_norm(at(x), ld, at(res), ld, at(w), 1, rows, cols, 1e-6, at(y), ld, at(h), ld, at(rstd), None, 0,
                                   None, 0, dt, torch.cuda.current_stream().cuda_stream) == 0
    return rstd


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(3, 5), (40000, 64), (5000, 1000), (700, 1001), (2500, 4096), (700, 8192), (500, 16376),
                                       (300, 9001), (40, 33000)])
def test_norms_in_place(mm, dtype, rows, cols):
    """y or h over x or the residual, dx over dy, the residual's gradient or h: the bits of separate outputs."""
    ld = cols + 24
    big = lambda seed: torch.randn(rows, ld, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)  # noqa: E731
    x, res, w = big(1), big(2), 1 + 0.1 * gen(3, cols).cuda()
    v = lambda t: t[:, :cols]  # noqa: E731
    y, h = torch.empty_like(x), torch.empty_like(x)
    rstd = _norm_in_place(mm, v(x), v(res), w, v(y), v(h), ld)
    assert bool(v(y).isfinite().all())
    for py, ph in (("x", None), ("res", None), (None, "x"), (None, "res"), ("x", "res"), ("res", "x")):
        t = {"x": x.clone(), "res": res.clone(), None: torch.empty_like(x)}
        out_y, out_h = t[py], (torch.empty_like(x) if ph is None else t[ph])
        got = _norm_in_place(mm, v(t["x"]), v(t["res"]), w, v(out_y), v(out_h), ld)
        assert torch.equal(got, rstd) and torch.equal(v(out_y), v(y)) and torch.equal(v(out_h), v(h)), (py, ph)
        for name, old in (("x", x), ("res", res)):  # between the rows, and what is only read
            assert torch.equal(t[name][:, cols:], old[:, cols:])
            assert name in (py, ph) or torch.equal(t[name], old)
    alone = x.clone()
    _norm_in_place(mm, v(alone), None, w, v(alone), None, ld)
    assert torch.equal(v(alone), mm.rms_norm(v(x), w).y)

    dy, lib = big(7), mm.load()
    dt = 0 if dtype == torch.bfloat16 else 1
    want, want_w = mm.rms_norm_backward(v(dy), v(h), w, rstd, v(res))
    ws = torch.empty(lib.muon_rms_norm_backward_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    for over in ("dy", "h", "res"):
        t = {"dy": dy.clone(), "h": h.clone(), "res": res.clone()}
        dw = torch.empty(cols, device="cuda")
        assert lib.muon_rms_norm_backward(t["dy"].data_ptr(), ld, t["h"].data_ptr(), ld, w.data_ptr(), 1, rstd.data_ptr(),
                                          t["res"].data_ptr(), ld, rows, cols, t[over].data_ptr(), ld, dw.data_ptr(),
                                          ws.data_ptr(), ws.numel(), dt, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(v(t[over]), want) and torch.equal(dw, want_w), over


def test_padding_of_an_8_bit_output_overlaps_too(mm):
    """Rows of 8-bit outputs are written up to the next multiple of 16 bytes: nothing else may lie there."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for hosts where nothing can be launched")
    lib = mm.load()
    q, scale, far = 1 << 30, 1 << 31, 1 << 32

    def norm(x, cols=100, rows=4, ldq=112):
        return lib.muon_rms_norm(x, cols, None, 0, None, 0, rows, cols, 1e-6, None, 0, None, 0, None, q, ldq, scale, 0, 0, None)

    def quantize(x, qt=None):
        return lib.muon_fp8_quantize(x, 100, 4, 100, 0, 0, 0, q, 112, scale, qt, 16, None if qt is None else far, None)

    end = q + 3 * 112 + 112
    assert norm(end) == quantize(end) == quantize(far << 1, end) not in (0, 1)
    assert norm(end - 2) == 1 and quantize(end - 2) == 1           # between the last column and the row's padded end
    assert quantize(far << 1, end - 16) == 1 and quantize(far << 1, end - 112) == 1


# ---------------------------------------------------------------- what the looser tests let pass

@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("size", [1, 9, 8193, 100_003, 2_000_001])
def test_clip_misses_no_element(mm, dtype, size):
    """One element alone makes the norm: at both ends, around every boundary of 32 KB, in the rest."""
    per = 32768 // (4 if dtype == torch.float32 else 2)
    at = sorted({p for c in range(0, size + per, per) for p in (c - 1, c, c + 1, c + 255, c + 256) if 0 <= p < size}
                | {0, size // 2, size - 1})
    for offset in (0, 1):  # aligned to 16 bytes, and not
        g = torch.zeros(size + offset, dtype=dtype, device="cuda")[offset:]
        other = torch.zeros(5, device="cuda")
        norms = []
        for p in at:
            g[p] = 3.0
            norms.append(mm.grad_norm([other, g, other]))
            g[p] = 0.0
        assert torch.stack(norms).tolist() == [3.0] * len(at)
    for p in (0, size // 2, size - 1):  # and all of it is scaled
        g = torch.full((size,), 2.0 ** -6, dtype=dtype, device="cuda")
        g[p] = 2.0 ** 6
        norm = mm.clip_grads([g], 0.25, eps=0.0)
        want = torch.full((size,), 2.0 ** -6, dtype=dtype, device="cuda")
        want[p] = 2.0 ** 6
        assert torch.equal(g, (want.float() * (0.25 / norm)).to(dtype))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("parts", [1, 7])
def test_clip_runs_of_many_chunks(mm, dtype, parts):
    """Six or more whole chunks for each CTA: the norm to its own chain, and every element."""
    width = 4 if dtype == torch.float32 else 2
    ctas = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    size = (7 * ctas * 32768 // width) // parts + 11
    g = [torch.randn(size + 3 * i, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(dtype) for i in range(parts)]
    old = [t.clone() for t in g]
    want = math.sqrt(math.fsum(float(t.double().square().sum()) for t in g))
    norm = mm.clip_grads(g, 1.0)
    # 16 elements of a chunk to each of a thread's four sums (8 in fp32, but 16 holds), 9 chunks, and the joins
    assert abs(float(norm) - want) <= (16 * 9 + 2 + 5 + 4) * F24 * want
    factor = 1.0 / (norm + 1e-6)
    for a, b in zip(g, old):
        assert torch.equal(a, (b.float() * factor).to(dtype))


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("m,n,k", [(1, 300, 129), (8, 33, 2500), (9, 33, 2500), (33, 100, 31), (64, 513, 1152), (225, 257, 513),
                                   (500, 40, 2049), (1000, 1500, 700)])
def test_products_without_nan(mm, out, fa, fb, m, n, k):
    a, av = _operand(mm, 1, m, k, fa)
    b, bv = _operand(mm, 3, n, k, fb)
    want = ref.matmul(av, bv)
    tol = _product_tol(av, bv, want, out, k)
    buf = torch.full((m, n), math.nan, dtype=out, device="cuda")
    close(mm.fp8_matmul(a, b, out=buf), want, tol)
    add = (gen(9, m, n) * float(want.abs().mean())).to(out)
    want = want + add.double()
    close(mm.fp8_matmul(a, b, add=add.cuda(), out=buf.fill_(math.nan)), want, tol + (U[out] + F24) * (want.abs() + add.double().abs()))


def test_empty_refuses_an_unknown_format(mm):
    with pytest.raises(ValueError, match="format"):
        mm.Fp8Tensor.empty(2, 128, "e3m4", device="cpu")
    assert mm.Fp8Tensor.empty(2, 100, "e5m2", device="cpu").data.stride(0) == 112


@gpu
def test_unknown_formats_are_refused(mm):
    x = torch.ones(2, 128, device="cuda")
    for call in (lambda: mm.fp8_quantize(x, fmt="e3m4"), lambda: mm.rms_norm(x, None, fp8="e3m4")):
        with pytest.raises(ValueError, match="format"):
            call()


@gpu
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("m,k", [(8, 131072), (40, 131072), (8, 1 << 20), (40, 1 << 20), (300, 1 << 20)])
def test_products_over_a_long_axis(mm, m, k, positive):
    """The stated bound of the sums over k, against 64 bits."""
    n = 64
    g = torch.Generator("cuda").manual_seed(1)
    x, w = torch.randn(m, k, device="cuda", generator=g), torch.randn(n, k, device="cuda", generator=g)
    if positive:
        x, w = x.abs(), w.abs()
    a, b = mm.fp8_quantize(x)[0], mm.fp8_quantize(w)[0]
    av, bv = a.dequantize(), b.dequantize()
    want, most = (torch.zeros(m, n, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, k, 65536):
        p, q = av[:, i:i + 65536].double(), bv[:, i:i + 65536].double()
        want += p @ q.t()
        most += p.abs() @ q.abs().t()
    close(mm.fp8_matmul(a, b, torch.float32), want, ((k * 2.0 ** -28 + 48 * 2.0 ** -23) * most + 2.0 ** -24 * want.abs()).cpu())
