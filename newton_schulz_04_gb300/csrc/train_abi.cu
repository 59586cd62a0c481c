// train_abi.cu -- C ABI of the operators around the update: gradient clipping, the RMS norm
// and its gradient, 8-bit quantisation and the 8-bit product.  Every argument is
// checked before the first launch; nothing throws across the ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "common.cuh"
#include "kernels.h"
#include "train_ops.h"

namespace muon {

static bool float_dt(int dt) { return dt == MUON_BF16 || dt == MUON_FP32 || dt == MUON_FP16; }
static bool fp8_fmt(int f) { return f == MUON_E4M3 || f == MUON_E5M2; }
static bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }
static bool aligned16(const void* p, long long ld, int size) { return !misaligned(p, 16) && ld * size % 16 == 0; }

// Bytes spanned by a matrix of `rows` rows of `cols` elements, `ld` apart.
static long long span(long long rows, long long cols, long long ld, int size) {
  return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * size : 0;
}
// And by an 8-bit one, whose rows are written up to the next multiple of 16 bytes.
static long long span8(long long rows, long long cols, long long ld) { return span(rows, (cols + 15) / 16 * 16, ld, 1); }
static bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// The device is an sm_103 GPU: its SM count (asked for once per device), or 0 with *st set.
static int gpu(muon_status* st) {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
    const int sms = known[dev].load(std::memory_order_relaxed);
    if (sms) {
      *st = MUON_OK;
      return sms;
    }
  }
  int major = 0, minor = 0;
  const int sms = device_sms(&major, &minor, st);
  if (*st != MUON_OK) return 0;
  if (major != 10 || minor != 3) {
    *st = fail(MUON_ERR_UNSUPPORTED, "this library is built for sm_103a (GB300); device is sm_%d%d", major, minor);
    return 0;
  }
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}
static muon_status launched(cudaError_t e, const char* what, const char* why = nullptr) {
  if (e == cudaSuccess) return MUON_OK;
  return fail(MUON_ERR_CUDA, "%s failed: %s%s%s", what, cudaGetErrorString(e), why ? ": " : "", why ? why : "");
}

}  // namespace muon

using namespace muon;

extern "C" {

// ------------------------------------------------------------------ clipping
// Clipped in two places at once a tensor would be scaled twice, or by one CTA while another reads it: no output may
// share memory with another tensor's output or gradient.  (out[i] is grads[i] or disjoint from it.)
struct ClipSpan {
  uintptr_t begin, end;
};
struct ClipSpans {
  ClipSpan* s;
  int n = 0;
  bool sorted = true;
  void put(const void* p, long long bytes) {
    const uintptr_t begin = reinterpret_cast<uintptr_t>(p);
    if (n > 0 && begin < s[n - 1].begin) sorted = false;
    s[n++] = {begin, begin + static_cast<uintptr_t>(bytes)};
  }
  void sort() {
    if (!sorted) std::sort(s, s + n, [](const ClipSpan& a, const ClipSpan& b) { return a.begin < b.begin; });
  }
};
static muon_status clip_disjoint(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dtypes,
                                 int count) {
  ClipSpan few[2 * kClipSmall];
  std::unique_ptr<ClipSpan[]> many;
  if (count > kClipSmall) {
    many.reset(new (std::nothrow) ClipSpan[2 * static_cast<size_t>(count)]);
    if (!many) return fail(MUON_ERR_ARG, "no memory to look over %d tensors", count);
  }
  ClipSpans written{many ? many.get() : few}, read{written.s + count};
  for (int i = 0; i < count; ++i) {
    const long long bytes = numel[i] * dtype_bytes(dtypes[i]);
    if (bytes == 0) continue;
    written.put(out[i], bytes);
    if (out[i] != grads[i]) read.put(grads[i], bytes);
  }
  written.sort();
  read.sort();
  uintptr_t last = 0, seen = 0;  // ends of the outputs so far, and of the gradients that begin before this output's end
  for (int i = 0, r = 0; i < written.n; ++i) {
    for (; r < read.n && read.s[r].begin < written.s[i].end; ++r) seen = std::max(seen, read.s[r].end);
    if (written.s[i].begin < last || written.s[i].begin < seen)
      return fail(MUON_ERR_ARG, "an output overlaps another tensor's output or gradient");
    last = written.s[i].end;
  }
  return MUON_OK;
}

size_t muon_clip_workspace_bytes(int count) {
  // one 64-bit partial sum for each CTA of each launch
  const size_t launches = count <= kClipSmall ? 1 : (static_cast<size_t>(count) + kClipLarge - 1) / kClipLarge;
  return launches * MUON_CLIP_CTAS * sizeof(double);
}

muon_status muon_clip_grads(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dtypes,
                            int count, float max_norm, float eps, float* norm, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (count < 0) return fail(MUON_ERR_ARG, "count=%d < 0", count);
  if (count > 0 && (!grads || !numel || !dtypes)) return fail(MUON_ERR_ARG, "NULL array");
  if (!norm && !out) return fail(MUON_ERR_ARG, "neither norm nor out is given");
  if (out && !(max_norm >= 0.f)) return fail(MUON_ERR_ARG, "need max_norm >= 0");
  if (!(std::isfinite(eps) && eps >= 0.f)) return fail(MUON_ERR_ARG, "need a finite eps >= 0");
  if (misaligned(norm, 4)) return fail(MUON_ERR_ALIGN, "norm is not 4-byte aligned");
  if (!ws) return fail(MUON_ERR_ARG, "workspace is NULL");
  if (misaligned(ws, 8)) return fail(MUON_ERR_ALIGN, "workspace is not 8-byte aligned");
  if (ws_bytes < muon_clip_workspace_bytes(count))
    return fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, muon_clip_workspace_bytes(count));
  long long chunks = 0;
  for (int i = 0; i < count; ++i) {
    if (!float_dt(dtypes[i])) return fail(MUON_ERR_ARG, "tensor %d has the bad dtype %d", i, dtypes[i]);
    if (numel[i] < 0) return fail(MUON_ERR_SHAPE, "numel[%d] < 0", i);
    if (numel[i] > 0 && (!grads[i] || (out && !out[i]))) return fail(MUON_ERR_ARG, "tensor %d has a NULL pointer", i);
    const int size = dtype_bytes(dtypes[i]);
    if (misaligned(grads[i], size) || (out && misaligned(out[i], size)))
      return fail(MUON_ERR_ALIGN, "tensor %d is not aligned to its element size", i);
    if (out && out[i] != grads[i] && overlap(out[i], numel[i] * size, grads[i], numel[i] * size))
      return fail(MUON_ERR_ARG, "tensor %d: out overlaps the gradient", i);
    if (overlap(grads[i], numel[i] * size, ws, static_cast<long long>(ws_bytes)) ||
        (out && overlap(out[i], numel[i] * size, ws, static_cast<long long>(ws_bytes))))
      return fail(MUON_ERR_ARG, "tensor %d overlaps the workspace", i);
    chunks += (numel[i] * size + kClipChunkBytes - 1) / kClipChunkBytes;
    if (chunks > 0x7fffffffLL) return fail(MUON_ERR_SHAPE, "too many elements");
  }
  if (out) {
    const muon_status apart = clip_disjoint(grads, out, numel, dtypes, count);
    if (apart != MUON_OK) return apart;
  }
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  const int grid = std::min(MUON_CLIP_CTAS, kClipCtasPerSm * sms);
  return launched(launch_clip(grads, out, numel, dtypes, count, max_norm, eps, static_cast<double*>(ws), grid, norm,
                              static_cast<cudaStream_t>(stream)),
                  "launch_clip");
}

// ------------------------------------------------------------------ RMS norm
// One matrix argument: NULL is allowed when `optional`; sets *vec to 0 where 16-byte accesses are not possible.
static muon_status check_rows(const char* name, const void* p, bool optional, long long rows, long long cols, long long ld,
                              int size, int* vec) {
  if (!p) return optional ? MUON_OK : fail(MUON_ERR_ARG, "%s is NULL", name);
  if (misaligned(p, size)) return fail(MUON_ERR_ALIGN, "%s is not aligned to its element size", name);
  if (rows > 1 && ld < cols) return fail(MUON_ERR_SHAPE, "%s: row stride %lld < %lld columns", name, ld, cols);
  if (misaligned(p, 16) || (rows > 1 && ld * size % 16)) *vec = 0;
  return MUON_OK;
}
static muon_status check_fp8_out(const char* name, const void* q, const void* scale, long long rows, long long cols,
                                 long long ld) {
  if (!q && !scale) return MUON_OK;
  if (!q || !scale) return fail(MUON_ERR_ARG, "%s: data and scale go together", name);
  if (misaligned(q, 16) || misaligned(scale, 16) || ld % 16)
    return fail(MUON_ERR_ALIGN, "%s: data and scale must be 16-byte aligned, the row stride a multiple of 16", name);
  if (ld < (cols + 15) / 16 * 16 && rows > 0)
    return fail(MUON_ERR_SHAPE, "%s: row stride %lld does not hold %lld columns padded to 16", name, ld, cols);
  return MUON_OK;
}
static muon_status check_norm_shape(long long rows, long long cols, int dt, const void* weight, int weight_dt) {
  if (rows < 0 || rows > MUON_MAX_ROWS) return fail(MUON_ERR_SHAPE, "rows=%lld out of [0, %lld]", rows, MUON_MAX_ROWS);
  if (cols < 1 || cols > MUON_MAX_DIM) return fail(MUON_ERR_SHAPE, "cols=%lld out of [1, %d]", cols, MUON_MAX_DIM);
  if (!float_dt(dt)) return fail(MUON_ERR_ARG, "bad dtype %d", dt);
  if (weight && !float_dt(weight_dt)) return fail(MUON_ERR_ARG, "bad weight dtype %d", weight_dt);
  if (weight && misaligned(weight, dtype_bytes(weight_dt)))
    return fail(MUON_ERR_ALIGN, "weight is not aligned to its element size");
  return MUON_OK;
}
// Two matrices may be the same one (same address and stride) but not overlap otherwise.
static bool clash(const void* a, long long lda, const void* b, long long ldb, long long rows, long long cols, int size) {
  if (a == b && (lda == ldb || rows <= 1)) return false;
  return overlap(a, span(rows, cols, lda, size), b, span(rows, cols, ldb, size));
}

#define TRY(expr)                         \
  do {                                    \
    const muon_status st_ = (expr);       \
    if (st_ != MUON_OK) return st_;       \
  } while (0)

muon_status muon_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                          muon_dtype weight_dt, int64_t rows, int64_t cols, float eps, void* y, int64_t ldy, void* h,
                          int64_t ldh, float* rstd, void* q, int64_t ldq, void* q_scale, muon_fp8 fmt, muon_dtype dt,
                          void* stream) {
  clear_error();
  TRY(check_norm_shape(rows, cols, dt, weight, weight_dt));
  if (!(std::isfinite(eps) && eps >= 0.f)) return fail(MUON_ERR_ARG, "need a finite eps >= 0");
  if (q && !fp8_fmt(fmt)) return fail(MUON_ERR_ARG, "bad 8-bit format %d", fmt);
  if (rows == 0) return MUON_OK;
  const int size = dtype_bytes(dt);
  RmsNormArgs a = {};
  a.vec = weight && misaligned(weight, 16) ? 0 : 1;
  TRY(check_rows("x", x, false, rows, cols, ldx, size, &a.vec));
  TRY(check_rows("residual", residual, true, rows, cols, ldr, size, &a.vec));
  TRY(check_rows("y", y, true, rows, cols, ldy, size, &a.vec));
  TRY(check_rows("h", h, true, rows, cols, ldh, size, &a.vec));
  TRY(check_fp8_out("q", q, q_scale, rows, cols, ldq));
  if (misaligned(rstd, 4)) return fail(MUON_ERR_ALIGN, "rstd is not 4-byte aligned");
  if (!y && !h && !rstd && !q) return fail(MUON_ERR_ARG, "no output is given");
  const void* outs[2] = {y, h};
  const long long ldo[2] = {ldy, ldh};
  for (int i = 0; i < 2; ++i)
    if (clash(outs[i], ldo[i], x, ldx, rows, cols, size) || clash(outs[i], ldo[i], residual, ldr, rows, cols, size))
      return fail(MUON_ERR_ARG, "an output partly overlaps an input");
  if (y && h && overlap(y, span(rows, cols, ldy, size), h, span(rows, cols, ldh, size)))
    return fail(MUON_ERR_ARG, "y and h overlap");
  const long long nq = span8(rows, cols, ldq);
  if (overlap(q, nq, x, span(rows, cols, ldx, size)) || overlap(q, nq, residual, span(rows, cols, ldr, size)) ||
      overlap(q, nq, y, span(rows, cols, ldy, size)) || overlap(q, nq, h, span(rows, cols, ldh, size)))
    return fail(MUON_ERR_ARG, "q overlaps another matrix");
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  a.x = x, a.residual = residual, a.weight = weight, a.y = y, a.h = h, a.rstd = rstd;
  a.q = static_cast<uint8_t*>(q), a.qscale = static_cast<uint8_t*>(q_scale);
  a.ldx = ldx, a.ldr = ldr, a.ldy = ldy, a.ldh = ldh, a.ldq = ldq;
  a.rows = rows, a.cols = static_cast<int>(cols), a.weight_dt = weight_dt, a.fmt = fmt, a.eps = eps;
  return launched(launch_rms_norm(a, dt, sms, static_cast<cudaStream_t>(stream)), "launch_rms_norm");
}

size_t muon_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1 || cols > MUON_MAX_DIM) return 0;
  // the most CTAs that any type and sm_103 device give the kernel
  const int c = static_cast<int>(cols);
  const int ctas = std::max(rms_norm_grad_ctas(rows, c, MUON_FP32, MUON_MAX_SMS), rms_norm_grad_ctas(rows, c, MUON_BF16, MUON_MAX_SMS));
  return static_cast<size_t>(ctas) * cols * sizeof(float);
}

muon_status muon_rms_norm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const void* weight,
                                   muon_dtype weight_dt, const float* rstd, const void* dresidual, int64_t lddr,
                                   int64_t rows, int64_t cols, void* dx, int64_t lddx, float* dweight, void* ws,
                                   size_t ws_bytes, muon_dtype dt, void* stream) {
  clear_error();
  TRY(check_norm_shape(rows, cols, dt, weight, weight_dt));
  if (!dx && !dweight) return fail(MUON_ERR_ARG, "no output is given");
  if (misaligned(dweight, 4)) return fail(MUON_ERR_ALIGN, "dweight is not 4-byte aligned");
  const int size = dtype_bytes(dt);
  RmsNormGradArgs a = {};
  a.vec = weight && misaligned(weight, 16) ? 0 : 1;
  if (rows > 0) {
    TRY(check_rows("dy", dy, false, rows, cols, lddy, size, &a.vec));
    TRY(check_rows("h", h, false, rows, cols, ldh, size, &a.vec));
    TRY(check_rows("dresidual", dresidual, true, rows, cols, lddr, size, &a.vec));
    TRY(check_rows("dx", dx, true, rows, cols, lddx, size, &a.vec));
    if (!rstd) return fail(MUON_ERR_ARG, "rstd is NULL");
    if (misaligned(rstd, 4)) return fail(MUON_ERR_ALIGN, "rstd is not 4-byte aligned");
    if (clash(dx, lddx, dy, lddy, rows, cols, size) || clash(dx, lddx, dresidual, lddr, rows, cols, size) ||
        clash(dx, lddx, h, ldh, rows, cols, size))
      return fail(MUON_ERR_ARG, "dx partly overlaps an input");
    if (dweight) {
      if (!ws) return fail(MUON_ERR_ARG, "workspace is NULL");
      if (misaligned(ws, 16)) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
      if (ws_bytes < muon_rms_norm_backward_workspace_bytes(rows, cols))
        return fail(MUON_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes,
                    muon_rms_norm_backward_workspace_bytes(rows, cols));
    }
  }
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0)
    return dweight ? launched(cudaMemsetAsync(dweight, 0, cols * sizeof(float), s), "cudaMemsetAsync") : MUON_OK;
  a.dy = dy, a.h = h, a.weight = weight, a.rstd = rstd, a.dres = dresidual, a.dx = dx;
  a.partial = dweight ? static_cast<float*>(ws) : nullptr;
  a.dweight = dweight;
  a.lddy = lddy, a.ldh = ldh, a.lddr = lddr, a.lddx = lddx;
  a.rows = rows, a.cols = static_cast<int>(cols), a.weight_dt = weight_dt;
  return launched(launch_rms_norm_grad(a, dt, std::min(sms, MUON_MAX_SMS), s), "launch_rms_norm_grad");
}

// ------------------------------------------------------------------ 8 bits
size_t muon_fp8_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return 0;
  return static_cast<size_t>((cols + 511) / 512) * ((rows + 3) / 4 * 4) * 4;
}

muon_status muon_fp8_quantize(const void* x, int64_t ldx, int64_t rows, int64_t cols, muon_dtype dt, muon_fp8 fmt,
                              int square, void* q, int64_t ldq, void* q_scale, void* qt, int64_t ldqt, void* qt_scale,
                              void* stream) {
  clear_error();
  if (rows < 0 || rows > MUON_MAX_ROWS || cols < 0 || cols > MUON_MAX_ROWS)
    return fail(MUON_ERR_SHAPE, "%lldx%lld: sizes up to %lld", static_cast<long long>(rows), static_cast<long long>(cols),
                MUON_MAX_ROWS);
  if (!float_dt(dt)) return fail(MUON_ERR_ARG, "bad dtype %d", dt);
  if (!fp8_fmt(fmt)) return fail(MUON_ERR_ARG, "bad 8-bit format %d", fmt);
  if (square != 0 && square != 1) return fail(MUON_ERR_ARG, "square must be 0 or 1");
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!q && !qt) return fail(MUON_ERR_ARG, "no output is given");
  Fp8QuantArgs a = {};
  a.vec = 1;
  TRY(check_rows("x", x, false, rows, cols, ldx, dtype_bytes(dt), &a.vec));
  TRY(check_fp8_out("q", q, q_scale, rows, cols, ldq));
  TRY(check_fp8_out("qt", qt, qt_scale, cols, rows, ldqt));
  const long long nx = span(rows, cols, ldx, dtype_bytes(dt));
  const long long nq = span8(rows, cols, ldq), nqt = span8(cols, rows, ldqt);
  if (overlap(x, nx, q, nq) || overlap(x, nx, qt, nqt) || overlap(q, nq, qt, nqt))
    return fail(MUON_ERR_ARG, "an output overlaps x or the other output");
  muon_status st;
  gpu(&st);
  if (st != MUON_OK) return st;
  a.x = x, a.ldx = ldx, a.rows = rows, a.cols = cols, a.fmt = fmt, a.square = square;
  a.q = static_cast<uint8_t*>(q), a.qs = static_cast<uint8_t*>(q_scale), a.ldq = ldq;
  a.qt = static_cast<uint8_t*>(qt), a.qts = static_cast<uint8_t*>(qt_scale), a.ldqt = ldqt;
  return launched(launch_fp8_quantize(a, dt, static_cast<cudaStream_t>(stream)), "launch_fp8_quantize");
}

muon_status muon_fp8_matmul(const void* a, int64_t lda, const void* a_scale, muon_fp8 a_fmt, const void* b, int64_t ldb,
                            const void* b_scale, muon_fp8 b_fmt, int64_t m, int64_t n, int64_t k, const void* add,
                            int64_t ldadd, void* out, int64_t ldc, muon_dtype out_dt, void* stream) {
  clear_error();
  if (m < 0 || n < 0 || k < 0 || m > MUON_MAX_ROWS || n > MUON_MAX_ROWS || k > MUON_MAX_ROWS)
    return fail(MUON_ERR_SHAPE, "m=%lld n=%lld k=%lld: sizes in [0, %lld]", static_cast<long long>(m),
                static_cast<long long>(n), static_cast<long long>(k), MUON_MAX_ROWS);
  if (!fp8_fmt(a_fmt) || !fp8_fmt(b_fmt)) return fail(MUON_ERR_ARG, "bad 8-bit format");
  if (!float_dt(out_dt)) return fail(MUON_ERR_ARG, "bad dtype %d", out_dt);
  if (m == 0 || n == 0) return MUON_OK;
  const int size = dtype_bytes(out_dt);
  int vec = 1;
  TRY(check_rows("out", out, false, m, n, ldc, size, &vec));
  TRY(check_rows("add", add, true, m, n, ldadd, size, &vec));
  if (k > 0) {
    const void* p[2] = {a, b};
    const void* s[2] = {a_scale, b_scale};
    const long long ld[2] = {lda, ldb}, rows[2] = {m, n};
    for (int i = 0; i < 2; ++i) {
      const char name = i ? 'b' : 'a';
      if (!p[i] || !s[i]) return fail(MUON_ERR_ARG, "%c or its scale is NULL", name);
      if (misaligned(p[i], 16) || ld[i] % 16 || misaligned(s[i], 16))
        return fail(MUON_ERR_ALIGN, "%c and its scale must be 16-byte aligned, %c's row stride a multiple of 16", name, name);
      if (ld[i] < k) return fail(MUON_ERR_SHAPE, "%c: row stride %lld < k=%lld", name, ld[i], static_cast<long long>(k));
      if (overlap(out, span(m, n, ldc, size), p[i], span(rows[i], k, ld[i], 1)) ||
          overlap(out, span(m, n, ldc, size), s[i], static_cast<long long>(muon_fp8_scale_bytes(rows[i], k))))
        return fail(MUON_ERR_ARG, "out overlaps %c", name);
    }
  }
  if (add && clash(out, ldc, add, ldadd, m, n, size)) return fail(MUON_ERR_ARG, "out partly overlaps add");
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  Fp8GemmDesc d = {};
  d.a = a, d.b = b, d.a_scale = a_scale, d.b_scale = b_scale, d.lda = lda, d.ldb = ldb, d.m = m, d.n = n, d.k = k;
  d.a_fmt = a_fmt, d.b_fmt = b_fmt, d.add = add, d.out = out, d.ldadd = ldadd, d.ldc = ldc, d.out_dt = out_dt;
  const char* why = nullptr;
  return launched(launch_fp8_gemm(d, sms, static_cast<cudaStream_t>(stream), &why), "launch_fp8_gemm", why);
}

muon_status muon_fp8_status(void* stream) {
  clear_error();
  int word = 0;
  const cudaError_t e = fp8_take_status(static_cast<cudaStream_t>(stream), &word);
  if (e != cudaSuccess) return fail(MUON_ERR_CUDA, "status: %s", cudaGetErrorString(e));
  if (word & kStatusTimeout) return fail(MUON_ERR_TIMEOUT, "a kernel gave up on a bounded wait");
  return MUON_OK;
}

muon_status muon_debug_bounded_wait_fp8(long long max_cycles, void* stream) {
  clear_error();
  if (max_cycles <= 0 || max_cycles > 10000000000LL) return fail(MUON_ERR_ARG, "max_cycles out of range");
  int* p = nullptr;
  cudaError_t e = fp8_status_address(&p);
  if (e == cudaSuccess) e = launch_debug_wait(p, max_cycles, static_cast<cudaStream_t>(stream));
  return launched(e, "launch_debug_wait");
}

}  // extern "C"
