// block_abi.cu -- C ABI of the norms around a block, the gated activation and the transposition of 8-bit matrices.
// Every argument is checked before the first launch; nothing throws across the ABI.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "abi.h"

using namespace muon;

static long long scale_bytes(long long rows, long long cols) { return static_cast<long long>(muon_fp8_scale_bytes(rows, cols)); }

// A matrix of dt that is read or written, entered into `all`.
static muon_status take(Spans* all, const char* name, const void* p, bool optional, long long rows, long long cols, long long ld,
                        int size, bool out, int* vec) {
  TRY(check_rows(name, p, optional, rows, cols, ld, size, vec));
  all->add_rows(p, rows, ld * size, cols * size, out);
  return MUON_OK;
}
static muon_status take8(Spans* all, const char* name, const muon_fp8_out& o, int fmt, long long rows, long long cols) {
  if (!o.data && !o.scale) return MUON_OK;
  if (!fp8_fmt(fmt)) return fail(MUON_ERR_ARG, "%s: bad 8-bit format %d", name, fmt);
  TRY(check_fp8_out(name, o.data, o.scale, rows, cols, rows == 1 ? (cols + 15) / 16 * 16 : o.ld));
  all->add(o.data, span8(rows, cols, o.ld), true);
  all->add(o.scale, scale_bytes(rows, cols), true);
  return MUON_OK;
}
// A kept matrix: of dt, or 8-bit where it comes with scales.
static muon_status take_kept(Spans* all, const char* name, const void* p, const void* scale, long long rows, long long cols,
                             long long ld, int size, int fmt, int* vec) {
  if (!scale) return take(all, name, p, false, rows, cols, ld, size, false, vec);
  if (!p) return fail(MUON_ERR_ARG, "%s is NULL", name);
  if (!fp8_fmt(fmt)) return fail(MUON_ERR_ARG, "%s: bad 8-bit format %d", name, fmt);
  if (misaligned(p, 16) || misaligned(scale, 16) || (rows > 1 && ld % 16))
    return fail(MUON_ERR_ALIGN, "%s: data and scale must be 16-byte aligned, the row stride a multiple of 16", name);
  if (rows > 1 && ld < cols) return fail(MUON_ERR_SHAPE, "%s: row stride %lld < %lld columns", name, ld, cols);
  all->add(p, span(rows, cols, ld, 1), false);
  all->add(scale, scale_bytes(rows, cols), false);
  return MUON_OK;
}
// post, scale, pre: [cols] of one type.
static muon_status take_weights(Spans* all, const void* post, const void* scale, const void* pre, int dt, long long cols, int* vec) {
  if (!float_dt(dt)) return fail(MUON_ERR_ARG, "bad weight dtype %d", dt);
  if (!post || !pre) return fail(MUON_ERR_ARG, "a norm's weight is NULL");
  for (const void* p : {post, scale, pre}) {
    if (misaligned(p, dtype_bytes(dt))) return fail(MUON_ERR_ALIGN, "a weight is not aligned to its element size");
    if (misaligned(p, 16)) *vec = 0;
    all->add(p, cols * dtype_bytes(dt), false);
  }
  return MUON_OK;
}
static muon_status check_norm(long long rows, long long cols, int dt, int gate_per_row, float alpha) {
  if (rows < 0 || rows > MUON_MAX_ROWS) return fail(MUON_ERR_SHAPE, "rows=%lld out of [0, %lld]", rows, MUON_MAX_ROWS);
  if (cols < 1 || cols > MUON_MAX_DIM) return fail(MUON_ERR_SHAPE, "cols=%lld out of [1, %d]", cols, MUON_MAX_DIM);
  if (!float_dt(dt)) return fail(MUON_ERR_ARG, "bad dtype %d", dt);
  if (gate_per_row != 0 && gate_per_row != 1) return fail(MUON_ERR_ARG, "gate_per_row must be 0 or 1");
  if (!std::isfinite(alpha)) return fail(MUON_ERR_ARG, "need a finite alpha");
  return MUON_OK;
}

extern "C" {

muon_status muon_block_norm(const muon_block_norm_args* args, void* stream) {
  clear_error();
  if (!args) return fail(MUON_ERR_ARG, "args is NULL");
  const muon_block_norm_args& a = *args;
  const long long rows = a.rows, cols = a.cols;
  TRY(check_norm(rows, cols, a.dt, a.gate_per_row, a.alpha));
  if (!(std::isfinite(a.eps) && a.eps >= 0.f)) return fail(MUON_ERR_ARG, "need a finite eps >= 0");
  if (rows == 0) return MUON_OK;
  if (!a.y && !a.h && !a.rstd_x && !a.rstd_h && !a.q.data && !a.x8.data && !a.h8.data && !a.gate8.data)
    return fail(MUON_ERR_ARG, "no output is given");
  if (a.gate8.data && (!a.gate || a.gate_per_row)) return fail(MUON_ERR_ARG, "gate8 needs a gate [rows, cols]");
  const int size = dtype_bytes(a.dt);
  const long long gate_cols = a.gate_per_row ? 1 : cols;
  Spans all;
  int vec = 1, gate_vec = 1;
  TRY(take(&all, "x", a.x, false, rows, cols, a.ldx, size, false, &vec));
  TRY(take(&all, "residual", a.residual, false, rows, cols, a.ldr, size, false, &vec));
  TRY(take(&all, "gate", a.gate, true, rows, gate_cols, a.ldg, size, false, a.gate_per_row ? &gate_vec : &vec));
  TRY(take_weights(&all, a.post, a.scale, a.pre, a.weight_dt, cols, &vec));
  TRY(take(&all, "y", a.y, true, rows, cols, a.ldy, size, true, &vec));
  TRY(take(&all, "h", a.h, true, rows, cols, a.ldh, size, true, &vec));
  for (float* p : {a.rstd_x, a.rstd_h}) {
    if (misaligned(p, 4)) return fail(MUON_ERR_ALIGN, "rstd_x or rstd_h is not 4-byte aligned");
    all.add(p, rows * 4, true);
  }
  TRY(take8(&all, "q", a.q, a.fmt, rows, cols));
  TRY(take8(&all, "x8", a.x8, a.kept_fmt, rows, cols));
  TRY(take8(&all, "h8", a.h8, a.kept_fmt, rows, cols));
  TRY(take8(&all, "gate8", a.gate8, a.kept_fmt, rows, cols));
  if (all.clash()) return fail(MUON_ERR_ARG, "an output overlaps another matrix");
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  return launched(launch_block_norm(a, vec, sms, static_cast<cudaStream_t>(stream)), "launch_block_norm");
}

size_t muon_block_norm_backward_workspace_bytes_for(int64_t rows, int64_t cols, muon_dtype dt) {
  if (rows < 0 || cols < 1 || cols > MUON_MAX_DIM || !float_dt(dt)) return 0;
  return static_cast<size_t>(block_norm_grad_parts(rows, cols, dtype_bytes(dt), MUON_MAX_SMS)) * 2 * cols * sizeof(float);
}
size_t muon_block_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  return std::max(muon_block_norm_backward_workspace_bytes_for(rows, cols, MUON_BF16),
                  muon_block_norm_backward_workspace_bytes_for(rows, cols, MUON_FP32));
}

muon_status muon_block_norm_backward(const muon_block_norm_grad_args* args, void* stream) {
  clear_error();
  if (!args) return fail(MUON_ERR_ARG, "args is NULL");
  const muon_block_norm_grad_args& a = *args;
  const long long rows = a.rows, cols = a.cols;
  TRY(check_norm(rows, cols, a.dt, a.gate_per_row, a.alpha));
  const bool weights = a.dpost || a.dpre || a.dscale;
  if (!a.dx && !a.dresidual && !a.dgate && !weights) return fail(MUON_ERR_ARG, "no output is given");
  if (a.dgate && !a.gate) return fail(MUON_ERR_ARG, "dgate without a gate");
  if (a.dscale && !a.scale) return fail(MUON_ERR_ARG, "dscale without a scale");
  const int size = dtype_bytes(a.dt);
  const long long gate_cols = a.gate_per_row ? 1 : cols;
  Spans all;
  int vec = 1, gate_vec = 1;
  int* const gvec = a.gate_per_row ? &gate_vec : &vec;
  TRY(take_weights(&all, a.post, a.scale, a.pre, a.weight_dt, cols, &vec));
  for (float* p : {a.dpost, a.dpre, a.dscale}) {
    if (misaligned(p, 4)) return fail(MUON_ERR_ALIGN, "dpost, dpre or dscale is not 4-byte aligned");
    all.add(p, cols * 4, true);
  }
  if (rows > 0) {
    const bool kept8 = a.x_scale != nullptr, element = a.gate && !a.gate_per_row;
    if (kept8 != (a.h_scale != nullptr) || (element && kept8 != (a.gate_scale != nullptr)) || (!element && a.gate_scale))
      return fail(MUON_ERR_ARG, "x, h and a gate [rows, cols] are all kept in 8 bits, or none of them");
    TRY(take(&all, "dy", a.dy, false, rows, cols, a.lddy, size, false, &vec));
    TRY(take(&all, "dh", a.dh, true, rows, cols, a.lddh, size, false, &vec));
    TRY(take_kept(&all, "x", a.x, a.x_scale, rows, cols, a.ldx, size, a.kept_fmt, &vec));
    TRY(take_kept(&all, "h", a.h, a.h_scale, rows, cols, a.ldh, size, a.kept_fmt, &vec));
    if (a.gate) TRY(take_kept(&all, "gate", a.gate, a.gate_scale, rows, gate_cols, a.ldg, size, a.kept_fmt, gvec));
    TRY(take(&all, "dx", a.dx, true, rows, cols, a.lddx, size, true, &vec));
    TRY(take(&all, "dresidual", a.dresidual, true, rows, cols, a.lddr, size, true, &vec));
    TRY(take(&all, "dgate", a.dgate, true, rows, gate_cols, a.lddgate, size, true, gvec));
    for (const float* p : {a.rstd_x, a.rstd_h}) {
      if (!p) return fail(MUON_ERR_ARG, "rstd_x or rstd_h is NULL");
      if (misaligned(p, 4)) return fail(MUON_ERR_ALIGN, "rstd_x or rstd_h is not 4-byte aligned");
      all.add(p, rows * 4, false);
    }
    if (weights) {
      const size_t need = muon_block_norm_backward_workspace_bytes_for(rows, cols, static_cast<muon_dtype>(a.dt));
      if (!a.ws) return fail(MUON_ERR_ARG, "workspace is NULL");
      if (misaligned(a.ws, 16)) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
      if (a.ws_bytes < 0 || static_cast<size_t>(a.ws_bytes) < need)
        return fail(MUON_ERR_WORKSPACE, "workspace of %lld bytes, %zu needed", static_cast<long long>(a.ws_bytes), need);
      all.add(a.ws, static_cast<long long>(need), true);
    }
  }
  if (all.clash()) return fail(MUON_ERR_ARG, "an output or the workspace overlaps another matrix");
  muon_status st;
  const int sms = gpu(&st);
  if (st != MUON_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    for (float* p : {a.dpost, a.dpre, a.dscale})
      if (p) TRY(launched(cudaMemsetAsync(p, 0, cols * sizeof(float), s), "cudaMemsetAsync"));
    return MUON_OK;
  }
  return launched(launch_block_norm_grad(a, weights ? static_cast<float*>(a.ws) : nullptr, vec, std::min(sms, MUON_MAX_SMS), s),
                  "launch_block_norm_grad");
}

static muon_status check_gated(long long rows, long long cols, int dt, int act) {
  if (rows < 0 || rows > MUON_MAX_ROWS || cols < 0 || cols > MUON_MAX_ROWS)
    return fail(MUON_ERR_SHAPE, "%lldx%lld: sizes up to %lld", rows, cols, MUON_MAX_ROWS);
  if (!float_dt(dt)) return fail(MUON_ERR_ARG, "bad dtype %d", dt);
  if (act != MUON_SILU && act != MUON_GELU) return fail(MUON_ERR_ARG, "bad activation %d", act);
  return MUON_OK;
}

muon_status muon_gated_activation(const muon_gated_args* args, void* stream) {
  clear_error();
  if (!args) return fail(MUON_ERR_ARG, "args is NULL");
  const muon_gated_args& a = *args;
  const long long rows = a.rows, cols = a.cols;
  TRY(check_gated(rows, cols, a.dt, a.act));
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!a.y && !a.q.data && !a.gate8.data && !a.up8.data) return fail(MUON_ERR_ARG, "no output is given");
  const int size = dtype_bytes(a.dt);
  Spans all;
  int vec = 1;
  TRY(take(&all, "gate", a.gate, false, rows, cols, a.ldg, size, false, &vec));
  TRY(take(&all, "up", a.up, false, rows, cols, a.ldu, size, false, &vec));
  TRY(take(&all, "y", a.y, true, rows, cols, a.ldy, size, true, &vec));
  TRY(take8(&all, "q", a.q, a.fmt, rows, cols));
  TRY(take8(&all, "gate8", a.gate8, a.kept_fmt, rows, cols));
  TRY(take8(&all, "up8", a.up8, a.kept_fmt, rows, cols));
  if (all.clash()) return fail(MUON_ERR_ARG, "an output overlaps another matrix");
  muon_status st;
  gpu(&st);
  if (st != MUON_OK) return st;
  return launched(launch_gated(a, vec, static_cast<cudaStream_t>(stream)), "launch_gated");
}

muon_status muon_gated_activation_backward(const muon_gated_grad_args* args, void* stream) {
  clear_error();
  if (!args) return fail(MUON_ERR_ARG, "args is NULL");
  const muon_gated_grad_args& a = *args;
  const long long rows = a.rows, cols = a.cols;
  TRY(check_gated(rows, cols, a.dt, a.act));
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!a.dgate && !a.dup && !a.dgate_rows.data && !a.dgate_cols.data && !a.dup_rows.data && !a.dup_cols.data && !a.y_cols.data)
    return fail(MUON_ERR_ARG, "no output is given");
  if ((a.gate_scale != nullptr) != (a.up_scale != nullptr))
    return fail(MUON_ERR_ARG, "gate and up are both kept in 8 bits, or neither");
  const int size = dtype_bytes(a.dt);
  Spans all;
  int vec = 1;
  TRY(take(&all, "dy", a.dy, false, rows, cols, a.lddy, size, false, &vec));
  TRY(take_kept(&all, "gate", a.gate, a.gate_scale, rows, cols, a.ldg, size, a.kept_fmt, &vec));
  TRY(take_kept(&all, "up", a.up, a.up_scale, rows, cols, a.ldu, size, a.kept_fmt, &vec));
  TRY(take(&all, "dgate", a.dgate, true, rows, cols, a.lddgate, size, true, &vec));
  TRY(take(&all, "dup", a.dup, true, rows, cols, a.lddup, size, true, &vec));
  TRY(take8(&all, "dgate_rows", a.dgate_rows, a.fmt, rows, cols));
  TRY(take8(&all, "dup_rows", a.dup_rows, a.fmt, rows, cols));
  TRY(take8(&all, "dgate_cols", a.dgate_cols, a.fmt, cols, rows));
  TRY(take8(&all, "dup_cols", a.dup_cols, a.fmt, cols, rows));
  TRY(take8(&all, "y_cols", a.y_cols, a.y_fmt, cols, rows));
  if (all.clash()) return fail(MUON_ERR_ARG, "an output overlaps another matrix");
  muon_status st;
  gpu(&st);
  if (st != MUON_OK) return st;
  return launched(launch_gated_grad(a, vec, static_cast<cudaStream_t>(stream)), "launch_gated_grad");
}

muon_status muon_fp8_transpose(const void* q, int64_t ldq, const void* q_scale, int64_t rows, int64_t cols, muon_fp8 fmt,
                               void* qt, int64_t ldqt, void* qt_scale, void* stream) {
  clear_error();
  if (rows < 0 || rows > MUON_MAX_ROWS || cols < 0 || cols > MUON_MAX_ROWS)
    return fail(MUON_ERR_SHAPE, "%lldx%lld: sizes up to %lld", static_cast<long long>(rows), static_cast<long long>(cols),
                MUON_MAX_ROWS);
  if (!fp8_fmt(fmt)) return fail(MUON_ERR_ARG, "bad 8-bit format %d", fmt);
  if (rows == 0 || cols == 0) return MUON_OK;
  if (!q_scale) return fail(MUON_ERR_ARG, "q_scale is NULL");
  if (!qt || !qt_scale) return fail(MUON_ERR_ARG, "qt or its scale is NULL");
  Spans all;
  int vec = 1;
  TRY(take_kept(&all, "q", q, q_scale, rows, cols, ldq, 1, fmt, &vec));
  TRY(take8(&all, "qt", {qt, qt_scale, ldqt}, fmt, cols, rows));
  if (all.clash()) return fail(MUON_ERR_ARG, "qt overlaps q");
  muon_status st;
  gpu(&st);
  if (st != MUON_OK) return st;
  Fp8TransposeArgs a = {};
  a.q = static_cast<const uint8_t*>(q), a.qs = static_cast<const uint8_t*>(q_scale), a.ldq = ldq, a.rows = rows, a.cols = cols;
  a.qt = static_cast<uint8_t*>(qt), a.qts = static_cast<uint8_t*>(qt_scale), a.ldqt = ldqt;
  return launched(launch_fp8_transpose(a, fmt, static_cast<cudaStream_t>(stream)), "launch_fp8_transpose");
}

}  // extern "C"
