// abi.h -- checks shared by the C entry points of the operators around the update.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "train_ops.h"

namespace muon {

inline bool float_dt(int dt) { return dt == MUON_BF16 || dt == MUON_FP32 || dt == MUON_FP16; }
inline bool fp8_fmt(int f) { return f == MUON_E4M3 || f == MUON_E5M2; }
inline bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// Bytes spanned by a matrix of `rows` rows of `cols` elements, `ld` apart.
inline long long span(long long rows, long long cols, long long ld, int size) {
  return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * size : 0;
}
// And by an 8-bit one, whose rows are written up to the next multiple of 16 bytes.
inline long long span8(long long rows, long long cols, long long ld) { return span(rows, (cols + 15) / 16 * 16, ld, 1); }
inline bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// The device is an sm_103 GPU: its SM count (asked for once per device), or 0 with *st set.
inline int gpu(muon_status* st) {
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
inline muon_status launched(cudaError_t e, const char* what, const char* why = nullptr) {
  if (e == cudaSuccess) return MUON_OK;
  return fail(MUON_ERR_CUDA, "%s failed: %s%s%s", what, cudaGetErrorString(e), why ? ": " : "", why ? why : "");
}

// One matrix argument: NULL is allowed when `optional`; sets *vec to 0 where 16-byte accesses are not possible.
inline muon_status check_rows(const char* name, const void* p, bool optional, long long rows, long long cols, long long ld,
                              int size, int* vec) {
  if (!p) return optional ? MUON_OK : fail(MUON_ERR_ARG, "%s is NULL", name);
  if (misaligned(p, size)) return fail(MUON_ERR_ALIGN, "%s is not aligned to its element size", name);
  if (rows > 1 && ld < cols) return fail(MUON_ERR_SHAPE, "%s: row stride %lld < %lld columns", name, ld, cols);
  if (misaligned(p, 16) || (rows > 1 && ld * size % 16)) *vec = 0;
  return MUON_OK;
}
inline muon_status check_fp8_out(const char* name, const void* q, const void* scale, long long rows, long long cols,
                                 long long ld) {
  if (!q && !scale) return MUON_OK;
  if (!q || !scale) return fail(MUON_ERR_ARG, "%s: data and scale go together", name);
  if (misaligned(q, 16) || misaligned(scale, 16) || ld % 16)
    return fail(MUON_ERR_ALIGN, "%s: data and scale must be 16-byte aligned, the row stride a multiple of 16", name);
  if (ld < (cols + 15) / 16 * 16 && rows > 0)
    return fail(MUON_ERR_SHAPE, "%s: row stride %lld does not hold %lld columns padded to 16", name, ld, cols);
  return MUON_OK;
}
#define TRY(expr)                         \
  do {                                    \
    const muon_status st_ = (expr);       \
    if (st_ != MUON_OK) return st_;       \
  } while (0)

// The memory that a call touches: what it writes may share no byte with anything else.  Matrices whose rows lie between one
// another's (the halves of a wider one, say) share none.
struct Spans {
  struct One {
    uintptr_t begin, end, pitch, width;  // pitch and width: of rows, in bytes
    bool out;
  } s[32];
  int n = 0;
  void add(const void* p, long long bytes, bool out) { add_rows(p, 1, bytes, bytes, out); }
  void add_rows(const void* p, long long rows, long long pitch, long long width, bool out) {
    if (!p || rows < 1 || width < 1) return;
    const uintptr_t b = reinterpret_cast<uintptr_t>(p), w = static_cast<uintptr_t>(width);
    s[n++] = {b, b + static_cast<uintptr_t>((rows - 1) * pitch) + w, rows > 1 ? static_cast<uintptr_t>(pitch) : 0, w, out};
  }
  static bool between(const One& a, const One& b) {  // a begins first
    if (a.pitch == 0 || a.pitch != b.pitch) return false;
    const uintptr_t d = (b.begin - a.begin) % a.pitch;
    return d >= a.width && d + b.width <= a.pitch;
  }
  bool clash() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((s[i].out || s[j].out) && s[i].begin < s[j].end && s[j].begin < s[i].end &&
            !(s[i].begin <= s[j].begin ? between(s[i], s[j]) : between(s[j], s[i])))
          return true;
    return false;
  }
};

}  // namespace muon
