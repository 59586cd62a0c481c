// rms_norm.cu -- root-mean-square norm with the residual's addition and an 8-bit copy, and its gradient.
//
//   s = x + residual          h = round(s)          rho = 1 / sqrt(mean_j s_j^2 + eps)
//   y = s rho w               q = y in 8 bits with one power-of-two scale for each 128 columns (fp8.cuh)
//
// Everything is computed from the unrounded fp32 s, and y, h and q are each
// rounded once.  The gradient, with h as stored (what the forward pass keeps):
//
//   g = dy w      dx = rho (g - h rho^2 mean_j(g_j h_j)) + dres      dw_j = sum_rows dy_j h_j rho
//
// Both are one pass over memory, and bound by it.  A row belongs to G threads,
// 16 bytes of it each, C times.  CTAs are persistent: every thread copies
// its own pieces of the next rows to a ring in shared memory (cp.async, S rows
// deep) that no other thread reads, so the ring needs no barrier, and the only
// synchronisation of a row is the one of its sum.  One short-lived CTA per row
// moved 8192 x 4096 bf16 rows in 60 us (forward) and, with its rows in a loop but
// nothing fetched ahead, 119 us (gradient); the ring takes 49 (6.2 TB/s) and 47.5 (5.7 TB/s,
// with the second kernel).  The depths below were measured at 33.5M elements: at 4096 columns, rings of 3
// to 6 rows on 2 CTAs per SM take 49 to 53 us, on 3 or 4 CTAs 56 to 69.
//
// The next kernel on the stream is let in only at a CTA's last row: started earlier, the CTAs of
// another ring kernel crowd onto the SMs that have room and leave others short of their share.
//
// Rows that allow no 16-byte accesses, or that are too wide for a ring, take kernels
// that load straight to registers, the widest (WIDE) a second time from L1 / L2.  They are a
// few times slower: 33.5M bf16 elements in rows of 1023 take 203 us (gradient 257), of 255 145 (245), of 16383 190
// (386); 16384 fp32 columns 113 (218).
//
// A block of 128 columns lies in 16 neighbouring lanes (32 in fp32), so its
// largest magnitude takes four or five shuffles.  The weight's gradient is summed over a CTA's rows in
// registers, written per CTA, and the CTAs' rows are added in a fixed order by a
// second kernel (no atomics: the same bits every time).
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

__device__ __forceinline__ void load_weight8(const void* w, int dt, int col, int n, bool full, float (&v)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  } else if (dt == MUON_FP32) {
    load8(static_cast<const float*>(w) + col, n, full, v);
  } else if (dt == MUON_BF16) {
    load8(static_cast<const __nv_bfloat16*>(w) + col, n, full, v);
  } else {
    load8(static_cast<const __half*>(w) + col, n, full, v);
  }
}

// Sum over the G threads of a row (G a power of two >= 32, R rows per CTA);
// every thread gets it.  sh: one float per warp.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 32) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  constexpr int W = G / 32;
  const int first = (threadIdx.x / G) * W;
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += sh[first + w];
  return s;
}

// y's 8-bit copy.  A thread holds pieces t, t + G, ... of E columns (G a multiple of 128 / E),
// so the 128 / E lanes of a 128-column block are neighbours.
template <int E>
struct QOut {
  uint8_t* data;   // this row, column E t
  uint8_t* scale;  // scale word of this row, first group
  int t;
  long long rows4;
  __device__ __forceinline__ QOut(const RmsNormArgs& a, long long row, int t_) : t(t_), rows4((a.rows + 3) & ~3LL) {
    data = a.q + (a.q ? row * a.ldq + E * t_ : 0);
    scale = a.qscale + (a.q ? row * 4 : 0);
  }
  __device__ __forceinline__ void advance(const RmsNormArgs& a, long long rows) {
    data += rows * a.ldq;
    scale += rows * 4;
  }
  // piece `piece` + t (piece a multiple of G); all lanes call.  Up to the row's
  // next multiple of 16 bytes: columns past the end hold 0.
  __device__ __forceinline__ void store(const RmsNormArgs& a, int piece, const float (&y)[E], bool live, bool last) const {
    constexpr int LANES = 128 / E;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < E; ++i) m = max(m, abs_bits(y[i]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t byte = fp8_scale_byte(m, a.fmt ? 15 : 8);
    if (!live) return;
    const float inv = fp8_inverse_scale(byte);
    if ((piece + t) * E < ((a.cols + 15) & ~15)) {
      if constexpr (E == 8) {
        *reinterpret_cast<uint2*>(data + piece * E) = a.fmt ? fp8_pack8<true>(y, inv) : fp8_pack8<false>(y, inv);
      } else {
        *reinterpret_cast<uint32_t*>(data + piece * E) =
            a.fmt ? fp8_pack4<true>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv)
                  : fp8_pack4<false>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
      }
    }
    const int kb = (piece + t) / LANES;
    if (t % LANES == 0 && kb < ((a.cols + 511) >> 9) * 4) {
      uint8_t* p = scale + (kb >> 2) * rows4 * 4 + (kb & 3);
      *p = static_cast<uint8_t>(byte);
      if (last)  // scales of no row are 1
        for (long long r = a.rows; r < rows4; ++r) p[(r - a.rows + 1) * 4] = 127;
    }
  }
};

// Scale words are four blocks: blocks first, first + step, ... past the last column.
__device__ __forceinline__ void pad_q_scales(const RmsNormArgs& a, long long row, int first, int step) {
  const long long rows4 = (a.rows + 3) & ~3LL;
  const int blocks = ((a.cols + 511) >> 9) * 4;
  for (int kb = first; kb < blocks; kb += step) {
    a.qscale[fp8_scale_offset(kb, row, rows4)] = 127;
    if (row == a.rows - 1)
      for (long long r = a.rows; r < rows4; ++r) a.qscale[fp8_scale_offset(kb, r, rows4)] = 127;
  }
}

// ------------------------------------------------------------------ ring of rows
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {  // the rest of 16 is zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

// E elements of 16 bytes: a thread's piece of a row.
template <typename T>
__device__ __forceinline__ void unpack_piece(const uint4& w, float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(w, v, T());
  } else {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
}
// n of the elements exist.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int n, const float (&v)[16 / sizeof(T)]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  union {
    uint4 w;
    T e[E];
  } u;
#pragma unroll
  for (int i = 0; i < E; ++i) u.e[i] = from_f32<T>(v[i]);
  if (n == E) {
    *reinterpret_cast<uint4*>(p) = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) p[i] = u.e[i];
  }
}
template <int E>
__device__ __forceinline__ void load_weight_piece(const void* w, int dt, int col, int n, float (&v)[E]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 1.f;
  } else if (dt == MUON_FP32) {
    const float* p = static_cast<const float*>(w) + col;
    if (n == E) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const float4 f = reinterpret_cast<const float4*>(p)[q];
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = i < n ? p[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      v[i] = i >= n               ? 0.f
             : dt == MUON_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(w)[col + i])
                               : to_f32(static_cast<const __half*>(w)[col + i]);
  }
}

// A thread's slots: S rows of NA arrays of C pieces; thread-private.
template <typename T, int TH, int C, int S, int NA>
struct Ring {
  static constexpr int BYTES = S * NA * C * TH * 16;
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int slot, int arr, int c) const {
    return base + (((slot * NA + arr) * C + c) * TH + static_cast<int>(threadIdx.x)) * 16;
  }
  // Piece c of a row: the 16 bytes at src, `bytes` of which exist (the rest reads as 0).
  __device__ __forceinline__ void fetch(int slot, int arr, int c, const T* src, int bytes) const {
    copy16(smem_u32(at(slot, arr, c)), src, bytes);
  }
  __device__ __forceinline__ void read(int slot, int arr, int c, float (&v)[16 / sizeof(T)]) const {
    unpack_piece<T>(*reinterpret_cast<const uint4*>(at(slot, arr, c)), v);
  }
};

// Sum over the G threads of a row, one barrier: `sh` alternates between two buffers.
template <int G, int TH>
__device__ __forceinline__ float ring_sum(float v, float (*sh)[TH / 32], int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 32) return v;
  if ((threadIdx.x & 31) == 0) sh[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  constexpr int W = G / 32;  // added as a tree: each of the last additions rounds the whole
  float s = sh[turn & 1][(threadIdx.x / G) * W + (threadIdx.x & (W - 1))];
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 1 / sqrt(sum / cols + eps), the quotient and the root corrected by a step of Newton's:
// y goes on to 8 bits, and an error common to a row moves all its values that lie near the middle of two.
__device__ __forceinline__ float row_rstd(float sum, float cols, float inv_cols, float eps) {
  const float q = sum * inv_cols;
  const float m = (isfinite(q) ? fmaf(fmaf(-q, cols, sum), inv_cols, q) : q) + eps;
  const float r = rsqrtf(m);
  const float better = fmaf(0.5f * r, fmaf(-(m * r), r, 1.f), r);
  return isfinite(better) ? better : r;  // of a sum of 0 (without eps), infinity or NaN
}

template <typename T, int G, int C, int S, int MINB>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB) rms_norm_ring_kernel(const RmsNormArgs a) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G, E = 16 / static_cast<int>(sizeof(T));
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float sh[2][TH / 32];
  const Ring<T, TH, C, S, 2> ring{ring_smem};
  const int t = threadIdx.x % G, rr = threadIdx.x / G;
  int n[C], off[C];  // existing columns of each piece, and its first (0 where none exists)
#pragma unroll
  for (int c = 0; c < C; ++c) {
    n[c] = max(0, min(E, a.cols - (c * G + t) * E));
    off[c] = n[c] ? (c * G + t) * E : 0;
  }
  const long long step = static_cast<long long>(gridDim.x) * R, row0 = static_cast<long long>(blockIdx.x) * R + rr;
  long long frow = row0;  // next row to fetch
  const T* fx = static_cast<const T*>(a.x) + row0 * a.ldx;
  const T* fr = a.residual ? static_cast<const T*>(a.residual) + row0 * a.ldr : nullptr;
  auto fetch = [&](int slot) {
    if (frow < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) ring.fetch(slot, 0, c, fx + off[c], n[c] * static_cast<int>(sizeof(T)));
      if (fr) {
#pragma unroll
        for (int c = 0; c < C; ++c) ring.fetch(slot, 1, c, fr + off[c], n[c] * static_cast<int>(sizeof(T)));
      }
    }
    cp_async_commit();
    frow += step;
    fx += step * a.ldx;
    if (fr) fr += step * a.ldr;
  };
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float w[C][E];  // the weight stays in registers
#pragma unroll
  for (int c = 0; c < C; ++c) load_weight_piece<E>(a.weight, a.weight_dt, off[c], n[c], w[c]);
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  T* ph = static_cast<T*>(a.h) + (a.h ? row0 * a.ldh : 0);
  T* py = static_cast<T*>(a.y) + (a.y ? row0 * a.ldy : 0);
  QOut<E> q(a, row0, t);
  int slot = 0, turn = 0;
  // all threads of a CTA take the same number of turns (the barrier in ring_sum)
  for (long long row = row0; row - rr < a.rows; row += step, ++turn) {
    const bool live = R == 1 || row < a.rows;
    if (row - rr + step >= a.rows) pdl_launch_dependents();  // the last row, see above
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    float s[C][E];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ring.read(slot, 0, c, s[c]);
      if (fr) {
        float r[E];
        ring.read(slot, 1, c, r);
#pragma unroll
        for (int i = 0; i < E; ++i) s[c][i] += r[i];
      }
      if (R > 1 && !live) {
#pragma unroll
        for (int i = 0; i < E; ++i) s[c][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) sum = fmaf(s[c][i], s[c][i], sum);
    }
    sum = ring_sum<G, TH>(sum, sh, turn);
    const float rstd = row_rstd(sum, static_cast<float>(a.cols), inv_cols, a.eps);
    if (live && t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (live && a.h) store_piece(ph + off[c], n[c], s[c]);
#pragma unroll
      for (int i = 0; i < E; ++i) s[c][i] = s[c][i] * rstd * w[c][i];
      if (n[c] < E) {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (i >= n[c]) s[c][i] = 0.f;
      }
      if (live && a.y) store_piece(py + off[c], n[c], s[c]);
      if (a.q) q.store(a, c * G, s[c], live, row == a.rows - 1);
    }
    if (a.q && live) pad_q_scales(a, row, C * G * E / 128 + t, G);
    ph += step * a.ldh;
    py += step * a.ldy;
    q.advance(a, step);
    slot = slot + 1 == S ? 0 : slot + 1;
  }
}

template <typename T, int G, int C, bool WIDE>
__global__ void __launch_bounds__(G < 128 ? 128 : G) rms_norm_kernel(const RmsNormArgs a) {
  constexpr int R = G < 128 ? 128 / G : 1;  // rows per CTA
  __shared__ float sh[(G < 128 ? 128 : G) / 32];
  pdl_launch_dependents();
  pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * R + threadIdx.x / G;
  const bool live = row < a.rows;
  const int t = threadIdx.x % G;
  const T* x = static_cast<const T*>(a.x) + (live ? row * a.ldx : 0);
  const T* res = a.residual ? static_cast<const T*>(a.residual) + (live ? row * a.ldr : 0) : nullptr;
  auto load = [&](int col, float (&s)[8]) {
    const int n = live ? max(0, min(8, a.cols - col)) : 0;
    const bool full = n == 8 && a.vec;
    load8(x + col, n, full, s);
    if (res) {
      float r[8];
      load8(res + col, n, full, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += r[i];
    }
  };
  float s[C][8];
  float sum = 0.f;
  const int chunks = WIDE ? (a.cols + 8 * G - 1) / (8 * G) : C;
  if (WIDE) {
    for (int c = 0; c < chunks; ++c) {
      load((c * G + t) * 8, s[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(s[0][i], s[0][i], sum);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) load((c * G + t) * 8, s[c]);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(s[c][i], s[c][i], sum);
  }
  sum = row_sum<G>(sum, sh);
  const float cols = static_cast<float>(a.cols), rstd = row_rstd(sum, cols, 1.f / cols, a.eps);
  const QOut<8> q(a, live ? row : 0, t);
  if (live && t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < (WIDE ? 1 : C); ++c) {
    for (int cc = c; cc < (WIDE ? chunks : c + 1); ++cc) {
      const int col = (cc * G + t) * 8;
      float v[8], w[8];
      if (WIDE) {
        load(col, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s[c][i];
      }
      const int n = live ? max(0, min(8, a.cols - col)) : 0;
      const bool full = n == 8 && a.vec;
      if (a.h) store8(static_cast<T*>(a.h) + row * a.ldh + col, n, full, v);
      load_weight8(a.weight, a.weight_dt, col, n, full, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] * rstd * w[i] : 0.f;
      if (a.y) store8(static_cast<T*>(a.y) + row * a.ldy + col, n, full, v);
      if (a.q) q.store(a, cc * G, v, live, row == a.rows - 1);
    }
  }
  if (a.q && live) pad_q_scales(a, row, chunks * G / 16 + t, G);
}

template <typename T, int G, int C, bool WIDE>
static cudaError_t launch_norm(const RmsNormArgs& a, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  return launch_pdl(rms_norm_kernel<T, G, C, WIDE>, dim3(static_cast<unsigned>((a.rows + R - 1) / R)), dim3(TH), 0, st,
                    a);
}

// The kernel's shared-memory limit, raised once per device.
template <typename F>
static cudaError_t ring_smem_limit(F kernel, int bytes, bool (&done)[64]) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <typename T, int G, int C, int S, int MINB>
static cudaError_t launch_norm_ring(const RmsNormArgs& a, int sms, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int smem = Ring<T, TH, C, S, 2>::BYTES;
  static_assert(smem * MINB <= 220 * 1024, "shared memory of an SM");
  static bool done[64] = {false};
  const cudaError_t e = ring_smem_limit(rms_norm_ring_kernel<T, G, C, S, MINB>, smem, done);
  if (e != cudaSuccess) return e;
  const long long want = (a.rows + R - 1) / R;
  return launch_pdl(rms_norm_ring_kernel<T, G, C, S, MINB>, dim3(static_cast<unsigned>(std::min<long long>(want, MINB * sms))),
                    dim3(TH), smem, st, a);
}

// Threads per row, pieces of 16 bytes per thread, rows of the ring and CTAs per SM by the row's width, as measured at
// 33.5M elements; without 16-byte accesses, 8 columns per thread.
template <typename T>
static cudaError_t dispatch_norm(const RmsNormArgs& a, int sms, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = (a.cols + E - 1) / E;
  if (a.vec) {
    if (pieces <= 32) return launch_norm_ring<T, 32, 1, 8, 6>(a, sms, st);
    if (pieces <= 64) return launch_norm_ring<T, 64, 1, 4, 8>(a, sms, st);
    if (pieces <= 128) return launch_norm_ring<T, 64, 2, 4, 4>(a, sms, st);
    if (pieces <= 256) return launch_norm_ring<T, 256, 1, 4, 3>(a, sms, st);
    if (pieces <= 512) return launch_norm_ring<T, 256, 2, 5, 2>(a, sms, st);
    if (pieces <= 1024) return launch_norm_ring<T, 512, 2, 4, 1>(a, sms, st);
    if (pieces <= 2048) return launch_norm_ring<T, 1024, 2, 3, 1>(a, sms, st);
  } else {
    if (a.cols <= 512) return launch_norm<T, 32, 2, false>(a, st);
    if (a.cols <= 4096) return launch_norm<T, 256, 2, false>(a, st);
    if (a.cols <= 16384) return launch_norm<T, 512, 4, false>(a, st);
  }
  return launch_norm<T, 512, 1, true>(a, st);
}

cudaError_t launch_rms_norm(const RmsNormArgs& a, int dt, int sms, cudaStream_t st) {
  if (dt == MUON_BF16) return dispatch_norm<__nv_bfloat16>(a, sms, st);
  if (dt == MUON_FP16) return dispatch_norm<__half>(a, sms, st);
  return dispatch_norm<float>(a, sms, st);
}

// ------------------------------------------------------------------ gradient
template <typename T, int G, int C, bool WIDE>
__global__ void __launch_bounds__(G < 128 ? 128 : G) rms_norm_grad_kernel(const RmsNormGradArgs a) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  __shared__ float sh[TH / 32];
  extern __shared__ float dwsh[];  // R > 1: [R - 1][cols]
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % G, rr = threadIdx.x / G;
  const int chunks = WIDE ? (a.cols + 8 * G - 1) / (8 * G) : C;
  float* part = a.partial ? a.partial + static_cast<long long>(blockIdx.x) * a.cols : nullptr;
  float dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.f;
  bool first = true;
  for (long long r0 = static_cast<long long>(blockIdx.x) * R; r0 < a.rows; r0 += static_cast<long long>(gridDim.x) * R) {
    const long long row = r0 + rr;
    const bool live = row < a.rows;
    const T* dy = static_cast<const T*>(a.dy) + (live ? row * a.lddy : 0);
    const T* h = static_cast<const T*>(a.h) + (live ? row * a.ldh : 0);
    const float rstd = live ? a.rstd[row] : 0.f;
    float d[C][8], x[C][8];
    float sum = 0.f;
    auto load = [&](int col, float (&dv)[8], float (&xv)[8], float (&w)[8]) {
      const int n = live ? max(0, min(8, a.cols - col)) : 0;
      const bool full = n == 8 && a.vec;
      load8(dy + col, n, full, dv);
      load8(h + col, n, full, xv);
      load_weight8(a.weight, a.weight_dt, col, n, full, w);
    };
    if (WIDE) {
      for (int c = 0; c < chunks; ++c) {
        float w[8];
        load((c * G + t) * 8, d[0], x[0], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(d[0][i] * w[i], x[0][i], sum);
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float w[8];
        load((c * G + t) * 8, d[c], x[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(d[c][i] * w[i], x[c][i], sum);
      }
    }
    sum = row_sum<G>(sum, sh);
    const float k = sum / static_cast<float>(a.cols) * rstd * rstd;
#pragma unroll
    for (int c = 0; c < (WIDE ? 1 : C); ++c) {
      for (int cc = c; cc < (WIDE ? chunks : c + 1); ++cc) {
        const int col = (cc * G + t) * 8;
        const int n = live ? max(0, min(8, a.cols - col)) : 0;
        const bool full = n == 8 && a.vec;
        float w[8];
        if (WIDE) load(col, d[0], x[0], w);
        else load_weight8(a.weight, a.weight_dt, col, n, full, w);
        if (a.dx) {
          float v[8];
          if (a.dres) {
            load8(static_cast<const T*>(a.dres) + (live ? row * a.lddr : 0) + col, n, full, v);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += rstd * (d[c][i] * w[i] - x[c][i] * k);
          store8(static_cast<T*>(a.dx) + (live ? row * a.lddx : 0) + col, n, full, v);
        }
        if (part) {
          if (WIDE) {  // this thread alone holds these columns of the CTA's partial row
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < n) part[col + i] = (first ? 0.f : part[col + i]) + d[0][i] * x[0][i] * rstd;
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dw[c][i] = fmaf(d[c][i] * x[c][i], rstd, dw[c][i]);
          }
        }
      }
    }
    first = false;
  }
  if (part && !WIDE) {
    if (R > 1) {  // join the CTA's row groups
      __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * G + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (rr > 0 && col + i < a.cols) dwsh[(rr - 1) * a.cols + col + i] = dw[c][i];
      }
      __syncthreads();
    }
    if (rr == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * G + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (col + i < a.cols) {
            float v = dw[c][i];
            for (int r = 1; r < R; ++r) v += dwsh[(r - 1) * a.cols + col + i];
            part[col + i] = v;
          }
        }
      }
    }
  }
}

template <typename T, int G, int C, int S, int MINB>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB) rms_norm_grad_ring_kernel(const RmsNormGradArgs a) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G, E = 16 / static_cast<int>(sizeof(T));
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ float sh[2][TH / 32];
  const Ring<T, TH, C, S, 3> ring{ring_smem};
  const int t = threadIdx.x % G, rr = threadIdx.x / G;
  int n[C], off[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    n[c] = max(0, min(E, a.cols - (c * G + t) * E));
    off[c] = n[c] ? (c * G + t) * E : 0;
  }
  const long long step = static_cast<long long>(gridDim.x) * R, row0 = static_cast<long long>(blockIdx.x) * R + rr;
  const bool add = a.dres && a.dx;
  long long frow = row0;  // next row to fetch
  const T* fd = static_cast<const T*>(a.dy) + row0 * a.lddy;
  const T* fh = static_cast<const T*>(a.h) + row0 * a.ldh;
  const T* fr = static_cast<const T*>(a.dres) + (add ? row0 * a.lddr : 0);
  auto fetch = [&](int slot) {
    if (frow < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int bytes = n[c] * static_cast<int>(sizeof(T));
        ring.fetch(slot, 0, c, fd + off[c], bytes);
        ring.fetch(slot, 1, c, fh + off[c], bytes);
        if (add) ring.fetch(slot, 2, c, fr + off[c], bytes);
      }
    }
    cp_async_commit();
    frow += step;
    fd += step * a.lddy;
    fh += step * a.ldh;
    fr += step * a.lddr;
  };
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float w[C][E], dw[C][E];  // the weight stays in registers
#pragma unroll
  for (int c = 0; c < C; ++c) load_weight_piece<E>(a.weight, a.weight_dt, off[c], n[c], w[c]);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < E; ++i) dw[c][i] = 0.f;
  const float inv_cols = 1.f / static_cast<float>(a.cols);
  int slot = 0, turn = 0;
  float next_rstd = row0 < a.rows ? __ldg(a.rstd + row0) : 0.f;  // a row ahead
  T* px = static_cast<T*>(a.dx) + (a.dx ? row0 * a.lddx : 0);
  for (long long row = row0; row - rr < a.rows; row += step, ++turn) {
    const bool live = R == 1 || row < a.rows;
    if (row - rr + step >= a.rows) pdl_launch_dependents();
    const float rstd = next_rstd;
    next_rstd = row + step < a.rows ? __ldg(a.rstd + row + step) : 0.f;
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    float d[C][E], x[C][E];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ring.read(slot, 0, c, d[c]);
      ring.read(slot, 1, c, x[c]);
      if (R > 1 && !live) {
#pragma unroll
        for (int i = 0; i < E; ++i) d[c][i] = x[c][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        sum = fmaf(d[c][i] * w[c][i], x[c][i], sum);
        dw[c][i] = fmaf(d[c][i] * x[c][i], rstd, dw[c][i]);
      }
    }
    sum = ring_sum<G, TH>(sum, sh, turn);
    const float k = sum * inv_cols * rstd * rstd;
    if (a.dx && live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[E];
        if (add) {
          ring.read(slot, 2, c, v);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) v[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += rstd * (d[c][i] * w[c][i] - x[c][i] * k);
        store_piece(px + off[c], n[c], v);
      }
    }
    px += step * a.lddx;
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  if (!a.partial) return;
  float* part = a.partial + static_cast<long long>(blockIdx.x) * a.cols;
  if (R > 1) {  // join the CTA's row groups through the ring's memory
    cp_async_wait<0>();
    __syncthreads();
    float* dwsh = reinterpret_cast<float*>(ring_smem);  // [R - 1][C * E][G]
    if (rr > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i) dwsh[((rr - 1) * C * E + c * E + i) * G + t] = dw[c][i];
    }
    __syncthreads();
    if (rr > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < E; ++i)
        for (int r = 1; r < R; ++r) dw[c][i] += dwsh[((r - 1) * C * E + c * E + i) * G + t];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * G + t) * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n[c]) part[col + i] = dw[c][i];
  }
}

// dweight[j] = sum over the CTAs' rows: 32 columns by 32 row groups per CTA, then a column to a
// warp (8 row groups, each a chain of 38 loads, took 2 us longer).
__global__ void __launch_bounds__(1024) rms_norm_dweight_kernel(const float* partial, int ctas, int cols, float* dweight) {
  __shared__ float sh[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int r = g; r < ctas; r += 32) s += partial[static_cast<long long>(r) * cols + col];
  }
  sh[g][lane] = s;
  __syncthreads();
  pdl_launch_dependents();  // not before: a persistent grid that starts beside these CTAs finds no room for all of its own
  s = sh[lane][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + g < cols) dweight[blockIdx.x * 32 + g] = s;
}

// CTAs of the gradient kernel: what an SM holds of the ring kernels (the others take as many).
struct GradPlan {
  int rows_per_cta, ctas_per_sm;
};
static GradPlan grad_plan(int cols, int dt) {
  const int pieces = dt == MUON_FP32 ? (cols + 3) / 4 : (cols + 7) / 8;
  if (pieces <= 32) return {4, 6};
  if (pieces <= 64) return {4, 3};
  if (pieces <= 128) return {2, 3};
  if (pieces <= 256) return {1, 3};
  if (pieces <= 512 || pieces > 2048) return {1, 2};
  return {1, 1};
}
int rms_norm_grad_ctas(long long rows, int cols, int dt, int sms) {
  const GradPlan p = grad_plan(cols, dt);
  return static_cast<int>(
      std::max(1LL, std::min<long long>((rows + p.rows_per_cta - 1) / p.rows_per_cta, static_cast<long long>(p.ctas_per_sm) * sms)));
}

template <typename T, int G, int C, bool WIDE>
static cudaError_t launch_grad(const RmsNormGradArgs& a, int ctas, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  const size_t smem = a.partial ? sizeof(float) * (R - 1) * a.cols : 0;
  return launch_pdl(rms_norm_grad_kernel<T, G, C, WIDE>, dim3(ctas), dim3(TH), smem, st, a);
}

template <typename T, int G, int C, int S, int MINB>
static cudaError_t launch_grad_ring(const RmsNormGradArgs& a, int ctas, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G;
  constexpr int smem = Ring<T, TH, C, S, 3>::BYTES;
  static_assert(smem * MINB <= 224 * 1024, "shared memory of an SM");
  static bool done[64] = {false};
  const cudaError_t e = ring_smem_limit(rms_norm_grad_ring_kernel<T, G, C, S, MINB>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(rms_norm_grad_ring_kernel<T, G, C, S, MINB>, dim3(ctas), dim3(TH), smem, st, a);
}

// The ring kernels' rows per CTA and CTAs per SM are grad_plan's; the others step over any number of CTAs.  Of 16384 columns
// in 16-bit types a thread has 64 registers, about half of what the loop wants, and spills, and the ring
// has room for two rows only: 33.5M elements take 73 us, at 8192 columns 48.
template <typename T>
static cudaError_t dispatch_grad(const RmsNormGradArgs& a, int ctas, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = (a.cols + E - 1) / E;
  if (a.vec) {
    if (pieces <= 32) return launch_grad_ring<T, 32, 1, 4, 6>(a, ctas, st);
    if (pieces <= 64) return launch_grad_ring<T, 32, 2, 4, 3>(a, ctas, st);
    if (pieces <= 128) return launch_grad_ring<T, 64, 2, 4, 3>(a, ctas, st);
    if (pieces <= 256) return launch_grad_ring<T, 256, 1, 5, 3>(a, ctas, st);
    if (pieces <= 512) return launch_grad_ring<T, 256, 2, 4, 2>(a, ctas, st);
    if (pieces <= 1024) return launch_grad_ring<T, 512, 2, 4, 1>(a, ctas, st);
    if (pieces <= 2048) return launch_grad_ring<T, 1024, 2, 2, 1>(a, ctas, st);
  } else {
    if (a.cols <= 512) return launch_grad<T, 32, 2, false>(a, ctas, st);
    if (a.cols <= 2048) return launch_grad<T, 128, 2, false>(a, ctas, st);
    if (a.cols <= 4096) return launch_grad<T, 256, 2, false>(a, ctas, st);
    if (a.cols <= 8192) return launch_grad<T, 512, 2, false>(a, ctas, st);
  }
  return launch_grad<T, 512, 1, true>(a, ctas, st);
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int dt, int sms, cudaStream_t st) {
  const int ctas = rms_norm_grad_ctas(a.rows, a.cols, dt, sms);
  cudaError_t e = dt == MUON_BF16   ? dispatch_grad<__nv_bfloat16>(a, ctas, st)
                  : dt == MUON_FP16 ? dispatch_grad<__half>(a, ctas, st)
                                    : dispatch_grad<float>(a, ctas, st);
  if (e != cudaSuccess || !a.partial) return e;
  return launch_pdl(rms_norm_dweight_kernel, dim3((a.cols + 31) / 32), dim3(1024), 0, st,
                    static_cast<const float*>(a.partial), ctas, a.cols, a.dweight);
}

}  // namespace muon
