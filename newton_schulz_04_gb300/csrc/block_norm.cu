// block_norm.cu -- the norms behind a block and before the next one, with the block's gate and scale between them.
//
//   rho_x = 1 / sqrt(mean_j x_j^2 + eps)       h = alpha residual + sigmoid(gate) scale post (x rho_x)
//   rho_h = 1 / sqrt(mean_j h_j^2 + eps)       y = h rho_h pre
//
// Everything goes on in fp32 from unrounded values; y, h, the 8-bit y and the 8-bit copies of x, h and gate are each
// rounded once.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_norm.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {

// W warps to a row, K blocks to a warp; K = 0: any number, computed from memory again in each phase.
template <typename T, int W, int K>
__global__ void __launch_bounds__(W * 32) block_norm_kernel(const muon_block_norm_args a) {
  constexpr int KK = K ? K : 1;
  __shared__ float sh[2][1][W];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cols = static_cast<int>(a.cols);
  const int turns = K ? K : ((cols + 127) / 128 + W - 1) / W;
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = static_cast<const T*>(a.residual) + row * a.ldr;
  const T* gate = static_cast<const T*>(a.gate) + (a.gate ? row * a.ldg : 0);
  float v[KK][4];
  float sum[1] = {0.f};
  float sig = 1.f;
  if (a.gate && a.gate_per_row) sig = sigmoid<T>(to_f32(*gate));
  auto column = [&](int k, int j) { return (warp + W * k) * 128 + lane + 32 * j; };
#pragma unroll
  for (int k = 0; k < turns; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = column(k, j);
      const float f = load_or<T>(x, col, col < cols, 0.f);
      if (K) v[k < KK ? k : 0][j] = f;
      sum[0] = fmaf(f, f, sum[0]);
    }
  cta_sums<W, 1>(sum, sh, 0);
  const float n = static_cast<float>(cols), inv_n = 1.f / n;
  const float rx = row_rstd(sum[0], n, inv_n, a.eps);
  auto stream = [&](int col, float f) {
    if (col >= cols) return 0.f;
    float b = f * rx * (load_weight(a.post, a.weight_dt, col, true) * load_weight(a.scale, a.weight_dt, col, true));
    b *= a.gate && !a.gate_per_row ? sigmoid<T>(to_f32(gate[col])) : sig;
    return fmaf(a.alpha, to_f32(res[col]), b);
  };
  sum[0] = 0.f;
#pragma unroll
  for (int k = 0; k < turns; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = column(k, j);
      const float h = stream(col, K ? v[k < KK ? k : 0][j] : load_or<T>(x, col, col < cols, 0.f));
      if (K) v[k < KK ? k : 0][j] = h;
      sum[0] = fmaf(h, h, sum[0]);
    }
  cta_sums<W, 1>(sum, sh, 1);
  const float rh = row_rstd(sum[0], n, inv_n, a.eps);
  if (threadIdx.x == 0) {
    if (a.rstd_x) a.rstd_x[row] = rx;
    if (a.rstd_h) a.rstd_h[row] = rh;
  }
#pragma unroll
  for (int k = 0; k < turns; ++k) {
    const int kb = warp + W * k;
    if (kb * 128 >= cols) break;
    float h[4], f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = column(k, j);
      h[j] = K ? v[k < KK ? k : 0][j] : stream(col, load_or<T>(x, col, col < cols, 0.f));
      if (a.h && col < cols) static_cast<T*>(a.h)[row * a.ldh + col] = from_f32<T>(h[j]);
      f[j] = h[j] * rh * load_weight(a.pre, a.weight_dt, col, col < cols);
      if (col >= cols) f[j] = 0.f;
      if (a.y && col < cols) static_cast<T*>(a.y)[row * a.ldy + col] = from_f32<T>(f[j]);
    }
    if (a.q.data) store_block8(a.q, a.fmt, row, a.rows, cols, kb, f);
    if (a.h8.data) store_block8(a.h8, a.kept_fmt, row, a.rows, cols, kb, h);
    if (a.x8.data) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_or<T>(x, column(k, j), column(k, j) < cols, 0.f);
      store_block8(a.x8, a.kept_fmt, row, a.rows, cols, kb, f);
    }
    if (a.gate8.data) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_or<T>(gate, column(k, j), column(k, j) < cols, 0.f);
      store_block8(a.gate8, a.kept_fmt, row, a.rows, cols, kb, f);
    }
  }
  if (a.q.data) pad_blocks8(a.q, row, a.rows, cols);
  if (a.h8.data) pad_blocks8(a.h8, row, a.rows, cols);
  if (a.x8.data) pad_blocks8(a.x8, row, a.rows, cols);
  if (a.gate8.data) pad_blocks8(a.gate8, row, a.rows, cols);
}

// ------------------------------------------------------------------ ring of rows
// Largest magnitude of a piece as the upper 16 bits of its fp32 bits, rounded up.  A scale byte is the exponent field of
// bits + 0x1fffff, whose only border within a binade (0x600000) is a multiple of 2^16: it comes out the same.
template <int E>
__device__ __forceinline__ uint32_t piece_max(const float (&v)[E]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < E; ++i) m = max(m, abs_bits(v[i]));
  return (m + 0xffffu) >> 16;
}
// A row's 8-bit copies: a block of 128 columns lies in 128 / E neighbouring lanes, two matrices share one exchange.
template <int E>
struct Row8 {
  long long row, rows, rows4;
  int cols, blocks;
  bool live;
  __device__ __forceinline__ void store(const muon_fp8_out& o, int fmt, int col, uint32_t amax, const float (&v)[E]) const {
    const uint32_t byte = fp8_scale_byte(amax, fmt ? 15 : 8);
    const float inv = fp8_inverse_scale(byte);
    if (!live) return;
    if (col < ((cols + 15) & ~15)) {
      uint8_t* p = static_cast<uint8_t*>(o.data) + row * o.ld + col;
      if constexpr (E == 8) {
        *reinterpret_cast<uint2*>(p) = fmt ? fp8_pack8<true>(v, inv) : fp8_pack8<false>(v, inv);
      } else {
        *reinterpret_cast<uint32_t*>(p) = fmt ? fp8_pack4<true>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv)
                                              : fp8_pack4<false>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      }
    }
    const int kb = col / 128;
    if (col % 128 == 0 && kb < blocks) scale(o, kb, byte);
  }
  __device__ __forceinline__ void scale(const muon_fp8_out& o, int kb, uint32_t byte) const {
    uint8_t* p = static_cast<uint8_t*>(o.scale) + fp8_scale_offset(kb, row, rows4);
    *p = static_cast<uint8_t>(byte);
    if (row == rows - 1)  // scales of no row are 1
      for (long long r = rows; r < rows4; ++r) p[(r - rows + 1) * 4] = 127;
  }
  // Pieces of two matrices, each stored where it is asked for; all lanes call.
  __device__ __forceinline__ void two(const muon_fp8_out& a, int fa, const float (&va)[E], const muon_fp8_out& b, int fb,
                                      const float (&vb)[E], int col) const {
    if (!a.data && !b.data) return;
    uint32_t m = piece_max(va) | piece_max(vb) << 16;
#pragma unroll
    for (int o = 64 / E; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (a.data) store(a, fa, col, m << 16, va);
    if (b.data) store(b, fb, col, m & 0xffff0000u, vb);
  }
};

// CL CTAs of a cluster to a row, G threads of each, C pieces of 16 bytes to a thread, a ring of S rows.
template <typename T, int G, int C, int S, int MINB, int CL>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB) block_norm_ring_kernel(const muon_block_norm_args a) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G, E = 16 / static_cast<int>(sizeof(T));
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ RowSums<G, TH, 1, CL> sums;
  const Ring<T, TH, C, S, 3> ring{ring_smem};
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int t = threadIdx.x % G, rr = threadIdx.x / G, cols = static_cast<int>(a.cols);
  int n[C], col[C], off[C];  // existing columns of each piece, its first, and the same where one exists
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = ((rank * C + c) * G + t) * E;
    n[c] = max(0, min(E, cols - col[c]));
    off[c] = n[c] ? col[c] : 0;
  }
  const bool element = a.gate && !a.gate_per_row;
  const long long step = static_cast<long long>(gridDim.x / CL) * R, row0 = static_cast<long long>(blockIdx.x / CL) * R + rr;
  long long frow = row0;  // next row to fetch
  auto fetch = [&](int slot) {
    if (frow < a.rows) {
      const T* fx = static_cast<const T*>(a.x) + frow * a.ldx;
      const T* fr = static_cast<const T*>(a.residual) + frow * a.ldr;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int bytes = n[c] * static_cast<int>(sizeof(T));
        ring.fetch(slot, 0, c, fx + off[c], bytes);
        ring.fetch(slot, 1, c, fr + off[c], bytes);
        if (element) ring.fetch(slot, 2, c, static_cast<const T*>(a.gate) + frow * a.ldg + off[c], bytes);
      }
    }
    cp_async_commit();
    frow += step;
  };
  if (CL > 1) cluster_sync();  // the others' shared memory is there
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float w1[C][E], w2[C][E];  // scale post, pre
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_weight_piece<E>(a.scale, a.weight_dt, off[c], n[c], w2[c]);
    load_weight_piece<E>(a.post, a.weight_dt, off[c], n[c], w1[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) w1[c][i] *= w2[c][i];
    load_weight_piece<E>(a.pre, a.weight_dt, off[c], n[c], w2[c]);
  }
  const auto row_gate = [&](long long row) {
    return a.gate && !element && row < a.rows ? to_f32(static_cast<const T*>(a.gate)[row * a.ldg]) : 0.f;
  };
  float next_gate = row_gate(row0);  // a row ahead
  const float fcols = static_cast<float>(cols), inv_cols = 1.f / fcols;
  Row8<E> out{row0, a.rows, (a.rows + 3) & ~3LL, cols, (cols + 127) / 128, true};
  int slot = 0, turn = 0;
  // all threads of a CTA take the same number of turns (the barriers of the sums)
  for (long long row = row0; row - rr < a.rows; row += step, turn += 2) {
    const bool live = R == 1 || row < a.rows;
    if (row - rr + step >= a.rows) pdl_launch_dependents();  // the last row: earlier, the next kernel's CTAs take SMs from these
    const float row_sig = a.gate && !element ? sigmoid<T>(next_gate) : 1.f;
    next_gate = row_gate(row + step);
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    float h[C][E], sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x[E];
      ring.read(slot, 0, c, x);
#pragma unroll
      for (int i = 0; i < E; ++i) sum[0] = fmaf(x[i], x[i], sum[0]);
    }
    sums(sum, turn);
    const float rx = row_rstd(sum[0], fcols, inv_cols, a.eps);
    sum[0] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float x[E], g[E];
      ring.read(slot, 0, c, x);
      ring.read(slot, 1, c, h[c]);
      if (element) ring.read(slot, 2, c, g);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float b = x[i] * rx * w1[c][i] * (element ? sigmoid<T>(g[i]) : row_sig);
        h[c][i] = fmaf(a.alpha, h[c][i], b);
        sum[0] = fmaf(h[c][i], h[c][i], sum[0]);
      }
    }
    sums(sum, turn + 1);
    const float rh = row_rstd(sum[0], fcols, inv_cols, a.eps);
    if (live && t == 0 && rank == 0) {
      if (a.rstd_x) a.rstd_x[row] = rx;
      if (a.rstd_h) a.rstd_h[row] = rh;
    }
    out.row = row, out.live = live;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const bool in = n[c] == E || i < n[c];
        y[i] = in ? h[c][i] * rh * w2[c][i] : 0.f;
        h[c][i] = in ? h[c][i] : 0.f;
      }
      if (live && a.h) store_piece(static_cast<T*>(a.h) + row * a.ldh + off[c], n[c], h[c]);
      if (live && a.y) store_piece(static_cast<T*>(a.y) + row * a.ldy + off[c], n[c], y);
      out.two(a.q, a.fmt, y, a.h8, a.kept_fmt, h[c], col[c]);
      if (a.x8.data || a.gate8.data) {
        ring.read(slot, 0, c, y);
        if (element) ring.read(slot, 2, c, h[c]);
        out.two(a.x8, a.kept_fmt, y, a.gate8, a.kept_fmt, h[c], col[c]);
      }
    }
    // blocks past the last column, up to a whole scale word
    if (rank == 0 && live && t < (cols + 511) / 512 * 4 - out.blocks) {
      const int kb = out.blocks + t;
      if (a.q.data) out.scale(a.q, kb, 127u);
      if (a.x8.data) out.scale(a.x8, kb, 127u);
      if (a.h8.data) out.scale(a.h8, kb, 127u);
      if (a.gate8.data) out.scale(a.gate8, kb, 127u);
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
}

template <typename T, int G, int C, int S, int MINB, int CL>
static cudaError_t launch_ring(const muon_block_norm_args& a, int sms, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int smem = Ring<T, TH, C, S, 3>::BYTES;
  static_assert(smem * MINB <= 220 * 1024, "shared memory of an SM");
  static bool done[64] = {false};
  static int known[64] = {0};
  const auto kernel = block_norm_ring_kernel<T, G, C, S, MINB, CL>;
  cudaError_t e = smem_limit(kernel, smem, done);
  if (e != cudaSuccess) return e;
  int most = MINB * sms;
  if (CL > 1) {
    e = resident_clusters(kernel, TH, smem, CL, known, &most);
    if (e != cudaSuccess) return e;
  }
  const long long want = (a.rows + R - 1) / R;
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(std::min<long long>(want, most)) * CL), dim3(TH), smem, CL, st, a);
}

// Threads, pieces and CTAs of a row by its width.
template <typename T>
static cudaError_t dispatch_ring(const muon_block_norm_args& a, int sms, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = static_cast<int>((a.cols + E - 1) / E);
  if (pieces <= 32) return launch_ring<T, 32, 1, 6, 5, 1>(a, sms, st);
  if (pieces <= 64) return launch_ring<T, 64, 1, 4, 8, 1>(a, sms, st);
  if (pieces <= 128) return launch_ring<T, 64, 2, 3, 5, 1>(a, sms, st);
  if (pieces <= 256) return launch_ring<T, 256, 1, 4, 4, 1>(a, sms, st);
  if (pieces <= 512) return launch_ring<T, 256, 2, 4, 2, 1>(a, sms, st);
  if (pieces <= 1024) return launch_ring<T, 512, 2, 4, 1, 1>(a, sms, st);
  if (pieces <= 2048) return launch_ring<T, 512, 2, 4, 1, 2>(a, sms, st);
  if (pieces <= 4096) return launch_ring<T, 512, 2, 4, 1, 4>(a, sms, st);
  return launch_ring<T, 512, 2, 4, 1, 8>(a, sms, st);
}

template <typename T>
static cudaError_t dispatch_norm(const muon_block_norm_args& a, cudaStream_t st) {
  const auto go = [&](auto kernel, int warps) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(a.rows)), dim3(warps * 32), 0, st, a);
  };
  if (a.cols <= 512) return go(block_norm_kernel<T, 4, 1>, 4);
  if (a.cols <= 2048) return go(block_norm_kernel<T, 8, 2>, 8);
  if (a.cols <= 4096) return go(block_norm_kernel<T, 16, 2>, 16);
  if (a.cols <= 16384) return go(block_norm_kernel<T, 16, 8>, 16);
  return go(block_norm_kernel<T, 16, 0>, 16);
}

cudaError_t launch_block_norm(const muon_block_norm_args& a, int vec, int sms, cudaStream_t st) {
  const auto go = [&](auto t) {
    using T = decltype(t);
    // 8 CTAs of 1024 pieces hold MUON_MAX_DIM 16-bit columns and half as many of fp32
    const bool ring = vec && a.cols <= 8 * 1024 * (16 / static_cast<int>(sizeof(T)));
    return ring ? dispatch_ring<T>(a, sms, st) : dispatch_norm<T>(a, st);
  };
  return a.dt == MUON_BF16 ? go(__nv_bfloat16()) : a.dt == MUON_FP16 ? go(__half()) : go(float());
}

}  // namespace muon
