// block_norm_rows.cu -- the norms behind a block and before the next one, with the block's gate and scale between them.
//
//   rho_x = 1 / sqrt(mean_j x_j^2 + eps)       h = alpha residual + sigmoid(gate) scale post (x rho_x)
//   rho_h = 1 / sqrt(mean_j h_j^2 + eps)       y = h rho_h pre
//
// Compiled once for each type and alignment of rows (MUON_ROWS_T, MUON_ROWS_ANYWHERE).
//
// Everything goes on in fp32 from unrounded values; y, h, the 8-bit y and the 8-bit copies of x, h and gate are each
// rounded once.
//
// One pass over memory from a ring of rows in shared memory, as in rms_norm.cu: persistent CTAs, each thread 16 bytes of a row
// C times, with the row's two sums behind one another.  Bound by memory and, close behind, by issuing: 8192 x 4096 bf16 with a
// gate, an 8-bit output and three 8-bit copies takes 71 us (5.7 TB/s, 45 instructions an element, 57 % of the issue
// slots); with scalars of fp32 and an exchange for the scales of each copy it took 126, with choices at run time 81.  A
// cluster's exchange takes half of a row's time, so a row belongs to one CTA up to 16384 16-bit columns (8192 columns 75 us,
// 16384 104, in clusters of two 123).  Rows that start anywhere: 113 at 4095 columns, 121 at 1023.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block_norm.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace muon {

// ------------------------------------------------------------------ the widest rows
// fp32 rows that a cluster's rings do not hold: 16 warps to a row, computed from memory again in each phase.
template <typename T>
__global__ void __launch_bounds__(512) block_norm_wide_kernel(const muon_block_norm_args a) {
  constexpr int W = 16;
  __shared__ float sh[2][1][W];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cols = static_cast<int>(a.cols);
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = static_cast<const T*>(a.residual) + row * a.ldr;
  const T* gate = static_cast<const T*>(a.gate) + (a.gate ? row * a.ldg : 0);
  float sum[1] = {0.f};
  float sig = 1.f;
  if (a.gate && a.gate_per_row) sig = sigmoid2<float>(both(to_f32(*gate))).x;
  for (int col = threadIdx.x; col < cols; col += 512) sum[0] = fmaf(to_f32(x[col]), to_f32(x[col]), sum[0]);
  cta_sums<W, 1>(sum, sh, 0);
  const float n = static_cast<float>(cols), inv_n = 1.f / n;
  const float rx = row_rstd(sum[0], n, inv_n, a.eps);
  auto stream = [&](int col) {
    if (col >= cols) return 0.f;
    float b = to_f32(x[col]) * rx * (load_weight(a.post, a.weight_dt, col, true) * load_weight(a.scale, a.weight_dt, col, true));
    b *= a.gate && !a.gate_per_row ? sigmoid2<T>(both(to_f32(gate[col]))).x : sig;
    return fmaf(a.alpha, to_f32(res[col]), b);
  };
  sum[0] = 0.f;
  for (int col = threadIdx.x; col < cols; col += 512) {
    const float h = stream(col);
    sum[0] = fmaf(h, h, sum[0]);
  }
  cta_sums<W, 1>(sum, sh, 1);
  const float rh = row_rstd(sum[0], n, inv_n, a.eps);
  if (threadIdx.x == 0) {
    if (a.rstd_x) a.rstd_x[row] = rx;
    if (a.rstd_h) a.rstd_h[row] = rh;
  }
  for (int kb = warp; kb * 128 < cols; kb += W) {
    float h[4], f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = kb * 128 + lane + 32 * j;
      h[j] = stream(col);
      f[j] = col < cols ? h[j] * rh * load_weight(a.pre, a.weight_dt, col, true) : 0.f;
      if (a.h && col < cols) static_cast<T*>(a.h)[row * a.ldh + col] = from_f32<T>(h[j]);
      if (a.y && col < cols) static_cast<T*>(a.y)[row * a.ldy + col] = from_f32<T>(f[j]);
    }
    if (a.q.data) store_block8(a.q, a.fmt, row, a.rows, cols, kb, f);
    if (a.h8.data) store_block8(a.h8, a.kept_fmt, row, a.rows, cols, kb, h);
    if (a.x8.data) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_or<T>(x, kb * 128 + lane + 32 * j, kb * 128 + lane + 32 * j < cols, 0.f);
      store_block8(a.x8, a.kept_fmt, row, a.rows, cols, kb, f);
    }
    if (a.gate8.data) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = load_or<T>(gate, kb * 128 + lane + 32 * j, kb * 128 + lane + 32 * j < cols, 0.f);
      store_block8(a.gate8, a.kept_fmt, row, a.rows, cols, kb, f);
    }
  }
  if (a.q.data) pad_blocks8(a.q, row, a.rows, cols);
  if (a.h8.data) pad_blocks8(a.h8, row, a.rows, cols);
  if (a.x8.data) pad_blocks8(a.x8, row, a.rows, cols);
  if (a.gate8.data) pad_blocks8(a.gate8, row, a.rows, cols);
}

// ------------------------------------------------------------------ ring of rows
// S rows of x, residual and gate, C pieces each: a thread's own 16 bytes, or (ANYWHERE) a warp's and a little more.
template <typename T, int G, int C, int S, bool ANYWHERE>
struct RowRing {
  static constexpr int TH = G < 128 ? 128 : G, LANES = G < 32 ? G : 32;
  static constexpr int ARRAY = ANYWHERE ? TH / 32 * kWarpSlot<LANES> : TH * 16, BYTES = S * 3 * C * ARRAY;
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int slot, int arr, int c) const {
    uint8_t* p = base + ((slot * 3 + arr) * C + c) * ARRAY;
    return ANYWHERE ? p + threadIdx.x / 32 * kWarpSlot<LANES> : p + threadIdx.x * 16;
  }
  __device__ __forceinline__ uint4 piece(int slot, int arr, int c, int off) const {
    if constexpr (ANYWHERE) return read_anywhere<LANES, C <= 2>(at(slot, arr, c), off);
    else return *reinterpret_cast<const uint4*>(at(slot, arr, c));
  }
};

// CL CTAs of a cluster to a row, G threads of each, C pieces of 16 bytes to a thread, a ring of S rows.  GATE: a gate of every
// element.  E4M3: all 8-bit outputs are of e4m3, and the copies for the gradient among them.  Compiled apart: choices at run
// time leave pieces of code too small to be overlapped.
template <typename T, int G, int C, int S, int MINB, int CL, bool GATE, bool E4M3, bool ANYWHERE>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB) block_norm_ring_kernel(const muon_block_norm_args a) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  using P = Pairs<T>;
  constexpr int E = P::E, N = P::N, PIECE = G * E;  // PIECE: from a thread's piece to its next
  constexpr int LANES = G < 32 ? G : 32;  // of a row in a warp
  using Scales = Scales4<(128 / E < G ? 128 / E : G), sizeof(T) == 2>;
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ RowSum<G, TH, CL> row_total;
  const RowRing<T, G, C, S, ANYWHERE> ring{ring_smem};
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int t = threadIdx.x % G, rr = threadIdx.x / G, cols = static_cast<int>(a.cols);
  const int col = (rank * C * G + t) * E;  // of the first piece
  int n[C];                                // existing columns of each
#pragma unroll
  for (int c = 0; c < C; ++c) n[c] = max(0, min(E, cols - col - c * PIECE));
  const bool row_gated = !GATE && a.gate;
  const long long step = static_cast<long long>(gridDim.x / CL) * R, row0 = static_cast<long long>(blockIdx.x / CL) * R + rr;
  long long frow = row0;  // next row to fetch
  constexpr int BEGIN = ANYWHERE ? 0 : 1;  // pointers to rows, or to the thread's pieces of them
  const T* fx = static_cast<const T*>(a.x) + row0 * a.ldx + BEGIN * col;
  const T* fr = static_cast<const T*>(a.residual) + row0 * a.ldr + BEGIN * col;
  const T* fg = static_cast<const T*>(a.gate) + (GATE ? row0 * a.ldg + BEGIN * col : 0);
  auto fetch = [&](int slot) {
    if (frow < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const auto get = [&](int arr, const T* row, const void* matrix) {
          if constexpr (ANYWHERE) {
            fetch_anywhere<T, LANES>(ring.at(slot, arr, c), row, (col + c * PIECE) / E, cols, static_cast<const uint8_t*>(matrix));
          } else {
            copy16(smem_u32(ring.at(slot, arr, c)), row + (n[c] ? c * PIECE : -col), n[c] * static_cast<int>(sizeof(T)));
          }
        };
        get(0, fx, a.x);
        get(1, fr, a.residual);
        if (GATE) get(2, fg, a.gate);
      }
    }
    cp_async_commit();
    frow += step, fx += step * a.ldx, fr += step * a.ldr;
    if (GATE) fg += step * a.ldg;
  };
  if (CL > 1) cluster_sync();  // the others' shared memory is there
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float2 w1[C][N], w2[C][N];  // scale post, pre
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = n[c] ? col + c * PIECE : 0;
    float v[E], s[E];
    load_weights<T, ANYWHERE>(a.scale, a.weight_dt, at, n[c], s);
    load_weights<T, ANYWHERE>(a.post, a.weight_dt, at, n[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) w1[c][i] = make_float2(v[2 * i] * s[2 * i], v[2 * i + 1] * s[2 * i + 1]);
    load_weights<T, ANYWHERE>(a.pre, a.weight_dt, at, n[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) w2[c][i] = make_float2(v[2 * i], v[2 * i + 1]);
  }
  const auto row_gate = [&](long long row) {
    return row_gated && row < a.rows ? to_f32(static_cast<const T*>(a.gate)[row * a.ldg]) : 0.f;
  };
  float next_gate = row_gate(row0);  // a row ahead
  const float fcols = static_cast<float>(cols), inv_cols = 1.f / fcols;
  T* ph = static_cast<T*>(a.h) + row0 * a.ldh + BEGIN * col;
  T* py = static_cast<T*>(a.y) + row0 * a.ldy + BEGIN * col;
  const auto put = [&](T* p, int c, bool live, const P& v) {
    if constexpr (ANYWHERE) store_anywhere<T, LANES>(p, (col + c * PIECE) / E, live ? cols - col - c * PIECE : 0, v);
    else if (live) v.store(p + c * PIECE, n[c]);
  };
  // rows' addresses modulo 16
  const auto off = [&](const void* p, long long ld, long long row) {
    return static_cast<int>((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) + static_cast<uint32_t>(row * ld) * sizeof(T)) & 15u);
  };
  // the 8-bit copies: y, h, x, gate; each lane keeps the scales of one of them
  uint8_t* p8[4] = {static_cast<uint8_t*>(a.q.data) + row0 * a.q.ld + col, static_cast<uint8_t*>(a.h8.data) + row0 * a.h8.ld + col,
                    static_cast<uint8_t*>(a.x8.data) + row0 * a.x8.ld + col, static_cast<uint8_t*>(a.gate8.data) + row0 * a.gate8.ld + col};
  const bool eight = E4M3 || a.q.data || a.h8.data || a.x8.data || a.gate8.data;
  const int mine = Scales::mine(), top = (mine ? a.kept_fmt : a.fmt) ? 15 : 8, cols16 = (cols + 15) & ~15;
  const long long rows4 = (a.rows + 3) & ~3LL;
  uint8_t* const scales = static_cast<uint8_t*>(mine == 0 ? a.q.scale : mine == 1 ? a.h8.scale : mine == 2 ? a.x8.scale : a.gate8.scale);
  uint8_t* ps = scales + row0 * 4;
  const bool keeper = scales && threadIdx.x % Scales::Q == 0;
  int slot = 0, turn = 0;
  // all threads of a CTA take the same number of turns (the barriers of the sums)
  for (long long row = row0; row - rr < a.rows; row += step, turn += 2) {
    const bool live = R == 1 || row < a.rows;
    if (row - rr + step >= a.rows) pdl_launch_dependents();  // the last row: earlier, the next kernel's CTAs take SMs from these
    float2 sig = both(1.f);
    if (row_gated) sig = both(sigmoid2<float>(both(next_gate)).x), next_gate = row_gate(row + step);
    if (ANYWHERE) __syncwarp();
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    if (ANYWHERE) __syncwarp();
    const int ox = ANYWHERE ? off(a.x, a.ldx, row) : 0, orr = ANYWHERE ? off(a.residual, a.ldr, row) : 0;
    const int og = ANYWHERE && GATE ? off(a.gate, a.ldg, row) : 0;
    P h[C];
    constexpr bool KEEP = ANYWHERE && C <= 2;  // what takes shifts to read, where there are registers for it
    uint4 kx[C], kg[C];
    float2 two = both(0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      P x;
      kx[c] = ring.piece(slot, 0, c, ox);
      x.unpack(kx[c]);
#pragma unroll
      for (int i = 0; i < N; ++i) two = fma2(x.v[i], x.v[i], two);
    }
    const float rx = row_rstd(row_total(total(two), turn), fcols, inv_cols, a.eps);
    two = both(0.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      P x, g;
      x.unpack(KEEP ? kx[c] : ring.piece(slot, 0, c, ox));
      h[c].unpack(ring.piece(slot, 1, c, orr));
      if (GATE) kg[c] = ring.piece(slot, 2, c, og), g.unpack(kg[c]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (GATE) sig = sigmoid2<T>(g.v[i]);
        const float2 b = mul2(mul2(mul2(x.v[i], both(rx)), w1[c][i]), sig);
        h[c].v[i] = fma2(both(a.alpha), h[c].v[i], b);
        two = fma2(h[c].v[i], h[c].v[i], two);
      }
    }
    const float rh = row_rstd(row_total(total(two), turn + 1), fcols, inv_cols, a.eps);
    if (live && t == 0 && rank == 0) {
      if (a.rstd_x) a.rstd_x[row] = rx;
      if (a.rstd_h) a.rstd_h[row] = rh;
    }
    // past the last column everything is 0 (or NaN, where a norm's factor is not finite and so the whole row)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      P y;
#pragma unroll
      for (int i = 0; i < N; ++i) y.v[i] = mul2(mul2(h[c].v[i], both(rh)), w2[c][i]);
      if (a.h) put(ph, c, live, h[c]);
      if (a.y) put(py, c, live, y);
      if (eight) {
        P x, g;
        uint32_t m[4] = {y.largest(), h[c].largest(), 0u, 0u};
        if (E4M3 || a.x8.data) x.unpack(KEEP ? kx[c] : ring.piece(slot, 0, c, ox)), m[2] = x.largest();
        if (GATE && (E4M3 || a.gate8.data)) g.unpack(KEEP ? kg[c] : ring.piece(slot, 2, c, og)), m[3] = g.largest();
        const Scales s(m, top);
        if (live && col + c * PIECE < cols16) {
          if constexpr (E4M3) {
            if (a.q.data) y.template store8<false>(p8[0] + c * PIECE, s.inv[0]);
            h[c].template store8<false>(p8[1] + c * PIECE, s.inv[1]);
            x.template store8<false>(p8[2] + c * PIECE, s.inv[2]);
            if (GATE) g.template store8<false>(p8[3] + c * PIECE, s.inv[3]);
          } else {
            if (a.q.data) y.store8(p8[0] + c * PIECE, s.inv[0], a.fmt);
            if (a.h8.data) h[c].store8(p8[1] + c * PIECE, s.inv[1], a.kept_fmt);
            if (a.x8.data) x.store8(p8[2] + c * PIECE, s.inv[2], a.kept_fmt);
            if (GATE && a.gate8.data) g.store8(p8[3] + c * PIECE, s.inv[3], a.kept_fmt);
          }
        }
        const int kb = (col + c * PIECE) / 128;
        if (keeper && live && kb * 128 < cols) ps[(kb >> 2) * rows4 * 4 + (kb & 3)] = static_cast<uint8_t>(s.byte);
      }
    }
    ph += step * a.ldh, py += step * a.ldy, ps += step * 4;
    p8[0] += step * a.q.ld, p8[1] += step * a.h8.ld, p8[2] += step * a.x8.ld, p8[3] += step * a.gate8.ld;
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  // scales of no block or row, up to whole words and to four rows, are 1
  if (!eight || rank != 0) return;
  const int blocks = (cols + 127) / 128, end = (cols + 511) / 512 * 4;
  const auto fill = [&](const muon_fp8_out& o, int kb, long long row) {
    if (o.data) static_cast<uint8_t*>(o.scale)[fp8_scale_offset(kb, row, rows4)] = 127;
  };
  for (long long row = row0; row < a.rows; row += step)
    for (int kb = blocks + t; kb < end; kb += G) fill(a.q, kb, row), fill(a.h8, kb, row), fill(a.x8, kb, row), fill(a.gate8, kb, row);
  if (blockIdx.x == 0)
    for (long long row = a.rows + rr; row < rows4; row += R)
      for (int kb = t; kb < end; kb += G) fill(a.q, kb, row), fill(a.h8, kb, row), fill(a.x8, kb, row), fill(a.gate8, kb, row);
}

template <typename T, int G, int C, int S, int MINB, int CL, bool GATE, bool E4M3, bool ANYWHERE>
static cudaError_t launch_ring(const muon_block_norm_args& a, int sms, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int smem = RowRing<T, G, C, S, ANYWHERE>::BYTES;
  static_assert(smem * MINB <= 220 * 1024, "shared memory of an SM");
  static bool done[64] = {false};
  static int known[64] = {0};
  const auto kernel = block_norm_ring_kernel<T, G, C, S, MINB, CL, GATE, E4M3, ANYWHERE>;
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

// Threads and pieces of a row, rows of the ring, CTAs of an SM and of a cluster by the row's width, as measured at 33.5M elements:
// 256, 512, 1024, 2048 columns take 77, 74, 71, 71 us; one piece to a thread 77, 76 to 80, 79 to 81, 84 to 94.  Four pieces of
// 16-bit rows, whose weights alone are 64 registers, spill 76 to 168 bytes a thread, and so do 40 two pieces with a gate of rows
// that start anywhere.
template <typename T, bool GATE, bool E4M3, bool ANYWHERE>
static cudaError_t dispatch_ring(const muon_block_norm_args& a, int sms, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = static_cast<int>((a.cols + E - 1) / E);
  if (pieces <= 16) return launch_ring<T, 16, 1, 8, 4, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 32) return launch_ring<T, 32, 1, 8, 4, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 64) return launch_ring<T, 32, 2, 5, 3, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 128) return launch_ring<T, 64, 2, 5, 3, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 256) return launch_ring<T, 128, 2, 5, 3, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 512) return launch_ring<T, 256, 2, 3, 2, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  if (pieces <= 1024) return launch_ring<T, 512, 2, 3, 1, 1, GATE, E4M3, ANYWHERE>(a, sms, st);
  // four pieces to a thread take the longest to compile: the general kernel serves e4m3 too
  if (pieces <= 2048) return launch_ring<T, 512, 4, 2, 1, 1, GATE, false, ANYWHERE>(a, sms, st);
  if (pieces <= 4096) return launch_ring<T, 512, 4, 2, 1, 2, GATE, false, ANYWHERE>(a, sms, st);
  return launch_ring<T, 512, 4, 2, 1, 4, GATE, false, ANYWHERE>(a, sms, st);
}

template <typename T, bool ANYWHERE>
cudaError_t launch_block_norm_rows(const muon_block_norm_args& a, int sms, cudaStream_t st) {
  // 4 CTAs of 2048 pieces hold MUON_MAX_DIM 16-bit columns and half as many of fp32
  if constexpr (sizeof(T) == 4) {
    if (a.cols > 4 * 2048 * 4) return launch_pdl(block_norm_wide_kernel<T>, dim3(static_cast<unsigned>(a.rows)), dim3(512), 0, st, a);
  }
  const bool element = a.gate && !a.gate_per_row, kept = a.x8.data && a.h8.data && (a.gate8.data || !element);
  const bool e4m3 = kept && a.kept_fmt == MUON_E4M3 && (!a.q.data || a.fmt == MUON_E4M3);
  const auto go = [&](auto gate) {
    constexpr bool GATE = decltype(gate)::value;
    return e4m3 ? dispatch_ring<T, GATE, true, ANYWHERE>(a, sms, st) : dispatch_ring<T, GATE, false, ANYWHERE>(a, sms, st);
  };
  return element ? go(std::true_type()) : go(std::false_type());
}
template cudaError_t launch_block_norm_rows<MUON_ROWS_T, MUON_ROWS_ANYWHERE>(const muon_block_norm_args&, int, cudaStream_t);

}  // namespace muon
