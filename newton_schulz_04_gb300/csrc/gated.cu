// gated.cu -- the product of an activation and a linear branch with 8-bit copies, and its gradient from them.
//
//   y = f(gate) up       f(g) = g / (1 + exp(-g)) (silu)  or  g Phi(g), Phi the normal distribution's function (gelu)
//   dgate = dy up f'(gate)       dup = dy f(gate)
//   f'(g) = s + f(g) (1 - s), s = 1 / (1 + exp(-g))       f'(g) = Phi(g) + g exp(-g^2 / 2) / sqrt(2 pi)
//
// Computed in fp32; every output is rounded once.
//
// The gradient's 8-bit operands are needed by rows (the products with the weights) and transposed (the weights'
// gradients, summed over the rows), and the weight behind y needs y transposed, computed again from what was kept.  A CTA
// takes a tile of 128 x 128, a warp 8 rows of it, a lane 4 columns: a row's largest magnitude is one reduction of a warp,
// and its bytes are written at once; the columns' are collected in shared memory, after which the transposed bytes are made
// from f and f' in registers and leave through shared memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block_norm.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace muon {

struct Activation {
  float value, slope;
};
template <typename T, bool GELU>
__device__ __forceinline__ float2 activation2(float2 g) {
  if (GELU) return make_float2(g.x * normcdff(g.x), g.y * normcdff(g.y));
  return mul2(g, sigmoid2<T>(g));
}
// The first n elements at p, the rest 0.
template <typename T>
__device__ __forceinline__ uint4 load_part(const T* p, int n) {
  union {
    uint4 w;
    T e[16 / sizeof(T)];
  } u;
  u.w = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i)
    if (i < n) u.e[i] = p[i];
  return u.w;
}
template <typename T, bool GELU>
__device__ __forceinline__ Activation activate(float g) {
  if (GELU) {
    const float phi = normcdff(g);
    return {g * phi, fmaf(g * 0.3989422804f, __expf(-0.5f * g * g), phi)};
  }
  const float s = sigmoid<T>(g), v = g * s;
  return {v, fmaf(v, 1.f - s, s)};
}

// ------------------------------------------------------------------ forward
// A block of 128 columns to 16 lanes (32 in fp32), U rows to a lane, fetched together.  EIGHT: 8-bit outputs; 0: none, 1: any, 2:
// both checkpoints, and all of e4m3.  ANYWHERE: rows that do not start on 16 bytes.
constexpr int kGatedRows = 2;
template <typename T, bool GELU, int EIGHT, bool ANYWHERE>
__global__ void __launch_bounds__(256) gated_kernel(const muon_gated_args a) {
  using P = Pairs<T>;
  constexpr int E = P::E, N = P::N, LANES = 128 / E, GROUPS = 256 / LANES, U = kGatedRows;
  using Scales = Scales4<LANES>;
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % LANES, kb = blockIdx.x, cols = static_cast<int>(a.cols), col = kb * 128 + t * E, left = cols - col;
  const long long group = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y, row0 = group * GROUPS * U + threadIdx.x / LANES;
  const T* gate = static_cast<const T*>(a.gate);
  const T* up = static_cast<const T*>(a.up);
  uint4 rg[U], ru[U];
  if constexpr (ANYWHERE) {
    const Span sg = Span::of<T>(gate, a.rows, cols, a.ldg), su = Span::of<T>(up, a.rows, cols, a.ldu);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = row0 + u * GROUPS;
      const bool in = row < a.rows;
      rg[u] = load_anywhere<T, LANES>(gate + (in ? row * a.ldg : 0), col / E, in ? left : 0, sg);
      ru[u] = load_anywhere<T, LANES>(up + (in ? row * a.ldu : 0), col / E, in ? left : 0, su);
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = row0 + u * GROUPS;
      rg[u] = ru[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < a.rows && left >= E) {
        rg[u] = *reinterpret_cast<const uint4*>(gate + row * a.ldg + col);
        ru[u] = *reinterpret_cast<const uint4*>(up + row * a.ldu + col);
      } else if (row < a.rows && left > 0) {
        rg[u] = load_part(gate + row * a.ldg + col, left);
        ru[u] = load_part(up + row * a.ldu + col, left);
      }
    }
  }
  const long long rows4 = (a.rows + 3) & ~3LL;
  const int mine = Scales::mine(), cols16 = (cols + 15) & ~15;
  const int top = (mine ? a.kept_fmt : a.fmt) ? 15 : 8;
  uint8_t* const scales = static_cast<uint8_t*>(mine == 0 ? a.q.scale : mine == 1 ? a.gate8.scale : mine == 2 ? a.up8.scale : nullptr);
  const bool keeper = scales && threadIdx.x % Scales::Q == 0;
  const int more = kb * 128 + 128 >= cols ? (cols + 511) / 512 * 4 - kb : 1;  // up to a whole scale word, in the last block
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + u * GROUPS;
    const bool live = row < a.rows;
    P g, v, y;
    g.unpack(rg[u]);
    v.unpack(ru[u]);
#pragma unroll
    for (int i = 0; i < N; ++i) y.v[i] = mul2(activation2<T, GELU>(g.v[i]), v.v[i]);
    if (a.y) {
      if constexpr (ANYWHERE) store_anywhere<T, LANES>(static_cast<T*>(a.y) + (live ? row * a.ldy : 0), col / E, live ? left : 0, y);
      else if (live) y.store(static_cast<T*>(a.y) + row * a.ldy + col, min(E, left));
    }
    if (EIGHT) {
      const uint32_t m[4] = {y.largest(), g.largest(), v.largest(), 0u};
      const Scales s(m, top);
      if (live && col < cols16) {
        if constexpr (EIGHT == 2) {
          if (a.q.data) y.template store8<false>(static_cast<uint8_t*>(a.q.data) + row * a.q.ld + col, s.inv[0]);
          g.template store8<false>(static_cast<uint8_t*>(a.gate8.data) + row * a.gate8.ld + col, s.inv[1]);
          v.template store8<false>(static_cast<uint8_t*>(a.up8.data) + row * a.up8.ld + col, s.inv[2]);
        } else {
          if (a.q.data) y.store8(static_cast<uint8_t*>(a.q.data) + row * a.q.ld + col, s.inv[0], a.fmt);
          if (a.gate8.data) g.store8(static_cast<uint8_t*>(a.gate8.data) + row * a.gate8.ld + col, s.inv[1], a.kept_fmt);
          if (a.up8.data) v.store8(static_cast<uint8_t*>(a.up8.data) + row * a.up8.ld + col, s.inv[2], a.kept_fmt);
        }
      }
      if (keeper) {  // scales of no block or row, up to whole words and to four rows, are 1
        if (row < rows4) scales[fp8_scale_offset(kb, row, rows4)] = static_cast<uint8_t>(live ? s.byte : 127u);
        if (more > 1 && row < rows4)
          for (int k = 1; k < more; ++k) scales[fp8_scale_offset(kb + k, row, rows4)] = 127;
      }
    }
  }
}

template <typename T>
static cudaError_t dispatch_gated(const muon_gated_args& a, int vec, cudaStream_t st) {
  constexpr int ROWS = 256 * 16 / static_cast<int>(sizeof(T)) / 128 * kGatedRows;  // of a CTA
  const long long groups = (a.rows + ROWS - 1) / ROWS;
  const long long y = std::min(groups, 32768LL);
  const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>(y), static_cast<unsigned>((groups + y - 1) / y));
  const bool any = a.q.data || a.gate8.data || a.up8.data;
  const bool e4m3 = a.gate8.data && a.up8.data && a.kept_fmt == MUON_E4M3 && (!a.q.data || a.fmt == MUON_E4M3);
  const auto go = [&](auto gelu, auto anywhere) {
    constexpr bool G = decltype(gelu)::value, A = decltype(anywhere)::value;
    if (!any) return launch_pdl(gated_kernel<T, G, 0, A>, grid, dim3(256), 0, st, a);
    return e4m3 ? launch_pdl(gated_kernel<T, G, 2, A>, grid, dim3(256), 0, st, a)
                : launch_pdl(gated_kernel<T, G, 1, A>, grid, dim3(256), 0, st, a);
  };
  const auto by_act = [&](auto anywhere) { return a.act ? go(std::true_type(), anywhere) : go(std::false_type(), anywhere); };
  return vec ? by_act(std::false_type()) : by_act(std::true_type());
}

cudaError_t launch_gated(const muon_gated_args& a, int vec, cudaStream_t st) {
  if (a.dt == MUON_BF16) return dispatch_gated<__nv_bfloat16>(a, vec, st);
  if (a.dt == MUON_FP16) return dispatch_gated<__half>(a, vec, st);
  return dispatch_gated<float>(a, vec, st);
}

// ------------------------------------------------------------------ gradient
// Four neighbouring elements of a row as they are in memory.
template <typename T>
struct Four {
  static constexpr int W = sizeof(T);  // 32-bit words
  uint32_t w[W];
  // n exist; `whole`: all four do, and the address allows one access
  __device__ __forceinline__ void load(const T* p, int n, bool whole) {
    if (whole) {
      if constexpr (W == 1) w[0] = *reinterpret_cast<const uint32_t*>(p);
      if constexpr (W == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        w[0] = x.x, w[1] = x.y;
      }
      if constexpr (W == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      }
    } else {
      union {
        T e[4];
        uint32_t u[W];
      } x;
#pragma unroll
      for (int i = 0; i < W; ++i) x.u[i] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) x.e[i] = p[i];
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = x.u[i];
    }
  }
};
__device__ __forceinline__ void values(const Four<float>& q, float, int, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(q.w[i]);
}
__device__ __forceinline__ void values(const Four<__nv_bfloat16>& q, float, int, float (&v)[4]) {
  v[0] = __uint_as_float(q.w[0] << 16), v[1] = __uint_as_float(q.w[0] & 0xffff0000u);
  v[2] = __uint_as_float(q.w[1] << 16), v[3] = __uint_as_float(q.w[1] & 0xffff0000u);
}
__device__ __forceinline__ void values(const Four<__half>& q, float, int, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q.w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void values(const Four<uint8_t>& q, float scale, int fmt, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = fp8_unpack2(q.w[0] >> (16 * i), fmt);
    v[2 * i] = f.x * scale, v[2 * i + 1] = f.y * scale;
  }
}

template <typename T>
__device__ __forceinline__ void store_four(T* p, int n, bool whole, const float (&v)[4]) {
  if (whole) {
    union {
      T e[4];
      uint2 two;
      uint4 four;
    } x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.e[i] = from_f32<T>(v[i]);
    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(p) = x.two;
    else *reinterpret_cast<uint4*>(p) = x.four;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

constexpr int kTile = 128, kTileWarps = 16, kTileRows = kTile / kTileWarps;

// A transposed 8-bit tile on its way out: 8 bytes (8 rows) to a slot, 16 slots to a column, swizzled so that both the
// writes (a lane has 4 neighbouring columns) and the reads are free of bank conflicts.
struct TransposedTile {
  uint2 slot[kTile][16];
  __device__ __forceinline__ uint2& at(int col, int s) { return slot[col][s ^ ((col >> 2) & 15)]; }
};

// Row-wise 8 bits of one row of the tile; a warp's lanes hold its 128 columns.  Returns nothing past the last row.
__device__ __forceinline__ void store_row8(const muon_fp8_out& o, int fmt, long long row, bool in, long long c0, long long cols,
                                           long long offset, const float (&v)[4]) {
  uint32_t m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
  m = __reduce_max_sync(0xffffffffu, m);
  const uint32_t byte = in ? fp8_scale_byte(m, fmt ? 15 : 8) : 127u;
  const float inv = fp8_inverse_scale(byte);
  if (in && c0 < ((cols + 15) & ~15LL))
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(o.data) + row * o.ld + c0) =
        fmt ? fp8_pack4<true>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv)
            : fp8_pack4<false>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  if (threadIdx.x % 32 == 0 && offset >= 0) static_cast<uint8_t*>(o.scale)[offset] = static_cast<uint8_t>(byte);
}

template <typename T, bool KEPT8, bool GELU>
__global__ void __launch_bounds__(kTileWarps * 32, 1) gated_grad_kernel(const muon_gated_grad_args a, const int vec) {
  using K = std::conditional_t<KEPT8, uint8_t, T>;
  extern __shared__ __align__(16) uint8_t gated_smem[];
  TransposedTile* tiles = reinterpret_cast<TransposedTile*>(gated_smem);  // dgate, dup, y
  __shared__ uint32_t cmax[3][kTile];  // [4 i + j] of the tile's columns at j * 32 + i
  pdl_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x < kTile) cmax[0][threadIdx.x] = cmax[1][threadIdx.x] = cmax[2][threadIdx.x] = 0u;
  __syncthreads();
  pdl_wait();
  const long long kbc = blockIdx.x, kbr = blockIdx.y, rows = a.rows, cols = a.cols;
  const long long c0 = kbc * kTile + lane * 4, r0 = kbr * kTile + warp * kTileRows, rows4 = (rows + 3) & ~3LL;
  const int nc = static_cast<int>(max(0LL, min(4LL, cols - c0)));
  const bool last = (kbc + 1) * kTile >= cols;
  const int more = static_cast<int>((cols + 511) / 512 * 4 - kbc - 1);  // blocks up to a whole scale word, in the last tile
  Four<T> dy[kTileRows];
  Four<K> up[kTileRows], gate[kTileRows];
  float gs[kTileRows], us[kTileRows];
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    const long long row = r0 + i;
    const bool in = row < rows;
    const int n = in ? nc : 0;
    dy[i].load(static_cast<const T*>(a.dy) + (n ? row * a.lddy + c0 : 0), n, n == 4 && vec);
    gate[i].load(static_cast<const K*>(a.gate) + (n ? row * a.ldg + c0 : 0), n, n == 4 && (KEPT8 || vec));
    up[i].load(static_cast<const K*>(a.up) + (n ? row * a.ldu + c0 : 0), n, n == 4 && (KEPT8 || vec));
    gs[i] = us[i] = 1.f;
    if (KEPT8 && in) {
      const long long o = fp8_scale_offset(kbc, row, rows4);
      gs[i] = fp8_scale_value(static_cast<const uint8_t*>(a.gate_scale)[o]);
      us[i] = fp8_scale_value(static_cast<const uint8_t*>(a.up_scale)[o]);
    }
  }
  float value[kTileRows][4], slope[kTileRows][4];
  uint32_t cm[3][4];
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[o][j] = 0u;
#pragma unroll
  for (int i = 0; i < kTileRows; ++i) {
    const long long row = r0 + i;
    const bool in = row < rows;
    float d[4], g[4], u[4], dg[4], du[4];
    values(dy[i], 1.f, 0, d);
    values(gate[i], gs[i], a.kept_fmt, g);
    values(up[i], us[i], a.kept_fmt, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= nc) g[j] = u[j] = 0.f;  // a NaN scale
      const Activation f = activate<T, GELU>(g[j]);
      value[i][j] = f.value, slope[i][j] = f.slope;
      dg[j] = d[j] * u[j] * f.slope;
      du[j] = d[j] * f.value;
      cm[0][j] = max(cm[0][j], abs_bits(dg[j]));
      cm[1][j] = max(cm[1][j], abs_bits(du[j]));
      cm[2][j] = max(cm[2][j], abs_bits(f.value * u[j]));
    }
    if (a.dgate && in) store_four(static_cast<T*>(a.dgate) + row * a.lddgate + c0, nc, nc == 4 && vec, dg);
    if (a.dup && in) store_four(static_cast<T*>(a.dup) + row * a.lddup + c0, nc, nc == 4 && vec, du);
    const long long offset = row < rows4 ? fp8_scale_offset(kbc, row, rows4) : -1;
    if (a.dgate_rows.data) store_row8(a.dgate_rows, a.fmt, row, in, c0, cols, offset, dg);
    if (a.dup_rows.data) store_row8(a.dup_rows, a.fmt, row, in, c0, cols, offset, du);
    if (last && offset >= 0 && lane < more) {
      if (a.dgate_rows.data) static_cast<uint8_t*>(a.dgate_rows.scale)[fp8_scale_offset(kbc + 1 + lane, row, rows4)] = 127;
      if (a.dup_rows.data) static_cast<uint8_t*>(a.dup_rows.scale)[fp8_scale_offset(kbc + 1 + lane, row, rows4)] = 127;
    }
  }
  if (!a.dgate_cols.data && !a.dup_cols.data && !a.y_cols.data) return;
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) atomicMax(&cmax[o][j * 32 + lane], cm[o][j]);
  __syncthreads();
  const long long cols4 = (cols + 3) & ~3LL, kend = (rows + 511) / 512 * 4;
  const bool bottom = (kbr + 1) * kTile >= rows;
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    const muon_fp8_out& out = o == 0 ? a.dgate_cols : o == 1 ? a.dup_cols : a.y_cols;
    if (!out.data) continue;
    const int fmt = o < 2 ? a.fmt : a.y_fmt;
    float inv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t byte = j < nc ? fp8_scale_byte(cmax[o][j * 32 + lane], fmt ? 15 : 8) : 127u;
      inv[j] = fp8_inverse_scale(byte);
      if (warp == 0 && c0 + j < cols4) {
        static_cast<uint8_t*>(out.scale)[fp8_scale_offset(kbr, c0 + j, cols4)] = static_cast<uint8_t>(byte);
        if (bottom)
          for (long long kb = kbr + 1; kb < kend; ++kb) static_cast<uint8_t*>(out.scale)[fp8_scale_offset(kb, c0 + j, cols4)] = 127;
      }
    }
    uint32_t bytes[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = 4 * h + k;
        float d[4], u[4];
        if (o < 2) values(dy[i], 1.f, 0, d);
        if (o != 1) values(up[i], us[i], a.kept_fmt, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (o != 1 && j >= nc) u[j] = 0.f;
          v[k][j] = (o == 0 ? d[j] * u[j] * slope[i][j] : o == 1 ? d[j] * value[i][j] : value[i][j] * u[j]) * inv[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bytes[h][j] = fmt ? fp8_pack4<true>(v[0][j], v[1][j], v[2][j], v[3][j]) : fp8_pack4<false>(v[0][j], v[1][j], v[2][j], v[3][j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) tiles[o].at(lane * 4 + j, warp) = make_uint2(bytes[0][j], bytes[1][j]);
  }
  __syncthreads();
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    const muon_fp8_out& out = o == 0 ? a.dgate_cols : o == 1 ? a.dup_cols : a.y_cols;
    if (!out.data) continue;
#pragma unroll
    for (int it = 0; it < 2; ++it) {  // 16 bytes per thread, 8 threads to a column; a warp's 4 columns are 4 apart
      const int q = it * 64 + (threadIdx.x >> 3), cl = (q % 32) * 4 + q / 32, s = (threadIdx.x & 7) * 2;
      const long long c = kbc * kTile + cl, r = kbr * kTile + s * 8;
      if (c < cols && r < rows) {
        const uint2 lo = tiles[o].at(cl, s), hi = tiles[o].at(cl, s + 1);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out.data) + c * out.ld + r) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

template <typename T, bool KEPT8>
static cudaError_t dispatch_gated_grad(const muon_gated_grad_args& a, int vec, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + kTile - 1) / kTile), static_cast<unsigned>((a.rows + kTile - 1) / kTile));
  constexpr int smem = 3 * static_cast<int>(sizeof(TransposedTile));
  const auto go = [&](auto kernel, bool (&done)[64]) {
    const cudaError_t e = smem_limit(kernel, smem, done);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(kTileWarps * 32), smem, st, a, vec);
  };
  static bool silu[64] = {false}, gelu[64] = {false};
  return a.act ? go(gated_grad_kernel<T, KEPT8, true>, gelu) : go(gated_grad_kernel<T, KEPT8, false>, silu);
}

cudaError_t launch_gated_grad(const muon_gated_grad_args& a, int vec, cudaStream_t st) {
  const auto go = [&](auto t) {
    using T = decltype(t);
    return a.gate_scale ? dispatch_gated_grad<T, true>(a, vec, st) : dispatch_gated_grad<T, false>(a, vec, st);
  };
  if (a.dt == MUON_BF16) return go(__nv_bfloat16());
  return a.dt == MUON_FP16 ? go(__half()) : go(float());
}

}  // namespace muon
