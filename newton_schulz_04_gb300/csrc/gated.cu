// gated.cu -- the product of an activation and a linear branch with 8-bit copies, and its gradient from them.
//
//   y = f(gate) up       f(g) = g / (1 + exp(-g)) (silu)  or  g Phi(g), Phi the normal distribution's function (gelu)
//   dgate = dy up f'(gate)       dup = dy f(gate)
//   f'(g) = s + f(g) (1 - s), s = 1 / (1 + exp(-g))       f'(g) = Phi(g) + g exp(-g^2 / 2) / sqrt(2 pi)
//
// Computed in fp32; every output is rounded once.
//
// The gradient's 8-bit operands are needed by rows (the products with the weights) and transposed (the weights'
// gradients, summed over the rows), and the weight behind y needs y transposed, computed again from what was kept.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block_norm.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace muon {

// Phi of a pair and exp(-g^2 / 2), for 16-bit data: erfc(z) = t R(t) exp(-z^2) with t = 1 / (1 + z / 2), the form of Press et
// al. (Numerical Recipes, erfcc), with R a polynomial fitted to 1.6e-7 of the value over all z >= 0.  Both tails keep their
// relative precision; the exponential's, (2 + 0.6 g^2) 2^-23, is the larger part.
struct Normal {
  float2 phi, bell;
};
__device__ __forceinline__ Normal normal2(float2 g) {
  const float2 a = make_float2(fabsf(g.x), fabsf(g.y));
  float2 bell = mul2(mul2(g, g), both(-0.5f * 1.4426950408889634f)), t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.x) : "f"(bell.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(bell.y) : "f"(bell.y));
  const float2 d = fma2(a, both(0.3535533905932738f), both(1.f));  // z = |g| / sqrt(2)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(d.y));
  constexpr float c[10] = {0.28209474704897347f, 0.2821042190368617f,  0.2465122105572134f,    0.1804148380537399f,
                           0.0582618433141641f,  0.07946854893160596f, -0.19854795364580055f,  0.030752471632890434f,
                           0.06446185801186056f, -0.02552294149528864f};
  float2 r = both(c[9]);
#pragma unroll
  for (int k = 8; k >= 0; --k) r = fma2(r, t, both(c[k]));
  const float2 tail = mul2(mul2(mul2(t, both(0.5f)), bell), r), rest = fma2(tail, both(-1.f), both(1.f));
  return {make_float2(g.x < 0.f ? tail.x : rest.x, g.y < 0.f ? tail.y : rest.y), bell};
}

template <typename T, bool GELU>
__device__ __forceinline__ float2 activation2(float2 g) {
  if constexpr (!GELU) return mul2(g, sigmoid2<T>(g));
  else if constexpr (sizeof(T) == 4) return make_float2(g.x * normcdff(g.x), g.y * normcdff(g.y));
  else return mul2(g, normal2(g).phi);
}
struct Activation {
  float2 value, slope;
};
template <typename T, bool GELU>
__device__ __forceinline__ Activation activate2(float2 g) {
  if constexpr (!GELU) {
    const float2 s = sigmoid2<T>(g), v = mul2(g, s);
    return {v, fma2(v, fma2(s, both(-1.f), both(1.f)), s)};
  } else {
    Normal n;
    if constexpr (sizeof(T) == 4)
      n = {make_float2(normcdff(g.x), normcdff(g.y)), make_float2(expf(-0.5f * g.x * g.x), expf(-0.5f * g.y * g.y))};
    else n = normal2(g);
    return {mul2(g, n.phi), fma2(mul2(g, both(0.3989422804014327f)), n.bell, n.phi)};
  }
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
// ------------------------------------------------------------------ forward
// Bound by memory and issuing: 8192 x 14336 bf16 with an 8-bit output and both checkpoints takes 142 us (5.8 TB/s, 32
// instructions an element); with a block to a warp, a column of it to a lane, 326.  gelu 53 us at 33.5M elements, silu 44, rows
// that start anywhere 59.
//
// A block of 128 columns to 16 lanes (32 in fp32), U rows to a lane, fetched together.  EIGHT: 8-bit outputs; 0: none, 1: any, 2:
// both checkpoints, and all of e4m3.  ANYWHERE: rows that do not start on 16 bytes.
constexpr int kGatedRows = 2;
template <typename T, bool GELU, int EIGHT, bool ANYWHERE>
__global__ void __launch_bounds__(256) gated_kernel(const muon_gated_args a) {
  using P = Pairs<T>;
  constexpr int E = P::E, N = P::N, LANES = 128 / E, GROUPS = 256 / LANES, U = kGatedRows;
  using Scales = Scales4<LANES, sizeof(T) == 2>;
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % LANES, kb = blockIdx.x, cols = static_cast<int>(a.cols), col = kb * 128 + t * E, left = cols - col;
  const long long group = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y, row0 = group * GROUPS * U + threadIdx.x / LANES;
  const T* gate = static_cast<const T*>(a.gate);
  const T* up = static_cast<const T*>(a.up);
  uint4 rg[U], ru[U];
  LoadAnywhere<T> lg[U], lu[U];
  if constexpr (ANYWHERE) {
    const Span sg = Span::of<T>(gate, a.rows, cols, a.ldg), su = Span::of<T>(up, a.rows, cols, a.ldu);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long row = row0 + u * GROUPS;
      const bool in = row < a.rows;
      lg[u].load(gate + (in ? row * a.ldg : 0), col / E, in ? left : 0, sg);
      lu[u].load(up + (in ? row * a.ldu : 0), col / E, in ? left : 0, su);
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
    if constexpr (ANYWHERE) rg[u] = lg[u].get(), ru[u] = lu[u].get();
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
static dim3 gated_grid(long long rows, long long cols) {
  constexpr int ROWS = 256 * 16 / static_cast<int>(sizeof(T)) / 128 * kGatedRows;  // of a CTA
  const long long groups = (rows + ROWS - 1) / ROWS, y = std::min(groups, 32768LL);
  return dim3(static_cast<unsigned>((cols + 127) / 128), static_cast<unsigned>(y), static_cast<unsigned>((groups + y - 1) / y));
}

template <typename T>
static cudaError_t dispatch_gated(const muon_gated_args& a, int vec, cudaStream_t st) {
  const dim3 grid = gated_grid<T>(a.rows, a.cols);
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
// A 128 x 128 tile to a CTA, 16 rows to each of its 8 warps, 4 neighbouring columns to a lane.  A warp copies its rows to shared
// memory in chunks of 4 and goes through them twice: for the gradients as they are, by rows, and the columns' largest
// magnitudes, which the CTA then joins; and, with the columns' scales, for the transposed bytes, which take the place of
// the chunk that they come from (a word of 4 rows for each column and output) and leave from there, 16 rows at a time.
// Computing everything twice costs a quarter of the instructions and saves the registers that three outputs of a tile
// would fill, so that three CTAs on an SM overlap one another's copies.  Bound by issuing: 8192 x 14336 bf16 from e4m3, e5m2
// both ways and the activation again, takes 272 us (58 % of the copy rate, 70 % of the issue slots, 65 instructions an
// element); one CTA of 512 threads with f and f' in registers took 715.
constexpr int kTile = 128, kTileWarps = 8, kChunkRows = 4, kChunks = kTile / kTileWarps / kChunkRows;

// Four neighbouring elements in shared memory.
__device__ __forceinline__ void four(const float* p, float2 (&v)[2]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = make_float2(f.x, f.y), v[1] = make_float2(f.z, f.w);
}
template <typename T>
__device__ __forceinline__ void four(const T* p, float2 (&v)[2]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = unpack2(w.x, T()), v[1] = unpack2(w.y, T());
}
template <bool E5M2>
__device__ __forceinline__ void four8(const uint8_t* p, float scale, float2 (&v)[2]) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  v[0] = mul2(fp8_unpack2<E5M2>(w), both(scale));
  v[1] = mul2(fp8_unpack2<E5M2>(w >> 16), both(scale));
}
__device__ __forceinline__ float largest3(float m, float a, float b) {
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}
template <bool E5M2>
__device__ __forceinline__ uint32_t pack_scaled(float2 a, float2 b, float inv) {
  a = mul2(a, both(inv)), b = mul2(b, both(inv));
  return fp8_pack4<E5M2>(a.x, a.y, b.x, b.y);
}
// Four elements of a lane's row, its neighbours' before and behind; rows that start anywhere.
template <typename T>
__device__ __forceinline__ void store_four_anywhere(T* row, int lane, long long left, const float2 (&v)[2]) {
  if constexpr (sizeof(T) == 4) {
    Pairs<T> p;
    p.v[0] = v[0], p.v[1] = v[1];
    store_anywhere<T, 32>(row, lane, static_cast<int>(max(-1LL << 30, min(1LL << 30, left))), p);
  } else {  // as store_anywhere, in pieces of 8 bytes
    union {
      uint32_t w[2];
      T e[4];
    } u;
    u.w[0] = pack2(v[0], T()), u.w[1] = pack2(v[1], T());
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 7), head = 4 - off / 2, bits = 64 - 8 * off;
    const uint32_t b0 = __shfl_up_sync(0xffffffffu, u.w[0], 1), b1 = __shfl_up_sync(0xffffffffu, u.w[1], 1);
    const bool whole = left >= head && (lane > 0 || off == 0);
    if (whole) {
      const unsigned long long before = b0 | static_cast<unsigned long long>(b1) << 32;
      const unsigned long long own = u.w[0] | static_cast<unsigned long long>(u.w[1]) << 32;
      *reinterpret_cast<unsigned long long*>(reinterpret_cast<uint8_t*>(row) - off + 8LL * lane) =
          off ? before >> bits | own << (64 - bits) : own;
    }
    const uint32_t first = (1u << head) - 1u, there = (1u << max(0LL, min(4LL, left))) - 1u;
    const uint32_t rest = there & ((whole ? 0u : first) | (lane == 31 || left - 4 < head ? ~first : 0u));
    if (rest) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (rest >> i & 1u) row[lane * 4 + i] = u.e[i];
    }
  }
}

// KEPT: of gate and up; 0: T, 1: e4m3, 2: e5m2.  ANYWHERE: rows of T that do not start on 16 bytes.
template <typename T, int KEPT, bool GELU, bool ANYWHERE>
struct GatedTile {
  using K = std::conditional_t<KEPT != 0, uint8_t, T>;
  static constexpr int DY = kTile * static_cast<int>(sizeof(T)), KEEP = kTile * static_cast<int>(sizeof(K));  // bytes of a row
  static constexpr int CHUNK = kChunkRows * (DY + 2 * KEEP), WARP = kChunks * CHUNK, BYTES = kTileWarps * WARP;
  static constexpr int CTAS = BYTES <= 72 * 1024 ? 3 : BYTES <= 108 * 1024 ? 2 : 1;  // on an SM
  static_assert(CHUNK >= 3 * 4 * 128, "a chunk's transposed words");
};

template <typename T, int KEPT, bool GELU, bool ANYWHERE>
__global__ void __launch_bounds__(kTileWarps * 32, GatedTile<T, KEPT, GELU, ANYWHERE>::CTAS)
    gated_grad_kernel(const muon_gated_grad_args a) {
  using G = GatedTile<T, KEPT, GELU, ANYWHERE>;
  using K = typename G::K;
  extern __shared__ __align__(16) uint8_t gated_smem[];
  __shared__ uint32_t cmax[3][kTile];  // of column 4 l + j at j * 32 + l; later the inverse scale
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint8_t* const mine = gated_smem + warp * G::WARP;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < 3 * kTile; i += kTileWarps * 32) cmax[0][i] = 0u;
  const long long kbc = blockIdx.x, kbr = blockIdx.y, rows = a.rows, cols = a.cols;
  const long long c00 = kbc * kTile, r0 = kbr * kTile + warp * (kTile / kTileWarps);
  const long long left = cols - c00;  // columns from the tile's first on
  pdl_wait();
  // ---- the warp's rows, a group of copies for each chunk
  const auto copy = [&](uint8_t* to, const auto* matrix, long long ld, auto anywhere) {  // one row after another
    using M = std::remove_const_t<std::remove_pointer_t<decltype(matrix)>>;
    constexpr int E = 16 / static_cast<int>(sizeof(M)), PER_ROW = kTile / E;
    return [=](int chunk) {
      LoadAnywhere<std::conditional_t<sizeof(M) == 1, __half, M>> loads[kChunkRows * PER_ROW / 32];  // of rows that start anywhere
#pragma unroll
      for (int k = 0; k < kChunkRows * PER_ROW / 32; ++k) {
        const int item = k * 32 + lane, r = item / PER_ROW, t = item % PER_ROW;
        const long long row = r0 + chunk * kChunkRows + r;
        const int n = row < rows ? static_cast<int>(max(0LL, min(static_cast<long long>(E), left - t * E))) : 0;
        uint8_t* dst = to + chunk * G::CHUNK + r * kTile * static_cast<int>(sizeof(M)) + t * 16;
        const M* src = matrix + (n ? row * ld + c00 + t * E : 0);
        if constexpr (decltype(anywhere)::value) {
          const Span all = Span::of<M>(matrix, rows, cols, ld);
          const int l = static_cast<int>(row < rows ? min(left - t * E, 1LL << 20) : 0LL);
          loads[k].load(matrix + (row < rows ? row * ld + c00 : 0), t, l, all);
        } else {
          copy16(smem_u32(dst), src, n * static_cast<int>(sizeof(M)));
        }
      }
      if constexpr (decltype(anywhere)::value) {
#pragma unroll
        for (int k = 0; k < kChunkRows * PER_ROW / 32; ++k) {
          const int item = k * 32 + lane;
          *reinterpret_cast<uint4*>(to + chunk * G::CHUNK + item / PER_ROW * kTile * static_cast<int>(sizeof(M)) + item % PER_ROW * 16) = loads[k].get();
        }
      }
    };
  };
  using Any = std::bool_constant<ANYWHERE>;
  const auto copy_dy = copy(mine, static_cast<const T*>(a.dy), a.lddy, Any());
  const auto copy_gate = copy(mine + kChunkRows * G::DY, static_cast<const K*>(a.gate), a.ldg, std::bool_constant<ANYWHERE && KEPT == 0>());
  const auto copy_up =
      copy(mine + kChunkRows * (G::DY + G::KEEP), static_cast<const K*>(a.up), a.ldu, std::bool_constant<ANYWHERE && KEPT == 0>());
#pragma unroll
  for (int chunk = 0; chunk < kChunks; ++chunk) {
    copy_dy(chunk), copy_gate(chunk), copy_up(chunk);
    cp_async_commit();
  }
  // the kept rows' scales: lane l has those of row l (gate) and row l - 16 (up)
  const long long rows4 = (rows + 3) & ~3LL;
  const int rows_here = static_cast<int>(max(0LL, min(16LL, rows - r0))), rows4_here = static_cast<int>(max(0LL, min(16LL, rows4 - r0)));
  uint32_t kept_scale = 127u;
  if (KEPT && lane % 16 < rows_here)
    kept_scale = static_cast<const uint8_t*>(lane < 16 ? a.gate_scale : a.up_scale)[fp8_scale_offset(kbc, r0 + lane % 16, rows4)];
  __shared__ float kept_values[kTileWarps][32];
  kept_values[warp][lane] = fp8_finite_scale_value<KEPT == 2>(kept_scale);
  const int n = static_cast<int>(max(0LL, min(4LL, left - lane * 4)));  // the lane's columns
  const long long col = c00 + lane * 4;
  const bool store8 = col < ((cols + 15) & ~15LL);
  const bool by_cols = a.dgate_cols.data || a.dup_cols.data || a.y_cols.data;
  // values of a row of a chunk, with the chunk's kept scales
  const auto load = [&](int chunk, int i, const float (&gs)[4], const float (&us)[4], float2 (&d)[2], float2 (&g)[2], float2 (&u)[2]) {
    const uint8_t* p = mine + chunk * G::CHUNK;
    four(reinterpret_cast<const T*>(p + i * G::DY) + lane * 4, d);
    const K* pg = reinterpret_cast<const K*>(p + kChunkRows * G::DY + i * G::KEEP) + lane * 4;
    const K* pu = reinterpret_cast<const K*>(p + kChunkRows * (G::DY + G::KEEP) + i * G::KEEP) + lane * 4;
    if constexpr (KEPT != 0) four8<KEPT == 2>(pg, gs[i], g), four8<KEPT == 2>(pu, us[i], u);
    else four(pg, g), four(pu, u);
  };
  const auto kept_of = [&](int at, float (&s)[4]) {
    if (KEPT) {
      const float4 f = *reinterpret_cast<const float4*>(&kept_values[warp][at]);
      s[0] = f.x, s[1] = f.y, s[2] = f.z, s[3] = f.w;
    }
  };
  float cm[3][4];
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[o][j] = 0.f;
  // the 8 scales of a chunk's rows (4 of dgate, 4 of dup): lane l keeps that of row l / 8 and output l / 4 % 2
  const int my_row = lane / 8, my_out = lane / 4 % 2, top = a.fmt ? 15 : 8;
  const muon_fp8_out& my_rows = my_out ? a.dup_rows : a.dgate_rows;
  uint8_t* const my_scales = lane % 4 == 0 ? static_cast<uint8_t*>(my_rows.scale) : nullptr;
  const bool by_rows = a.dgate_rows.data || a.dup_rows.data;
  uint8_t* rows_g = static_cast<uint8_t*>(a.dgate_rows.data) + r0 * a.dgate_rows.ld + col;
  uint8_t* rows_u = static_cast<uint8_t*>(a.dup_rows.data) + r0 * a.dup_rows.ld + col;
#pragma unroll 1
  for (int chunk = 0; chunk < kChunks; ++chunk) {
    if (chunk == 0) cp_async_wait<kChunks - 1>();
    else if (chunk == 1) cp_async_wait<kChunks - 2>();
    else if (chunk == 2) cp_async_wait<kChunks - 3>();
    else cp_async_wait<0>();
    __syncwarp();
    float2 dg[kChunkRows][2], du[kChunkRows][2], y_before[2];
    uint32_t m[kChunkRows];
    float gs[4], us[4];
    kept_of(chunk * kChunkRows, gs), kept_of(16 + chunk * kChunkRows, us);
#pragma unroll
    for (int r = 0; r < kChunkRows; ++r) {
      float2 d[2], g[2], u[2];
      load(chunk, r, gs, us, d, g, u);
      float mg = 0.f, mu = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Activation f = activate2<T, GELU>(g[i]);
        const float2 y = mul2(f.value, u[i]);
        dg[r][i] = mul2(mul2(d[i], u[i]), f.slope);
        du[r][i] = mul2(d[i], f.value);
        mg = largest3(mg, dg[r][i].x, dg[r][i].y);
        mu = largest3(mu, du[r][i].x, du[r][i].y);
        if (r % 2 == 0) {
          y_before[i] = y;
        } else {
          cm[2][2 * i] = largest3(cm[2][2 * i], y_before[i].x, y.x);
          cm[2][2 * i + 1] = largest3(cm[2][2 * i + 1], y_before[i].y, y.y);
        }
      }
      m[r] = upper_halves(__float_as_uint(mg), __float_as_uint(mu));
      if (r % 2 == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          cm[0][2 * i] = largest3(cm[0][2 * i], dg[r - 1][i].x, dg[r][i].x);
          cm[0][2 * i + 1] = largest3(cm[0][2 * i + 1], dg[r - 1][i].y, dg[r][i].y);
          cm[1][2 * i] = largest3(cm[1][2 * i], du[r - 1][i].x, du[r][i].x);
          cm[1][2 * i + 1] = largest3(cm[1][2 * i + 1], du[r - 1][i].y, du[r][i].y);
        }
      }
    }
    const long long row0 = r0 + chunk * kChunkRows;
    if (a.dgate || a.dup) {
#pragma unroll
      for (int r = 0; r < kChunkRows; ++r) {
        const bool in = row0 + r < rows;
        const auto put = [&](void* p, long long ld, const float2(&v)[2]) {
          T* to = static_cast<T*>(p) + (in ? (row0 + r) * ld + c00 : 0);
          if constexpr (ANYWHERE) {
            store_four_anywhere(to, lane, in ? left - lane * 4 : 0LL, v);
          } else if (in && n == 4) {
            if constexpr (sizeof(T) == 2) *reinterpret_cast<uint2*>(to + lane * 4) = make_uint2(pack2(v[0], T()), pack2(v[1], T()));
            else *reinterpret_cast<float4*>(to + lane * 4) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
          } else if (in) {
            if (n > 0) to[lane * 4] = from_f32<T>(v[0].x);
            if (n > 1) to[lane * 4 + 1] = from_f32<T>(v[0].y);
            if (n > 2) to[lane * 4 + 2] = from_f32<T>(v[1].x);
          }
        };
        if (a.dgate) put(a.dgate, a.lddgate, dg[r]);
        if (a.dup) put(a.dup, a.lddup, du[r]);
      }
    }
    if (by_rows) {
      // largest magnitudes over the row's lanes, four words of two shared out as they shrink: lane l ends with row l / 8
      const bool hi = lane & 16, odd = lane & 8;
      const uint32_t w0 = __vmaxu2(hi ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 16));
      const uint32_t w1 = __vmaxu2(hi ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], 16));
      uint32_t w = __vmaxu2(odd ? w1 : w0, __shfl_xor_sync(0xffffffffu, odd ? w0 : w1, 8));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, o));
      const uint32_t byte = chunk * kChunkRows + my_row < rows_here ? fp8_scale_byte(my_out ? w & 0xffff0000u : w << 16, top) : 127u;
      if (my_scales && chunk * kChunkRows + my_row < rows4_here) {
        my_scales[fp8_scale_offset(kbc, row0 + my_row, rows4)] = static_cast<uint8_t>(byte);
        if (left <= kTile)  // blocks past the last column, up to a whole scale word
          for (long long kb = kbc + 1; kb < (cols + 511) / 512 * 4; ++kb) my_scales[fp8_scale_offset(kb, row0 + my_row, rows4)] = 127;
      }
      const float my_inv = fp8_inverse_scale(byte);
      float ig[kChunkRows], iu[kChunkRows];
#pragma unroll
      for (int r = 0; r < kChunkRows; ++r) {
        ig[r] = __shfl_sync(0xffffffffu, my_inv, 8 * r);
        iu[r] = __shfl_sync(0xffffffffu, my_inv, 8 * r + 4);
      }
      uint8_t *pg = rows_g, *pu = rows_u;
      rows_g += kChunkRows * a.dgate_rows.ld, rows_u += kChunkRows * a.dup_rows.ld;
      const auto put = [&](auto e5m2) {
        constexpr bool E5M2 = decltype(e5m2)::value;
#pragma unroll
        for (int r = 0; r < kChunkRows; ++r) {
          const uint32_t wg = pack_scaled<E5M2>(dg[r][0], dg[r][1], ig[r]), wu = pack_scaled<E5M2>(du[r][0], du[r][1], iu[r]);
          const bool in = store8 && chunk * kChunkRows + r < rows_here;
          if (in && a.dgate_rows.data) *reinterpret_cast<uint32_t*>(pg) = wg;
          if (in && a.dup_rows.data) *reinterpret_cast<uint32_t*>(pu) = wu;
          pg += a.dgate_rows.ld, pu += a.dup_rows.ld;
        }
      };
      if (a.fmt) put(std::true_type());
      else put(std::false_type());
    }
  }
  if (!by_cols) return;
  __syncthreads();  // cmax is 0
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int j = 0; j < 4; ++j) atomicMax(&cmax[o][j * 32 + lane], __float_as_uint(cm[o][j]));
  __syncthreads();
  // ---- a scale for each column and output
  for (int i = threadIdx.x; i < 3 * kTile; i += kTileWarps * 32) {
    const int o = i / kTile, c = i % 32 * 4 + i % kTile / 32;  // the column
    const muon_fp8_out& out = o == 0 ? a.dgate_cols : o == 1 ? a.dup_cols : a.y_cols;
    const uint32_t byte = c < left ? fp8_scale_byte(cmax[0][i], (o < 2 ? a.fmt : a.y_fmt) ? 15 : 8) : 127u;
    cmax[0][i] = __float_as_uint(fp8_inverse_scale(byte));
    const long long cols4 = (cols + 3) & ~3LL;
    if (out.data && c00 + c < cols4) {
      uint8_t* s = static_cast<uint8_t*>(out.scale);
      s[fp8_scale_offset(kbr, c00 + c, cols4)] = static_cast<uint8_t>(byte);
      if ((kbr + 1) * kTile >= rows)
        for (long long kb = kbr + 1; kb < (rows + 511) / 512 * 4; ++kb) s[fp8_scale_offset(kb, c00 + c, cols4)] = 127;
    }
  }
  __syncthreads();
  float2 inv[3][2];
#pragma unroll
  for (int o = 0; o < 3; ++o)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      inv[o][i] = make_float2(__uint_as_float(cmax[o][2 * i * 32 + lane]), __uint_as_float(cmax[o][(2 * i + 1) * 32 + lane]));
  // ---- transposed words; lanes are turned by 4 for each warp, so that reading a column from 8 warps meets 8 banks
  const int turned = (lane + 4 * warp) % 32;
#pragma unroll 1
  for (int chunk = 0; chunk < kChunks; ++chunk) {
    float2 v[3][kChunkRows][2];
    float gs[4], us[4];
    kept_of(chunk * kChunkRows, gs), kept_of(16 + chunk * kChunkRows, us);
#pragma unroll
    for (int r = 0; r < kChunkRows; ++r) {
      float2 d[2], g[2], u[2];
      load(chunk, r, gs, us, d, g, u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Activation f = activate2<T, GELU>(g[i]);
        v[0][r][i] = mul2(mul2(mul2(d[i], u[i]), f.slope), inv[0][i]);
        v[1][r][i] = mul2(mul2(d[i], f.value), inv[1][i]);
        v[2][r][i] = mul2(mul2(f.value, u[i]), inv[2][i]);
      }
    }
    __syncwarp();  // the chunk has been read
    uint32_t* words = reinterpret_cast<uint32_t*>(mine + chunk * G::CHUNK);
    const auto put = [&](int o, auto e5m2) {
      constexpr bool E5M2 = decltype(e5m2)::value;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const auto at = [&](int r) { return j & 1 ? v[o][r][j / 2].y : v[o][r][j / 2].x; };
        words[(o * 4 + j) * 32 + turned] = fp8_pack4<E5M2>(at(0), at(1), at(2), at(3));
      }
    };
    if (a.fmt) put(0, std::true_type()), put(1, std::true_type());
    else put(0, std::false_type()), put(1, std::false_type());
    if (a.y_fmt) put(2, std::true_type());
    else put(2, std::false_type());
  }
  __syncthreads();
#pragma unroll
  for (int o = 0; o < 3; ++o) {
    const muon_fp8_out& out = o == 0 ? a.dgate_cols : o == 1 ? a.dup_cols : a.y_cols;
    if (!out.data) continue;
    // 16 bytes (the 16 rows of warp w) to a thread, 8 threads to a column; a warp has 4 columns
    const int w = threadIdx.x / 4 % 8, l4 = threadIdx.x % 4 + threadIdx.x / 32 * 4;
    const long long r = kbr * kTile + w * 16;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(gated_smem + w * G::WARP) + (l4 + 4 * w) % 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long c = c00 + l4 * 4 + j;
      if (c < cols && r < rows) {
        constexpr int STEP = G::CHUNK / 4;
        const int at = (o * 4 + j) * 32;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out.data) + c * out.ld + r) =
            make_uint4(words[at], words[STEP + at], words[2 * STEP + at], words[3 * STEP + at]);
      }
    }
  }
}

// ------------------------------------------------------------------ gradient of the data's type alone
// Without 8-bit outputs no block has to be gathered, and the forward kernel's layout gives small matrices more CTAs: 777 x 1101
// fp16 takes 7.3 us (22 in tiles), 8192 x 4096 bf16 51 (96 % of the copy rate).
template <typename T, int KEPT, bool GELU, bool ANYWHERE>
__global__ void __launch_bounds__(256) gated_grad_dense_kernel(const muon_gated_grad_args a) {
  using P = Pairs<T>;
  using K = std::conditional_t<KEPT != 0, uint8_t, T>;
  constexpr int E = P::E, N = P::N, LANES = 128 / E, GROUPS = 256 / LANES, U = kGatedRows;
  pdl_launch_dependents();
  pdl_wait();
  const int t = threadIdx.x % LANES, kb = blockIdx.x, cols = static_cast<int>(a.cols), col = kb * 128 + t * E, left = cols - col;
  const long long group = blockIdx.y + static_cast<long long>(blockIdx.z) * gridDim.y, row0 = group * GROUPS * U + threadIdx.x / LANES;
  const long long rows4 = (a.rows + 3) & ~3LL;
  P d[U], g[U], v[U];
  LoadAnywhere<T> ld[U], lg[U], lv[U];  // of rows that start anywhere
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + u * GROUPS;
    const bool in = row < a.rows;
    const auto plain = [&](P& p, LoadAnywhere<T>& l, const void* matrix, long long ld) {
      const T* m = static_cast<const T*>(matrix);
      if constexpr (ANYWHERE) {
        l.load(m + (in ? row * ld : 0), col / E, in ? left : 0, Span::of<T>(m, a.rows, cols, ld));
      } else {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (in && left >= E) w = *reinterpret_cast<const uint4*>(m + row * ld + col);
        else if (in && left > 0) w = load_part(m + row * ld + col, left);
        p.unpack(w);
      }
    };
    const auto kept = [&](P& p, LoadAnywhere<T>& l, const void* matrix, const void* scale, long long ld) {
      if constexpr (KEPT == 0) {
        plain(p, l, matrix, ld);
      } else {
        __align__(8) uint8_t b[E] = {};
        const uint8_t* q = static_cast<const uint8_t*>(matrix) + row * ld + col;
        float s = 1.f;
        if (in && left > 0) {
          s = fp8_finite_scale_value<KEPT == 2>(static_cast<const uint8_t*>(scale)[fp8_scale_offset(kb, row, rows4)]);
          if (left >= E) {
            if constexpr (E == 8) *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(q);
            else *reinterpret_cast<uint32_t*>(b) = *reinterpret_cast<const uint32_t*>(q);
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
              if (i < left) b[i] = q[i];
          }
        }
        p.template unpack8<KEPT == 2>(b);
#pragma unroll
        for (int i = 0; i < N; ++i) p.v[i] = mul2(p.v[i], both(s));
      }
    };
    plain(d[u], ld[u], a.dy, a.lddy);
    kept(g[u], lg[u], a.gate, a.gate_scale, a.ldg);
    kept(v[u], lv[u], a.up, a.up_scale, a.ldu);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = row0 + u * GROUPS;
    const bool in = row < a.rows;
    P dg, du;
    if constexpr (ANYWHERE) {
      d[u].unpack(ld[u].get());
      if constexpr (KEPT == 0) g[u].unpack(lg[u].get()), v[u].unpack(lv[u].get());
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Activation f = activate2<T, GELU>(g[u].v[i]);
      dg.v[i] = mul2(mul2(d[u].v[i], v[u].v[i]), f.slope);
      du.v[i] = mul2(d[u].v[i], f.value);
    }
    const auto put = [&](void* matrix, long long ld, const P& p) {
      T* m = static_cast<T*>(matrix);
      if constexpr (ANYWHERE) store_anywhere<T, LANES>(m + (in ? row * ld : 0), col / E, in ? left : 0, p);
      else if (in) p.store(m + row * ld + col, min(E, left));
    };
    if (a.dgate) put(a.dgate, a.lddgate, dg);
    if (a.dup) put(a.dup, a.lddup, du);
  }
}

template <typename T>
static cudaError_t dispatch_gated_grad(const muon_gated_grad_args& a, int vec, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + kTile - 1) / kTile), static_cast<unsigned>((a.rows + kTile - 1) / kTile));
  const bool eight = a.dgate_rows.data || a.dgate_cols.data || a.dup_rows.data || a.dup_cols.data || a.y_cols.data;
  const auto go = [&](auto kept, auto gelu, auto anywhere) {
    constexpr int KEPT = decltype(kept)::value;
    constexpr bool GELU = decltype(gelu)::value, ANYWHERE = decltype(anywhere)::value;
    if (!eight) return launch_pdl(gated_grad_dense_kernel<T, KEPT, GELU, ANYWHERE>, gated_grid<T>(a.rows, a.cols), dim3(256), 0, st, a);
    static bool done[64] = {false};
    constexpr int smem = GatedTile<T, KEPT, GELU, ANYWHERE>::BYTES;
    const auto kernel = gated_grad_kernel<T, KEPT, GELU, ANYWHERE>;
    const cudaError_t e = smem_limit(kernel, smem, done);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(kTileWarps * 32), smem, st, a);
  };
  const auto by_kept = [&](auto gelu, auto anywhere) {
    if (!a.gate_scale) return go(std::integral_constant<int, 0>(), gelu, anywhere);
    return a.kept_fmt ? go(std::integral_constant<int, 2>(), gelu, anywhere) : go(std::integral_constant<int, 1>(), gelu, anywhere);
  };
  const auto by_act = [&](auto anywhere) { return a.act ? by_kept(std::true_type(), anywhere) : by_kept(std::false_type(), anywhere); };
  return vec ? by_act(std::false_type()) : by_act(std::true_type());
}

cudaError_t launch_gated_grad(const muon_gated_grad_args& a, int vec, cudaStream_t st) {
  if (a.dt == MUON_BF16) return dispatch_gated_grad<__nv_bfloat16>(a, vec, st);
  return a.dt == MUON_FP16 ? dispatch_gated_grad<__half>(a, vec, st) : dispatch_gated_grad<float>(a, vec, st);
}

}  // namespace muon
