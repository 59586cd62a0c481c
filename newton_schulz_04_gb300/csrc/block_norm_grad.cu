// block_norm_grad.cu -- gradient of the norms around a block, from what the forward pass kept (of the data's type, or in 8
// bits).  With X = x rho_x and H = h rho_h as kept and c = scale post:
//
//   a = dy pre       D = dh + rho_h (a - H mean(a H))       dresidual = alpha D
//   b = D sigmoid(gate) c       dx = rho_x (b - X mean(b X))       dgate = (1 - sigmoid(gate)) b X
//   dpre = sum_rows dy H       S = sum_rows D sigmoid(gate) X       dpost = S scale       dscale = S post
//
// mean(b X) needs mean(a H) first.  With u = dh + rho_h a and e = sigmoid(gate) c X it is mean(u e) - rho_h mean(a H)
// mean(H e), so a row takes one pass and one exchange of three sums.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "block_norm.cuh"
#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace muon {

// A kept matrix: T, or 8 bits.
template <typename T, bool KEPT8>
struct Kept {
  const uint8_t* data;
  const uint8_t* scale;  // this row's first scale
  long long rows4;
  int fmt;
  __device__ __forceinline__ Kept(const void* p, const void* s, long long ld, long long row, long long rows, int fmt_)
      : data(static_cast<const uint8_t*>(p) + (p ? row * ld * (KEPT8 ? 1 : static_cast<long long>(sizeof(T))) : 0)),
        scale(static_cast<const uint8_t*>(s) + (KEPT8 && p ? row * 4 : 0)),
        rows4((rows + 3) & ~3LL),
        fmt(fmt_) {}
  __device__ __forceinline__ float block_scale(int kb) const {
    return KEPT8 ? fp8_scale_value(scale[(kb >> 2) * rows4 * 4 + (kb & 3)]) : 1.f;
  }
  __device__ __forceinline__ float at(int col, float block) const {
    if constexpr (KEPT8) return fp8_unpack2(data[col], fmt).x * block;
    else return to_f32(reinterpret_cast<const T*>(data)[col]);
  }
};

template <typename T, int W, int K, bool KEPT8>
__global__ void __launch_bounds__(W * 32) block_norm_grad_kernel(const muon_block_norm_grad_args a, float* partial) {
  constexpr int KK = K ? K : 1;
  __shared__ float sh[2][3][W];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cols = static_cast<int>(a.cols);
  const int blocks = (cols + 127) / 128, turns = K ? K : (blocks + W - 1) / W;
  float* part = partial ? partial + static_cast<long long>(blockIdx.x) * 2 * cols : nullptr;
  float dpre[KK][4], sx[KK][4];
#pragma unroll
  for (int k = 0; k < KK; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dpre[k][j] = sx[k][j] = 0.f;
  const float inv_n = 1.f / static_cast<float>(cols);
  int turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* dh = static_cast<const T*>(a.dh) + (a.dh ? row * a.lddh : 0);
    const Kept<T, KEPT8> kx(a.x, a.x_scale, a.ldx, row, a.rows, a.kept_fmt), kh(a.h, a.h_scale, a.ldh, row, a.rows, a.kept_fmt);
    const bool element = a.gate && !a.gate_per_row;
    const Kept<T, KEPT8> kg(element ? a.gate : nullptr, a.gate_scale, a.ldg, row, a.rows, a.kept_fmt);
    const float rx = a.rstd_x[row], rh = a.rstd_h[row];
    const float row_sig = a.gate && !element ? sigmoid<T>(to_f32(static_cast<const T*>(a.gate)[row * a.ldg])) : 1.f;
    struct Element {
      float d, u, hn, xn, sig, c;  // dy, dh + rho_h dy pre, H, X, sigmoid(gate), scale post
    };
    auto load = [&](int col, float xs, float hs, float gs) {
      Element e;
      e.d = to_f32(dy[col]);
      e.hn = kh.at(col, hs) * rh;
      e.xn = kx.at(col, xs) * rx;
      e.sig = element ? sigmoid<T>(kg.at(col, gs)) : row_sig;
      e.c = load_weight(a.post, a.weight_dt, col, true) * load_weight(a.scale, a.weight_dt, col, true);
      e.u = fmaf(rh, e.d * load_weight(a.pre, a.weight_dt, col, true), a.dh ? to_f32(dh[col]) : 0.f);
      return e;
    };
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < turns; ++k) {
      const int kb = warp + W * k;
      if (kb >= blocks) break;
      const float xs = kx.block_scale(kb), hs = kh.block_scale(kb), gs = element ? kg.block_scale(kb) : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = kb * 128 + lane + 32 * j;
        if (col >= cols) break;
        const Element e = load(col, xs, hs, gs);
        const float f = e.sig * e.c * e.xn;
        sum[0] = fmaf(e.d * load_weight(a.pre, a.weight_dt, col, true), e.hn, sum[0]);
        sum[1] = fmaf(e.u, f, sum[1]);
        sum[2] = fmaf(e.hn, f, sum[2]);
      }
    }
    cta_sums<W, 3>(sum, sh, turn);
    const float k1 = sum[0] * inv_n * rh, along = sum[1] - k1 * sum[2], k2 = along * inv_n;
    if (threadIdx.x == 0 && a.dgate && !element) static_cast<T*>(a.dgate)[row * a.lddgate] = from_f32<T>((1.f - row_sig) * along);
#pragma unroll
    for (int k = 0; k < turns; ++k) {
      const int kb = warp + W * k, kk = K ? k : 0;
      if (kb >= blocks) break;
      const float xs = kx.block_scale(kb), hs = kh.block_scale(kb), gs = element ? kg.block_scale(kb) : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = kb * 128 + lane + 32 * j;
        if (col >= cols) break;
        const Element e = load(col, xs, hs, gs);
        const float d = e.u - k1 * e.hn, t = d * e.sig, b = t * e.c;
        if (a.dresidual) static_cast<T*>(a.dresidual)[row * a.lddr + col] = from_f32<T>(a.alpha * d);
        if (a.dx) static_cast<T*>(a.dx)[row * a.lddx + col] = from_f32<T>(rx * (b - e.xn * k2));
        if (a.dgate && element) static_cast<T*>(a.dgate)[row * a.lddgate + col] = from_f32<T>((1.f - e.sig) * (b * e.xn));
        if (K) {
          dpre[kk][j] = fmaf(e.d, e.hn, dpre[kk][j]);
          sx[kk][j] = fmaf(t, e.xn, sx[kk][j]);
        } else if (part) {  // this thread alone holds these columns of the CTA's sums
          part[col] = (turn ? part[col] : 0.f) + e.d * e.hn;
          part[cols + col] = (turn ? part[cols + col] : 0.f) + t * e.xn;
        }
      }
    }
  }
  if (!K || !part) return;
#pragma unroll
  for (int k = 0; k < KK; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = (warp + W * k) * 128 + lane + 32 * j;
      if (col < cols) part[col] = dpre[k][j], part[cols + col] = sx[k][j];
    }
}

// ------------------------------------------------------------------ ring of rows
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, int bytes) {  // the rest is zero
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "n"(BYTES), "r"(bytes)
               : "memory");
}

// A thread's slots: S rows of dy, dh, x, h and gate, C pieces each; kept 8-bit ones take E bytes a piece instead of 16.
template <typename T, int TH, int C, int S, bool KEPT8>
struct GradRing {
  static constexpr int E = 16 / static_cast<int>(sizeof(T)), WIDE = KEPT8 ? 2 : 5;
  static constexpr int STAGE = TH * C * (WIDE * 16 + (5 - WIDE) * E), BYTES = S * STAGE;
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int slot, int arr, int c) const {
    uint8_t* stage = base + slot * STAGE;
    if (arr < WIDE) return stage + ((arr * C + c) * TH + static_cast<int>(threadIdx.x)) * 16;
    return stage + WIDE * C * TH * 16 + (((arr - WIDE) * C + c) * TH + static_cast<int>(threadIdx.x)) * E;
  }
  // n of the piece's elements exist.
  __device__ __forceinline__ void fetch(int slot, int arr, int c, const void* src, int n) const {
    if (arr < WIDE) copy16(smem_u32(at(slot, arr, c)), src, n * static_cast<int>(sizeof(T)));
    else copy_small<E>(smem_u32(at(slot, arr, c)), src, n);
  }
  __device__ __forceinline__ void read(int slot, int arr, int c, int fmt, Pairs<T>& p) const {
    if (arr < WIDE) p.unpack(*reinterpret_cast<const uint4*>(at(slot, arr, c)));
    else if (fmt) p.template unpack8<true>(at(slot, arr, c));
    else p.template unpack8<false>(at(slot, arr, c));
  }
};

template <typename T, int G, int C, int S, int MINB, int CL, bool KEPT8>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB)
    block_norm_grad_ring_kernel(const muon_block_norm_grad_args a, float* partial) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int DY = 0, DH = 1, X = 2, H = 3, GATE = 4;
  using P = Pairs<T>;
  using K = std::conditional_t<KEPT8, uint8_t, T>;
  constexpr int E = P::E, N = P::N, PIECE = G * E;  // PIECE: from a thread's piece to its next
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ RowSums<G, TH, 3, CL> sums;
  const GradRing<T, TH, C, S, KEPT8> ring{ring_smem};
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int t = threadIdx.x % G, rr = threadIdx.x / G, cols = static_cast<int>(a.cols);
  const int col = (rank * C * G + t) * E;  // of the first piece
  int n[C];                                // existing columns of each
#pragma unroll
  for (int c = 0; c < C; ++c) n[c] = max(0, min(E, cols - col - c * PIECE));
  const bool element = a.gate && !a.gate_per_row;
  const long long step = static_cast<long long>(gridDim.x / CL) * R, row0 = static_cast<long long>(blockIdx.x / CL) * R + rr;
  const long long rows4 = (a.rows + 3) & ~3LL;
  long long frow = row0;  // next row to fetch
  const T* fdy = static_cast<const T*>(a.dy) + row0 * a.lddy + col;
  const T* fdh = static_cast<const T*>(a.dh) + (a.dh ? row0 * a.lddh + col : 0);
  const K* fx = static_cast<const K*>(a.x) + row0 * a.ldx + col;
  const K* fh = static_cast<const K*>(a.h) + row0 * a.ldh + col;
  const K* fg = static_cast<const K*>(a.gate) + (element ? row0 * a.ldg + col : 0);
  auto fetch = [&](int slot) {
    if (frow < a.rows) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int at = n[c] ? c * PIECE : -col;
        ring.fetch(slot, DY, c, fdy + at, n[c]);
        if (a.dh) ring.fetch(slot, DH, c, fdh + at, n[c]);
        ring.fetch(slot, X, c, fx + at, n[c]);
        ring.fetch(slot, H, c, fh + at, n[c]);
        if (element) ring.fetch(slot, GATE, c, fg + at, n[c]);
      }
    }
    cp_async_commit();
    frow += step, fdy += step * a.lddy, fx += step * a.ldx, fh += step * a.ldh;
    if (a.dh) fdh += step * a.lddh;
    if (element) fg += step * a.ldg;
  };
  if (CL > 1) cluster_sync();  // the others' shared memory is there
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float2 w1[C][N], w2[C][N], dpre[C][N], sx[C][N];  // scale post, pre, and the columns' sums
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int at = n[c] ? col + c * PIECE : 0;
    float v[E], s[E];
    load_weight_piece<E>(a.scale, a.weight_dt, at, n[c], s);
    load_weight_piece<E>(a.post, a.weight_dt, at, n[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) w1[c][i] = make_float2(v[2 * i] * s[2 * i], v[2 * i + 1] * s[2 * i + 1]);
    load_weight_piece<E>(a.pre, a.weight_dt, at, n[c], v);
#pragma unroll
    for (int i = 0; i < N; ++i) w2[c][i] = make_float2(v[2 * i], v[2 * i + 1]), dpre[c][i] = sx[c][i] = both(0.f);
  }
  // of a row: the norms' factors, its gate, the scales of the kept pieces; fetched a row ahead
  struct RowHead {
    float rx, rh, gate;
    uint32_t xs[C], hs[C], gs[C];
  };
  const auto head = [&](long long row) {
    RowHead r = {};
    if (row < a.rows) {
      r.rx = __ldg(a.rstd_x + row);
      r.rh = __ldg(a.rstd_h + row);
      if (a.gate && !element) r.gate = to_f32(static_cast<const T*>(a.gate)[row * a.ldg]);
      if (KEPT8) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const long long o = fp8_scale_offset(n[c] ? (col + c * PIECE) / 128 : 0, row, rows4);
          r.xs[c] = __ldg(static_cast<const uint8_t*>(a.x_scale) + o);
          r.hs[c] = __ldg(static_cast<const uint8_t*>(a.h_scale) + o);
          if (element) r.gs[c] = __ldg(static_cast<const uint8_t*>(a.gate_scale) + o);
        }
      }
    }
    return r;
  };
  RowHead next = head(row0);
  const float inv_cols = 1.f / static_cast<float>(cols);
  T* pdr = static_cast<T*>(a.dresidual) + row0 * a.lddr + col;
  T* pdx = static_cast<T*>(a.dx) + row0 * a.lddx + col;
  T* pdg = static_cast<T*>(a.dgate) + (element ? row0 * a.lddgate + col : 0);
  int slot = 0, turn = 0;
  for (long long row = row0; row - rr < a.rows; row += step, ++turn) {
    const bool live = R == 1 || row < a.rows;
    if (row - rr + step >= a.rows) pdl_launch_dependents();  // the last row, as in the forward kernel
    const RowHead now = next;
    next = head(row + step);
    const float row_sig = a.gate && !element ? sigmoid2<T>(both(now.gate)).x : 1.f;
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    P u[C], sig[C], xn[C], hn[C];
    float2 s0 = both(0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      P d;
      ring.read(slot, DY, c, a.kept_fmt, d);
      ring.read(slot, X, c, a.kept_fmt, xn[c]);
      ring.read(slot, H, c, a.kept_fmt, hn[c]);
      if (a.dh) {
        ring.read(slot, DH, c, a.kept_fmt, u[c]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) u[c].v[i] = both(0.f);
      }
      if (element) ring.read(slot, GATE, c, a.kept_fmt, sig[c]);
      if (R > 1 && !live) {  // the slot holds another row's remains
#pragma unroll
        for (int i = 0; i < N; ++i) d.v[i] = xn[c].v[i] = hn[c].v[i] = u[c].v[i] = sig[c].v[i] = both(0.f);
      }
      const float2 xf = both(KEPT8 ? now.rx * fp8_scale_value(now.xs[c]) : now.rx);
      const float2 hf = both(KEPT8 ? now.rh * fp8_scale_value(now.hs[c]) : now.rh);
      const float2 gf = both(KEPT8 ? fp8_scale_value(now.gs[c]) : 1.f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        hn[c].v[i] = mul2(hn[c].v[i], hf);
        xn[c].v[i] = mul2(xn[c].v[i], xf);
        const float2 ad = mul2(d.v[i], w2[c][i]);
        u[c].v[i] = fma2(both(now.rh), ad, u[c].v[i]);
        sig[c].v[i] = element ? sigmoid2<T>(KEPT8 ? mul2(sig[c].v[i], gf) : sig[c].v[i]) : both(row_sig);
        const float2 e = mul2(mul2(sig[c].v[i], w1[c][i]), xn[c].v[i]);
        s0 = fma2(ad, hn[c].v[i], s0);
        s1 = fma2(u[c].v[i], e, s1);
        s2 = fma2(hn[c].v[i], e, s2);
        dpre[c][i] = fma2(d.v[i], hn[c].v[i], dpre[c][i]);
      }
    }
    float sum[3] = {total(s0), total(s1), total(s2)};
    sums(sum, turn);
    const float k1 = sum[0] * inv_cols * now.rh, along = sum[1] - k1 * sum[2], k2 = along * inv_cols;
    if (live && a.dgate && !element && t == 0 && rank == 0)
      static_cast<T*>(a.dgate)[row * a.lddgate] = from_f32<T>((1.f - row_sig) * along);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      P dr, dx, dg;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 d = fma2(both(-k1), hn[c].v[i], u[c].v[i]), td = mul2(d, sig[c].v[i]), b = mul2(td, w1[c][i]);
        sx[c][i] = fma2(td, xn[c].v[i], sx[c][i]);
        dr.v[i] = mul2(both(a.alpha), d);
        dx.v[i] = mul2(both(now.rx), fma2(both(-k2), xn[c].v[i], b));
        dg.v[i] = mul2(fma2(both(-1.f), sig[c].v[i], both(1.f)), mul2(b, xn[c].v[i]));
      }
      if (live) {
        if (a.dresidual) dr.store(pdr + c * PIECE, n[c]);
        if (a.dx) dx.store(pdx + c * PIECE, n[c]);
        if (element && a.dgate) dg.store(pdg + c * PIECE, n[c]);
      }
    }
    pdr += step * a.lddr, pdx += step * a.lddx;
    if (element) pdg += step * a.lddgate;
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  if (!partial) return;
  float* part = partial + static_cast<long long>(blockIdx.x / CL) * 2 * cols;
  if (R > 1) {  // join the CTA's row groups through the ring's memory
    static_assert(R == 1 || (R - 1) * 2 * C * N * G * 8 <= GradRing<T, TH, C, S, KEPT8>::BYTES, "room to join");
    cp_async_wait<0>();
    __syncthreads();
    float2* all = reinterpret_cast<float2*>(ring_smem);  // [R - 1][2][C * N][G]
    if (rr > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          all[(((rr - 1) * 2 + 0) * C * N + c * N + i) * G + t] = dpre[c][i];
          all[(((rr - 1) * 2 + 1) * C * N + c * N + i) * G + t] = sx[c][i];
        }
    }
    __syncthreads();
    if (rr > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < N; ++i)
        for (int r = 1; r < R; ++r) {
          dpre[c][i] = add2(dpre[c][i], all[(((r - 1) * 2 + 0) * C * N + c * N + i) * G + t]);
          sx[c][i] = add2(sx[c][i], all[(((r - 1) * 2 + 1) * C * N + c * N + i) * G + t]);
        }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float* p = part + col + c * PIECE + 2 * i;
      if (2 * i < n[c]) p[0] = dpre[c][i].x, p[cols] = sx[c][i].x;
      if (2 * i + 1 < n[c]) p[1] = dpre[c][i].y, p[cols + 1] = sx[c][i].y;
    }
}

// Sums over the CTAs' rows in a fixed order, 32 columns by 32 row groups per CTA; blockIdx.y 0: dpre, 1: dpost and dscale.
__global__ void __launch_bounds__(1024) block_norm_weights_kernel(const float* partial, int ctas,
                                                                  const muon_block_norm_grad_args a) {
  __shared__ float sh[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, cols = static_cast<int>(a.cols);
  int col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int r = g; r < ctas; r += 32) s += partial[(static_cast<long long>(r) * 2 + blockIdx.y) * cols + col];
  }
  sh[g][lane] = s;
  __syncthreads();
  pdl_launch_dependents();  // not before: a persistent grid that starts beside these CTAs finds no room for all of its own
  s = sh[lane][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  col = blockIdx.x * 32 + g;
  if (lane != 0 || col >= cols) return;
  if (blockIdx.y == 0) {
    if (a.dpre) a.dpre[col] = s;
  } else {
    if (a.dpost) a.dpost[col] = s * load_weight(a.scale, a.weight_dt, col, true);
    if (a.dscale) a.dscale[col] = s * load_weight(a.post, a.weight_dt, col, true);
  }
}

// The kernels add up rows of `partial` for at most this many CTAs (or clusters).
static int most_ctas(int sms) { return kBlockNormCtasPerSm * sms; }
int block_norm_grad_ctas(long long rows, int sms) {
  return static_cast<int>(std::max(1LL, std::min<long long>(rows, most_ctas(sms))));
}

template <typename T, bool KEPT8>
static cudaError_t dispatch_grad(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  *ctas = static_cast<int>(std::min<long long>(a.rows, 2 * sms));
  const auto go = [&](auto kernel, int warps) { return launch_pdl(kernel, dim3(*ctas), dim3(warps * 32), 0, st, a, partial); };
  if (a.cols <= 512) return go(block_norm_grad_kernel<T, 4, 1, KEPT8>, 4);
  if (a.cols <= 2048) return go(block_norm_grad_kernel<T, 8, 2, KEPT8>, 8);
  if (a.cols <= 4096) return go(block_norm_grad_kernel<T, 16, 2, KEPT8>, 16);
  if (a.cols <= 16384) return go(block_norm_grad_kernel<T, 16, 8, KEPT8>, 16);
  return go(block_norm_grad_kernel<T, 16, 0, KEPT8>, 16);
}

template <typename T, int G, int C, int S, int MINB, int CL, bool KEPT8>
static cudaError_t launch_ring(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int smem = GradRing<T, TH, C, S, KEPT8>::BYTES;
  static_assert(smem * MINB <= 224 * 1024, "shared memory of an SM");
  static_assert(MINB <= kBlockNormCtasPerSm, "rows of partial");
  static bool done[64] = {false};
  static int known[64] = {0};
  const auto kernel = block_norm_grad_ring_kernel<T, G, C, S, MINB, CL, KEPT8>;
  cudaError_t e = smem_limit(kernel, smem, done);
  if (e != cudaSuccess) return e;
  int most = MINB * sms;
  if (CL > 1) {
    e = resident_clusters(kernel, TH, smem, CL, known, &most);
    if (e != cudaSuccess) return e;
  }
  *ctas = static_cast<int>(std::min<long long>((a.rows + R - 1) / R, std::min(most, most_ctas(sms))));
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(*ctas * CL)), dim3(TH), smem, CL, st, a, partial);
}

// Threads, pieces and CTAs of a row by its width.
template <typename T, bool KEPT8>
static cudaError_t dispatch_ring(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = static_cast<int>((a.cols + E - 1) / E);
  if (pieces <= 32) return launch_ring<T, 32, 1, 4, 4, 1, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 64) return launch_ring<T, 64, 1, 4, 4, 1, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 128) return launch_ring<T, 128, 1, 4, 4, 1, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 256) return launch_ring<T, 256, 1, 4, 2, 1, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 512) return launch_ring<T, 512, 1, 5, 1, 1, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 1024) return launch_ring<T, 512, 1, 5, 1, 2, KEPT8>(a, partial, sms, ctas, st);
  if (pieces <= 2048) return launch_ring<T, 512, 1, 5, 1, 4, KEPT8>(a, partial, sms, ctas, st);
  return launch_ring<T, 512, 1, 5, 1, 8, KEPT8>(a, partial, sms, ctas, st);
}

cudaError_t launch_block_norm_grad(const muon_block_norm_grad_args& a, float* partial, int vec, int sms, cudaStream_t st) {
  int ctas = 0;
  const auto go = [&](auto t) {
    using T = decltype(t);
    // 8 CTAs of 512 pieces: 32768 16-bit columns, half as many of fp32
    if (vec && a.cols <= 8 * 512 * (16 / static_cast<int>(sizeof(T))))
      return a.x_scale ? dispatch_ring<T, true>(a, partial, sms, &ctas, st) : dispatch_ring<T, false>(a, partial, sms, &ctas, st);
    return a.x_scale ? dispatch_grad<T, true>(a, partial, sms, &ctas, st) : dispatch_grad<T, false>(a, partial, sms, &ctas, st);
  };
  const cudaError_t e = a.dt == MUON_BF16 ? go(__nv_bfloat16()) : a.dt == MUON_FP16 ? go(__half()) : go(float());
  if (e != cudaSuccess || !partial) return e;
  return launch_pdl(block_norm_weights_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32), 2), dim3(1024), 0, st,
                    static_cast<const float*>(partial), ctas, a);
}

}  // namespace muon
