// block_norm_grad_rows.cu -- gradient of the norms around a block, from what the forward pass kept (of the data's type, or in 8
// bits).  With X = x rho_x and H = h rho_h as kept and c = scale post:
//
//   a = dy pre       D = dh + rho_h (a - H mean(a H))       dresidual = alpha D
//   b = D sigmoid(gate) c       dx = rho_x (b - X mean(b X))       dgate = (1 - sigmoid(gate)) b X
//   dpre = sum_rows dy H       S = sum_rows D sigmoid(gate) X       dpost = S scale       dscale = S post
//
// mean(b X) needs mean(a H) first.  With u = dh + rho_h a and e = sigmoid(gate) c X it is mean(u e) - rho_h mean(a H)
// mean(H e), so a row takes one pass and one exchange of three sums.  The columns' sums stay in registers, are written per CTA
// and added in a fixed order by a second kernel.
//
// A ring of rows as in the forward kernel, one piece to a thread.  8191 x 4096 bf16 takes 92 us from e4m3 (4.7 TB/s, 70 % of the
// copy rate) and 94 from bf16 (84 %): 16 warps of 128 registers on an SM issue 60 % of its slots, 60 instructions an element.
// With scalars of fp32 it took 125, with choices at run time 120; there two rows a turn, or the rows' factors and scales copied
// with the rows, gained nothing.  Rows that start anywhere: 142 and 164 at 4095 columns.
//
// Compiled once for each type and alignment of rows (MUON_ROWS_T, MUON_ROWS_ANYWHERE).
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

// The widest rows, which a cluster's rings do not hold: 16 warps to a row, read again for the second phase, the columns' sums
// in the CTA's part of the workspace.
template <typename T, bool KEPT8>
__global__ void __launch_bounds__(512) block_norm_grad_wide_kernel(const muon_block_norm_grad_args a, float* partial) {
  constexpr int W = 16;
  __shared__ float sh[2][3][W];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, cols = static_cast<int>(a.cols);
  const int blocks = (cols + 127) / 128, turns = (blocks + W - 1) / W;
  float* part = partial ? partial + static_cast<long long>(blockIdx.x) * 2 * cols : nullptr;
  const float inv_n = 1.f / static_cast<float>(cols);
  int turn = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
    const T* dh = static_cast<const T*>(a.dh) + (a.dh ? row * a.lddh : 0);
    const Kept<T, KEPT8> kx(a.x, a.x_scale, a.ldx, row, a.rows, a.kept_fmt), kh(a.h, a.h_scale, a.ldh, row, a.rows, a.kept_fmt);
    const bool element = a.gate && !a.gate_per_row;
    const Kept<T, KEPT8> kg(element ? a.gate : nullptr, a.gate_scale, a.ldg, row, a.rows, a.kept_fmt);
    const float rx = a.rstd_x[row], rh = a.rstd_h[row];
    const float2 row_exp = exp_minus2<float>(both(a.gate && !element ? to_f32(static_cast<const T*>(a.gate)[row * a.ldg]) : 0.f));
    const float row_sig = a.gate && !element ? sigmoid_of2<float>(row_exp).x : 1.f;
    struct Element {
      float d, u, hn, xn, sig, shut, c;  // dy, dh + rho_h dy pre, H, X, sigmoid(gate) and 1 less, scale post
    };
    auto load = [&](int col, float xs, float hs, float gs) {
      Element e;
      e.d = to_f32(dy[col]);
      e.hn = kh.at(col, hs) * rh;
      e.xn = kx.at(col, xs) * rx;
      const float2 ex = exp_minus2<T>(both(element ? kg.at(col, gs) : 0.f)), s = sigmoid_of2<T>(ex);
      e.sig = element ? s.x : row_sig;
      e.shut = shut2(ex, s).x;
      e.c = load_weight(a.post, a.weight_dt, col, true) * load_weight(a.scale, a.weight_dt, col, true);
      e.u = fmaf(rh, e.d * load_weight(a.pre, a.weight_dt, col, true), a.dh ? to_f32(dh[col]) : 0.f);
      return e;
    };
    float sum[3] = {0.f, 0.f, 0.f};
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
    if (threadIdx.x == 0 && a.dgate && !element) static_cast<T*>(a.dgate)[row * a.lddgate] = from_f32<T>(shut2(row_exp, both(row_sig)).x * along);
    for (int k = 0; k < turns; ++k) {
      const int kb = warp + W * k;
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
        if (a.dgate && element) static_cast<T*>(a.dgate)[row * a.lddgate + col] = from_f32<T>(e.shut * (b * e.xn));
        if (part) {  // this thread alone holds these columns of the CTA's sums
          part[col] = (turn ? part[col] : 0.f) + e.d * e.hn;
          part[cols + col] = (turn ? part[cols + col] : 0.f) + t * e.xn;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ ring of rows
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, int bytes) {  // the rest is zero
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "n"(BYTES), "r"(bytes)
               : "memory");
}

// A thread's slots: S times ROWS rows of dy, dh, x, h and gate, a piece each; kept 8-bit ones take E bytes instead of 16.
// ANYWHERE: of T, a warp's and a little more.
template <typename T, int G, int S, int ROWS, bool KEPT8, bool ANYWHERE>
struct GradRing {
  static constexpr int TH = G < 128 ? 128 : G, LANES = G < 32 ? G : 32;
  static constexpr int E = 16 / static_cast<int>(sizeof(T)), WIDE = KEPT8 ? 2 : 5, ARRAY = ANYWHERE ? TH / 32 * kWarpSlot<LANES> : TH * 16;
  static constexpr int STAGE = WIDE * ARRAY + (5 - WIDE) * TH * E, BYTES = S * ROWS * STAGE;
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int slot, int arr) const {
    uint8_t* stage = base + slot * STAGE;
    if (arr < WIDE) return stage + arr * ARRAY + (ANYWHERE ? threadIdx.x / 32 * kWarpSlot<LANES> : threadIdx.x * 16);
    return stage + WIDE * ARRAY + ((arr - WIDE) * TH + static_cast<int>(threadIdx.x)) * E;
  }
};

// CL CTAs of a cluster to a row, G threads of each with a piece of 16 bytes, ROWS rows at a time, a ring S times as deep.
// KEPT: of x, h and an element's gate; 0: T, 1: e4m3, 2: e5m2.  GATE: a gate of every element.  Both compiled apart: chosen
// at run time they cost 8192 x 4096 a third more instructions, in pieces too small to be overlapped.
template <typename T, int G, int S, int ROWS, int MINB, int CL, int KEPT, bool GATE, bool ANYWHERE>
__global__ void __launch_bounds__(G < 128 ? 128 : G, MINB)
    block_norm_grad_ring_kernel(const muon_block_norm_grad_args a, float* partial) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int DY = 0, DH = 1, X = 2, H = 3, GA = 4;
  using P = Pairs<T>;
  using K = std::conditional_t<KEPT != 0, uint8_t, T>;
  using Slots = GradRing<T, G, S, ROWS, KEPT != 0, ANYWHERE>;
  constexpr int E = P::E, N = P::N;
  // For the second phase a gate's exponential is kept and its sigmoid formed again (TWICE), or, where not even the exponentials of
  // two rows fit, the gate is read from the ring once more (AGAIN: 8192 bf16 columns 112 us, exponentials kept 134, with 188 bytes
  // of spills).  fp32 rows, whose quotients are dear, keep exponential and sigmoid where one row at a time leaves the registers:
  // 2048 columns from e4m3 145 us, formed twice 162; two rows of 4096 at a time from e4m3 237, formed twice 193.
  constexpr bool AGAIN = GATE && KEPT == 0 && sizeof(T) == 2 && ROWS > 1;
  constexpr bool TWICE = GATE && !AGAIN && (sizeof(T) == 2 || (KEPT != 0 && ROWS > 1));
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ RowSums3<G, TH, CL, ROWS> sums;
  const Slots ring{ring_smem};
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int t = threadIdx.x % G, rr = threadIdx.x / G, cols = static_cast<int>(a.cols);
  const int n = max(0, min(E, cols - (rank * G + t) * E));  // existing columns of the piece
  const int col = n ? (rank * G + t) * E : 0;
  const long long step = static_cast<long long>(gridDim.x / CL) * R, row0 = static_cast<long long>(blockIdx.x / CL) * R + rr;
  const long long rows4 = (a.rows + 3) & ~3LL;
  long long frow = row0;  // next row to fetch
  // pointers to rows, or to the thread's pieces of them
  constexpr int BEGIN = ANYWHERE ? 0 : 1, KBEGIN = ANYWHERE && KEPT == 0 ? 0 : 1;
  const void* const dh = a.dh ? a.dh : a.dy;  // without dh nothing is read, and zeros arrive
  const long long lddh = a.dh ? a.lddh : a.lddy;
  const T* fdy = static_cast<const T*>(a.dy) + row0 * a.lddy + BEGIN * col;
  const T* fdh = static_cast<const T*>(dh) + row0 * lddh + BEGIN * col;
  const K* fx = static_cast<const K*>(a.x) + row0 * a.ldx + KBEGIN * col;
  const K* fh = static_cast<const K*>(a.h) + row0 * a.ldh + KBEGIN * col;
  const K* fg = static_cast<const K*>(a.gate) + (GATE ? row0 * a.ldg + KBEGIN * col : 0);
  auto fetch = [&](int slot) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int at = slot * ROWS + r;
      if (frow < a.rows) {
        const auto plain = [&](int arr, const T* row, const void* matrix, bool there) {
          if constexpr (ANYWHERE)
            fetch_anywhere<T, Slots::LANES>(ring.at(at, arr), row, rank * G + t, there ? cols : 0, static_cast<const uint8_t*>(matrix));
          else copy16(smem_u32(ring.at(at, arr)), row, there ? n * static_cast<int>(sizeof(T)) : 0);
        };
        const auto kept = [&](int arr, const K* row, const void* matrix) {
          if constexpr (KEPT == 0) plain(arr, row, matrix, true);
          else copy_small<E>(smem_u32(ring.at(at, arr)), row, n);
        };
        plain(DY, fdy, a.dy, true);
        plain(DH, fdh, dh, a.dh != nullptr);
        kept(X, fx, a.x);
        kept(H, fh, a.h);
        if (GATE) kept(GA, fg, a.gate);
      }
      frow += step, fdy += step * a.lddy, fdh += step * lddh, fx += step * a.ldx, fh += step * a.ldh;
      if (GATE) fg += step * a.ldg;
    }
    cp_async_commit();
  };
  // row: for its address modulo 16
  const auto read = [&](int slot, int arr, const void* matrix, long long ld, long long row, P& p) {
    if constexpr (ANYWHERE) {
      const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(matrix)) + static_cast<uint32_t>(row * ld) * sizeof(T);
      p.unpack(read_anywhere<Slots::LANES, false>(ring.at(slot, arr), static_cast<int>(at & 15u)));
    } else {
      p.unpack(*reinterpret_cast<const uint4*>(ring.at(slot, arr)));
    }
  };
  const auto read_kept = [&](int slot, int arr, const void* matrix, long long ld, long long row, P& p) {
    if constexpr (KEPT == 0) read(slot, arr, matrix, ld, row, p);
    else p.template unpack8<KEPT == 2>(ring.at(slot, arr));
  };
  if (CL > 1) cluster_sync();  // the others' shared memory is there
  pdl_wait();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s);
  float2 w1[N], w2[N], dpre[N], sx[N];  // scale post, pre, and the columns' sums
  {
    float v[E], s[E];
    load_weights<T, ANYWHERE>(a.scale, a.weight_dt, col, n, s);
    load_weights<T, ANYWHERE>(a.post, a.weight_dt, col, n, v);
#pragma unroll
    for (int i = 0; i < N; ++i) w1[i] = make_float2(v[2 * i] * s[2 * i], v[2 * i + 1] * s[2 * i + 1]);
    load_weights<T, ANYWHERE>(a.pre, a.weight_dt, col, n, v);
#pragma unroll
    for (int i = 0; i < N; ++i) w2[i] = make_float2(v[2 * i], v[2 * i + 1]), dpre[i] = sx[i] = both(0.f);
  }
  // of a row: the norms' factors, its gate, the scales of the kept pieces; fetched a row ahead
  struct RowHead {
    float rx, rh, gate;
    uint32_t xs, hs, gs;
  };
  const bool row_gated = !GATE && a.gate;
  const float* prx = a.rstd_x + row0;
  const float* prh = a.rstd_h + row0;
  long long so = fp8_scale_offset(col / 128, row0, rows4);
  const auto head = [&](long long row) {
    RowHead r = {};
    if (row < a.rows) {
      r.rx = __ldg(prx);
      r.rh = __ldg(prh);
      if (row_gated) r.gate = to_f32(static_cast<const T*>(a.gate)[row * a.ldg]);
      if (KEPT) {
        r.xs = __ldg(static_cast<const uint8_t*>(a.x_scale) + so);
        r.hs = __ldg(static_cast<const uint8_t*>(a.h_scale) + so);
        if (GATE) r.gs = __ldg(static_cast<const uint8_t*>(a.gate_scale) + so);
      }
    }
    prx += step, prh += step, so += 4 * step;
    return r;
  };
  RowHead next[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) next[r] = head(row0 + r * step);
  const float inv_cols = 1.f / static_cast<float>(cols);
  T* pdr = static_cast<T*>(a.dresidual) + row0 * a.lddr + BEGIN * col;
  T* pdx = static_cast<T*>(a.dx) + row0 * a.lddx + BEGIN * col;
  T* pdg = static_cast<T*>(a.dgate) + (GATE ? row0 * a.lddgate + BEGIN * col : 0);
  const auto put = [&](T* p, bool there, const P& v) {
    if constexpr (ANYWHERE) store_anywhere<T, Slots::LANES>(p, rank * G + t, there ? cols - (rank * G + t) * E : 0, v);
    else if (there) v.store(p, n);
  };
  const bool gate_out = row_gated && a.dgate && t == 0 && rank == 0;
  int slot = 0, turn = 0;
  for (long long row = row0; row - rr < a.rows; row += ROWS * step, ++turn) {
    if (row - rr + ROWS * step >= a.rows) pdl_launch_dependents();  // the last turn, as in the forward kernel
    RowHead now[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) now[r] = next[r], next[r] = head(row + (ROWS + r) * step);
    if (ANYWHERE) __syncwarp();
    fetch(slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    if (ANYWHERE) __syncwarp();
    P u[ROWS], ex[ROWS], xn[ROWS], hn[ROWS];  // ex: the gate, then exp(-gate), from which its sigmoid is formed twice
    float sum[ROWS][3];
    float2 row_exp[ROWS], row_sig[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int at = slot * ROWS + r;
      const long long here = row + r * step;
      P d;
      read(at, DY, a.dy, a.lddy, here, d);
      read(at, DH, dh, lddh, here, u[r]);
      read_kept(at, X, a.x, a.ldx, here, xn[r]);
      read_kept(at, H, a.h, a.ldh, here, hn[r]);
      if (GATE) read_kept(at, GA, a.gate, a.ldg, here, ex[r]);
      if ((R > 1 || ROWS > 1) && here >= a.rows) {  // the slot holds another row's remains
#pragma unroll
        for (int i = 0; i < N; ++i) d.v[i] = xn[r].v[i] = hn[r].v[i] = u[r].v[i] = ex[r].v[i] = both(0.f);
      }
      const float2 xf = both(KEPT ? now[r].rx * fp8_scale_value(now[r].xs) : now[r].rx);
      const float2 hf = both(KEPT ? now[r].rh * fp8_scale_value(now[r].hs) : now[r].rh);
      const float2 gf = both(KEPT ? fp8_scale_value(now[r].gs) : 1.f);
      row_exp[r] = both(row_gated ? exp_minus2<float>(both(now[r].gate)).x : 0.f);
      row_sig[r] = both(row_gated ? sigmoid_of2<float>(row_exp[r]).x : 1.f);
      float2 s0 = both(0.f), s1 = s0, s2 = s0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        hn[r].v[i] = mul2(hn[r].v[i], hf);
        xn[r].v[i] = mul2(xn[r].v[i], xf);
        const float2 ad = mul2(d.v[i], w2[i]);
        u[r].v[i] = fma2(both(now[r].rh), ad, u[r].v[i]);
        if (GATE) ex[r].v[i] = exp_minus2<T>(KEPT ? mul2(ex[r].v[i], gf) : ex[r].v[i]);
        const float2 e = mul2(mul2(GATE ? sigmoid_of2<T>(ex[r].v[i]) : row_sig[r], w1[i]), xn[r].v[i]);
        s0 = fma2(ad, hn[r].v[i], s0);
        s1 = fma2(u[r].v[i], e, s1);
        s2 = fma2(hn[r].v[i], e, s2);
        dpre[i] = fma2(d.v[i], hn[r].v[i], dpre[i]);
      }
      sum[r][0] = total(s0), sum[r][1] = total(s1), sum[r][2] = total(s2);
    }
    sums(sum, turn);
    if (TWICE) {  // the compiler would keep both
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+f"(ex[r].v[i].x), "+f"(ex[r].v[i].y));
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long long here = row + r * step;
      const bool live = (R == 1 && ROWS == 1) || here < a.rows;
      const float k1 = sum[r][0] * inv_cols * now[r].rh, along = sum[r][1] - k1 * sum[r][2], k2 = along * inv_cols;
      if (gate_out && live) static_cast<T*>(a.dgate)[here * a.lddgate] = from_f32<T>(shut2(row_exp[r], row_sig[r]).x * along);
      P dr, dx, dg;
      if (AGAIN) {
        read(slot * ROWS + r, GA, a.gate, a.ldg, here, ex[r]);
#pragma unroll
        for (int i = 0; i < N; ++i) ex[r].v[i] = live ? exp_minus2<T>(ex[r].v[i]) : both(0.f);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 sig = GATE ? sigmoid_of2<T>(ex[r].v[i]) : row_sig[r];
        const float2 v = fma2(both(-k1), hn[r].v[i], u[r].v[i]), td = mul2(v, sig), b = mul2(td, w1[i]);
        sx[i] = fma2(td, xn[r].v[i], sx[i]);
        dr.v[i] = mul2(both(a.alpha), v);
        dx.v[i] = mul2(both(now[r].rx), fma2(both(-k2), xn[r].v[i], b));
        if (GATE) dg.v[i] = mul2(shut2(ex[r].v[i], sig), mul2(b, xn[r].v[i]));
      }
      put(pdr, live && a.dresidual, dr);
      put(pdx, live && a.dx, dx);
      if (GATE) put(pdg, live && a.dgate, dg);
      pdr += step * a.lddr, pdx += step * a.lddx;
      if (GATE) pdg += step * a.lddgate;
    }
    slot = slot + 1 == S ? 0 : slot + 1;
  }
  if (!partial) return;
  float* part = partial + static_cast<long long>(blockIdx.x / CL) * 2 * cols;
  if (R > 1) {  // join the CTA's row groups through the ring's memory
    static_assert(R == 1 || (R - 1) * 2 * N * G * 8 <= Slots::BYTES, "room to join");
    cp_async_wait<0>();
    __syncthreads();
    float2* all = reinterpret_cast<float2*>(ring_smem);  // [R - 1][2][N][G]
    if (rr > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        all[(((rr - 1) * 2 + 0) * N + i) * G + t] = dpre[i];
        all[(((rr - 1) * 2 + 1) * N + i) * G + t] = sx[i];
      }
    }
    __syncthreads();
    if (rr > 0) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
      for (int r = 1; r < R; ++r) {
        dpre[i] = add2(dpre[i], all[(((r - 1) * 2 + 0) * N + i) * G + t]);
        sx[i] = add2(sx[i], all[(((r - 1) * 2 + 1) * N + i) * G + t]);
      }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float* p = part + col + 2 * i;
    if (2 * i < n) p[0] = dpre[i].x, p[cols] = sx[i].x;
    if (2 * i + 1 < n) p[1] = dpre[i].y, p[cols + 1] = sx[i].y;
  }
}

template <typename T, int G, int S, int ROWS, int MINB, int CL, int KEPT, bool GATE, bool ANYWHERE>
static cudaError_t launch_ring(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  constexpr int smem = GradRing<T, G, S, ROWS, KEPT != 0, ANYWHERE>::BYTES;
  static_assert(smem * MINB <= 224 * 1024, "shared memory of an SM");
  static bool done[64] = {false};
  static int known[64] = {0};
  const auto kernel = block_norm_grad_ring_kernel<T, G, S, ROWS, MINB, CL, KEPT, GATE, ANYWHERE>;
  cudaError_t e = smem_limit(kernel, smem, done);
  if (e != cudaSuccess) return e;
  int most = MINB * sms;
  if (CL > 1) {
    e = resident_clusters(kernel, TH, smem, CL, known, &most);
    if (e != cudaSuccess) return e;
  }
  most = std::min(most, block_norm_grad_parts(a.rows, a.cols, sizeof(T), sms));
  *ctas = static_cast<int>(std::min<long long>((a.rows + R - 1) / R, most));
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(*ctas * CL)), dim3(TH), smem, CL, st, a, partial);
}

template <int N>
using Int = std::integral_constant<int, N>;
// Threads of a CTA, rows of the ring, CTAs of an SM and of a cluster by a row's width, as measured at 33.5M elements.
template <typename T, int KEPT, bool GATE, bool ANYWHERE>
static cudaError_t dispatch_ring(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int pieces = static_cast<int>((a.cols + E - 1) / E);
  const auto go = [&](auto threads, auto depth, auto rows, auto ctas_per_sm, auto cluster) {
    return launch_ring<T, decltype(threads)::value, decltype(depth)::value, decltype(rows)::value, decltype(ctas_per_sm)::value,
                       decltype(cluster)::value, KEPT, GATE, ANYWHERE>(a, partial, sms, ctas, st);
  };
  if (pieces <= 16) return go(Int<16>(), Int<4>(), Int<1>(), Int<4>(), Int<1>());
  if (pieces <= 32) return go(Int<32>(), Int<4>(), Int<1>(), Int<4>(), Int<1>());
  if (pieces <= 64) return go(Int<64>(), Int<4>(), Int<1>(), Int<4>(), Int<1>());
  if (pieces <= 128) return go(Int<128>(), Int<4>(), Int<1>(), Int<4>(), Int<1>());
  if (pieces <= 256) return go(Int<256>(), Int<4>(), Int<1>(), Int<2>(), Int<1>());
  if (pieces <= 512) return go(Int<512>(), Int<4>(), Int<1>(), Int<1>(), Int<1>());
  // Rows over a cluster, which waits for its exchange: two rows at a time share it where that was measured faster, which is where
  // their values fit the registers but for a few bytes (none to 24 of spills).  33.5M elements at 8192 and 16384 columns: 16-bit
  // rows 112 and 123 us (one row at a time 141 and 157), fp32 237 and 282 (270 and 329), fp32 from 8 bits 211 and 294 (243 and 292).
  // 16-bit rows from 8 bits, one at a time: 126 and 150, two at a time 140 and 159 with spills; at 8192 columns they take clusters
  // of four small CTAs, two of which share an SM, against two large ones' 139
  if constexpr (KEPT == 0 || sizeof(T) == 4) {
    if (pieces <= 1024) return go(Int<512>(), Int<2>(), Int<2>(), Int<1>(), Int<2>());
    if (pieces <= 2048) return go(Int<512>(), Int<2>(), Int<2>(), Int<1>(), Int<4>());
    return go(Int<512>(), Int<2>(), Int<2>(), Int<1>(), Int<8>());
  } else {
    if (pieces <= 1024) return go(Int<256>(), Int<5>(), Int<1>(), Int<2>(), Int<4>());
    if (pieces <= 2048) return go(Int<512>(), Int<5>(), Int<1>(), Int<1>(), Int<4>());
    return go(Int<512>(), Int<5>(), Int<1>(), Int<1>(), Int<8>());
  }
}

template <typename T, bool ANYWHERE>
cudaError_t launch_block_norm_grad_rows(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st) {
  // 8 CTAs of 512 pieces: 32768 16-bit columns, half as many of fp32
  if (a.cols > 8 * 512 * (16 / static_cast<int>(sizeof(T)))) {
    *ctas = block_norm_grad_parts(a.rows, a.cols, sizeof(T), sms);
    return a.x_scale ? launch_pdl(block_norm_grad_wide_kernel<T, true>, dim3(*ctas), dim3(512), 0, st, a, partial)
                     : launch_pdl(block_norm_grad_wide_kernel<T, false>, dim3(*ctas), dim3(512), 0, st, a, partial);
  }
  const int kept = !a.x_scale ? 0 : a.kept_fmt ? 2 : 1;
  const auto go = [&](auto gate) {
    constexpr bool GATE = decltype(gate)::value;
    if (kept == 0) return dispatch_ring<T, 0, GATE, ANYWHERE>(a, partial, sms, ctas, st);
    return kept == 1 ? dispatch_ring<T, 1, GATE, ANYWHERE>(a, partial, sms, ctas, st) : dispatch_ring<T, 2, GATE, ANYWHERE>(a, partial, sms, ctas, st);
  };
  return a.gate && !a.gate_per_row ? go(std::true_type()) : go(std::false_type());
}
template cudaError_t launch_block_norm_grad_rows<MUON_ROWS_T, MUON_ROWS_ANYWHERE>(const muon_block_norm_grad_args&, float*, int, int*,
                                                                                   cudaStream_t);

}  // namespace muon
