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
// Both are one pass over memory.  A row is held in registers by G threads, 8
// consecutive columns each, C times; rows wider than that (WIDE) are read a
// second time, from L1 / L2.  A block of 128 columns lies in 16 neighbouring
// lanes, so its largest magnitude takes four shuffles.  The weight's gradient is
// summed over a CTA's rows in registers, written per CTA, and the CTAs' rows are
// added in a fixed order by a second kernel (no atomics: the same bits every time).
#include <cuda_runtime.h>

#include <algorithm>

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

// y's 8-bit copy of one 8-column piece: all 16 lanes of the 128-column block call.
__device__ __forceinline__ void store_q8(const RmsNormArgs& a, long long row, int col, const float (&y)[8], bool live) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(y[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t byte = fp8_scale_byte(m, a.fmt ? 15 : 8);
  if (!live) return;
  // up to the row's next multiple of 16 bytes: columns past the end hold 0
  if (col < ((a.cols + 15) & ~15))
    *reinterpret_cast<uint2*>(a.q + row * a.ldq + col) =
        a.fmt ? fp8_pack8<true>(y, fp8_inverse_scale(byte)) : fp8_pack8<false>(y, fp8_inverse_scale(byte));
  const int kb = col >> 7, blocks = ((a.cols + 511) >> 9) * 4;
  if ((threadIdx.x & 15) == 0 && kb < blocks) {
    const long long rows4 = (a.rows + 3) & ~3LL;
    a.qscale[fp8_scale_offset(kb, row, rows4)] = static_cast<uint8_t>(byte);
    if (row == a.rows - 1)  // scales of no row are 1
      for (long long r = a.rows; r < rows4; ++r) a.qscale[fp8_scale_offset(kb, r, rows4)] = 127;
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
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
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
      if (a.q) store_q8(a, row, col, v, live);
    }
  }
  // scale words are four blocks: the blocks past the last chunk of threads
  if (a.q && live) {
    const long long rows4 = (a.rows + 3) & ~3LL;
    const int blocks = ((a.cols + 511) >> 9) * 4;
    for (int kb = chunks * G / 16 + t; kb < blocks; kb += G) {
      a.qscale[fp8_scale_offset(kb, row, rows4)] = 127;
      if (row == a.rows - 1)
        for (long long r = a.rows; r < rows4; ++r) a.qscale[fp8_scale_offset(kb, r, rows4)] = 127;
    }
  }
}

template <typename T, int G, int C, bool WIDE>
static cudaError_t launch_norm(const RmsNormArgs& a, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  return launch_pdl(rms_norm_kernel<T, G, C, WIDE>, dim3(static_cast<unsigned>((a.rows + R - 1) / R)), dim3(TH), 0, st,
                    a);
}

template <typename T>
static cudaError_t dispatch_norm(const RmsNormArgs& a, cudaStream_t st) {
  const int pieces = (a.cols + 7) / 8;
  if (pieces <= 32) return launch_norm<T, 32, 1, false>(a, st);
  if (pieces <= 64) return launch_norm<T, 32, 2, false>(a, st);
  if (pieces <= 128) return launch_norm<T, 32, 4, false>(a, st);
  if (pieces <= 256) return launch_norm<T, 128, 2, false>(a, st);
  if (pieces <= 512) return launch_norm<T, 256, 2, false>(a, st);
  if (pieces <= 1024) return launch_norm<T, 512, 2, false>(a, st);
  if (pieces <= 2048) return launch_norm<T, 512, 4, false>(a, st);
  return launch_norm<T, 512, 1, true>(a, st);
}

cudaError_t launch_rms_norm(const RmsNormArgs& a, int dt, int sms, cudaStream_t st) {
  (void)sms;
  if (dt == MUON_BF16) return dispatch_norm<__nv_bfloat16>(a, st);
  if (dt == MUON_FP16) return dispatch_norm<__half>(a, st);
  return dispatch_norm<float>(a, st);
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

// dweight[j] = sum over the CTAs' rows: 32 columns by 8 row groups per CTA.
__global__ void __launch_bounds__(256) rms_norm_dweight_kernel(const float* partial, int ctas, int cols, float* dweight) {
  __shared__ float sh[8][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (col < cols)
    for (int r = g; r < ctas; r += 8) s += partial[static_cast<long long>(r) * cols + col];
  sh[g][lane] = s;
  __syncthreads();
  if (g == 0 && col < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sh[k][lane];
    dweight[col] = s;
  }
}

int rms_norm_grad_ctas(long long rows, int cols, int sms) {
  const int per = cols <= 1024 ? 4 : 1;  // rows per CTA
  return static_cast<int>(std::max(1LL, std::min<long long>((rows + per - 1) / per, 4LL * sms)));
}

template <typename T, int G, int C, bool WIDE>
static cudaError_t launch_grad(const RmsNormGradArgs& a, int ctas, cudaStream_t st) {
  constexpr int TH = G < 128 ? 128 : G, R = TH / G;
  const size_t smem = a.partial ? sizeof(float) * (R - 1) * a.cols : 0;
  return launch_pdl(rms_norm_grad_kernel<T, G, C, WIDE>, dim3(ctas), dim3(TH), smem, st, a);
}

template <typename T>
static cudaError_t dispatch_grad(const RmsNormGradArgs& a, int ctas, cudaStream_t st) {
  const int pieces = (a.cols + 7) / 8;
  if (pieces <= 32) return launch_grad<T, 32, 1, false>(a, ctas, st);
  if (pieces <= 64) return launch_grad<T, 32, 2, false>(a, ctas, st);
  if (pieces <= 128) return launch_grad<T, 32, 4, false>(a, ctas, st);
  if (pieces <= 256) return launch_grad<T, 128, 2, false>(a, ctas, st);
  if (pieces <= 512) return launch_grad<T, 256, 2, false>(a, ctas, st);
  if (pieces <= 1024) return launch_grad<T, 512, 2, false>(a, ctas, st);
  return launch_grad<T, 512, 1, true>(a, ctas, st);
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int dt, int sms, cudaStream_t st) {
  const int ctas = rms_norm_grad_ctas(a.rows, a.cols, sms);
  cudaError_t e = dt == MUON_BF16   ? dispatch_grad<__nv_bfloat16>(a, ctas, st)
                  : dt == MUON_FP16 ? dispatch_grad<__half>(a, ctas, st)
                                    : dispatch_grad<float>(a, ctas, st);
  if (e != cudaSuccess || !a.partial) return e;
  return launch_pdl(rms_norm_dweight_kernel, dim3((a.cols + 31) / 32), dim3(256), 0, st,
                    static_cast<const float*>(a.partial), ctas, a.cols, a.dweight);
}

}  // namespace muon
