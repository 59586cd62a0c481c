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

#include "block_norm.cuh"
#include "kernels.h"
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

int block_norm_grad_ctas(long long rows, int sms) {
  return static_cast<int>(std::max(1LL, std::min<long long>(rows, static_cast<long long>(kBlockNormCtasPerSm) * sms)));
}

template <typename T, bool KEPT8>
static cudaError_t dispatch_grad(const muon_block_norm_grad_args& a, float* partial, int ctas, cudaStream_t st) {
  const auto go = [&](auto kernel, int warps) { return launch_pdl(kernel, dim3(ctas), dim3(warps * 32), 0, st, a, partial); };
  if (a.cols <= 512) return go(block_norm_grad_kernel<T, 4, 1, KEPT8>, 4);
  if (a.cols <= 2048) return go(block_norm_grad_kernel<T, 8, 2, KEPT8>, 8);
  if (a.cols <= 4096) return go(block_norm_grad_kernel<T, 16, 2, KEPT8>, 16);
  if (a.cols <= 16384) return go(block_norm_grad_kernel<T, 16, 8, KEPT8>, 16);
  return go(block_norm_grad_kernel<T, 16, 0, KEPT8>, 16);
}

cudaError_t launch_block_norm_grad(const muon_block_norm_grad_args& a, float* partial, int vec, int sms, cudaStream_t st) {
  const int ctas = block_norm_grad_ctas(a.rows, sms);
  const auto go = [&](auto t) {
    using T = decltype(t);
    return a.x_scale ? dispatch_grad<T, true>(a, partial, ctas, st) : dispatch_grad<T, false>(a, partial, ctas, st);
  };
  const cudaError_t e = a.dt == MUON_BF16 ? go(__nv_bfloat16()) : a.dt == MUON_FP16 ? go(__half()) : go(float());
  if (e != cudaSuccess || !partial) return e;
  return launch_pdl(block_norm_weights_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32), 2), dim3(1024), 0, st,
                    static_cast<const float*>(partial), ctas, a);
}

}  // namespace muon
