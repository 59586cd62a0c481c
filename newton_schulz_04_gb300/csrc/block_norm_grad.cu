// block_norm_grad.cu -- gradient of the norms around a block: the choice by type and alignment, and the sums of the weights'
// gradients.
#include <cuda_runtime.h>

#include <algorithm>

#include "block_norm.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {

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

// As many as the shapes in block_norm_grad_rows.cu let run at the same time.
int block_norm_grad_parts(long long rows, long long cols, int elem_size, int sms) {
  const long long pieces = (cols * elem_size + 15) / 16;
  const int most = pieces > 4096   ? 2 * sms  // the widest rows
                   : pieces <= 128 ? 4 * sms
                   : pieces <= 256 ? 2 * sms
                   : pieces <= 512 ? sms
                   : pieces <= 1024 ? sms / 2
                   : pieces <= 2048 ? sms / 4
                                    : sms / 8;
  return static_cast<int>(std::max(1LL, std::min<long long>(rows, most)));
}

cudaError_t launch_block_norm_grad(const muon_block_norm_grad_args& a, float* partial, int vec, int sms, cudaStream_t st) {
  int ctas = 0;
  const auto go = [&](auto t) {
    using T = decltype(t);
    return vec ? launch_block_norm_grad_rows<T, false>(a, partial, sms, &ctas, st)
               : launch_block_norm_grad_rows<T, true>(a, partial, sms, &ctas, st);
  };
  const cudaError_t e = a.dt == MUON_BF16 ? go(__nv_bfloat16()) : a.dt == MUON_FP16 ? go(__half()) : go(float());
  if (e != cudaSuccess || !partial) return e;
  return launch_pdl(block_norm_weights_kernel, dim3(static_cast<unsigned>((a.cols + 31) / 32), 2), dim3(1024), 0, st,
                    static_cast<const float*>(partial), ctas, a);
}

}  // namespace muon
