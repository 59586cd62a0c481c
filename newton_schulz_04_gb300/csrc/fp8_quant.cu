// fp8_quant.cu -- bf16 / fp16 / fp32 matrices to 8 bits with power-of-two scales, along rows, along columns, or both.
//
//   e = the smallest exponent with  largest |x| of the block <= top 2^e        q = round8(x 2^-e)
//
// Blocks are 1 x 128 along the axis that the product sums over, or 128 x 128.
// `q` keeps x's orientation (blocks along its columns); `qt` is x transposed
// (blocks along x's rows), what a weight gradient reads, where the summed axis is
// the tokens.  One pass over x writes both: bound by memory (2 + 1 + 1 bytes per
// bf16 element).  A CTA takes a 128 x 128 tile, each thread 8 x 8 of it in
// registers; row maxima are four shuffles, column maxima and the transposed bytes go
// through 16 KB of shared memory (8-byte slots swizzled, so both the writes by
// column and the reads by row are free of bank conflicts).
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const Fp8QuantArgs a) {
  __shared__ uint2 tile[128][16];     // transposed bytes: [column][8-row slot, swizzled]
  __shared__ uint32_t cmax[8][128];   // column maxima of each warp's 16 rows
  pdl_launch_dependents();
  pdl_wait();
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // 8 columns, 8 rows of this thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long kbc = blockIdx.x, kbr = blockIdx.y;  // column block, row block of the tile
  const long long c0 = kbc * 128 + cg * 8, r0 = kbr * 128 + rg * 8;
  const bool e5m2 = a.fmt != 0;
  const int top = e5m2 ? 15 : 8;
  float v[8][8];
  const int nc = static_cast<int>(max(0LL, min(8LL, a.cols - c0)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = r0 + i < a.rows;
    const T* p = static_cast<const T*>(a.x) + (in ? (r0 + i) * a.ldx + (nc ? c0 : 0) : 0);
    load8(p, in ? nc : 0, in && nc == 8 && a.vec, v[i]);
  }
  uint32_t rm[8], cm[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rm[i] = cm[i] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = abs_bits(v[i][j]);
      rm[i] = max(rm[i], b);
      cm[j] = max(cm[j], b);
    }
  if (a.square) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) cmax[0][warp] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, cmax[0][w]);
#pragma unroll
    for (int i = 0; i < 8; ++i) rm[i] = cm[i] = m;
  }
  if (a.q) {
    const long long rows4 = (a.rows + 3) & ~3LL, kend = (a.cols + 511) / 512 * 4;
    const bool last = c0 - cg * 8 + 128 >= a.cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = rm[i];
      if (!a.square) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      const long long r = r0 + i;
      const uint32_t byte = r < a.rows ? fp8_scale_byte(m, top) : 127u;
      if (r < a.rows && c0 < ((a.cols + 15) & ~15LL))
        *reinterpret_cast<uint2*>(a.q + r * a.ldq + c0) = fp8_pack8(v[i], fp8_inverse_scale(byte), e5m2);
      if (r < rows4) {
        if (cg == 0) a.qs[fp8_scale_offset(kbc, r, rows4)] = static_cast<uint8_t>(byte);
        if (last && cg > 0 && kbc + cg < kend) a.qs[fp8_scale_offset(kbc + cg, r, rows4)] = 127;
      }
    }
  }
  if (a.qt) {
    if (!a.square) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
        if (lane < 16) cmax[warp][cg * 8 + j] = cm[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, cmax[w][cg * 8 + j]);
        cm[j] = m;
      }
    }
    const long long cols4 = (a.cols + 3) & ~3LL, kend = (a.rows + 511) / 512 * 4;
    const bool last = (kbr + 1) * 128 >= a.rows;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long c = c0 + j;
      const uint32_t byte = c < a.cols ? fp8_scale_byte(cm[j], top) : 127u;
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[i][j];
      tile[cg * 8 + j][rg ^ cg] = fp8_pack8(u, fp8_inverse_scale(byte), e5m2);
      if (c < cols4) {
        if (rg == 0) a.qts[fp8_scale_offset(kbr, c, cols4)] = static_cast<uint8_t>(byte);
        if (last && rg > 0 && rg < 4 && kbr + rg < kend) a.qts[fp8_scale_offset(kbr + rg, c, cols4)] = 127;
      }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int cl = it * 16 + rg, slot = cg;
      const long long c = kbc * 128 + cl, r = kbr * 128 + slot * 8;
      if (c < a.cols && r < ((a.rows + 15) & ~15LL))
        *reinterpret_cast<uint2*>(a.qt + c * a.ldqt + r) = tile[cl][slot ^ (cl >> 3)];
    }
  }
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dt, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>((a.rows + 127) / 128));
  if (dt == MUON_BF16) return launch_pdl(fp8_quantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, a);
  if (dt == MUON_FP16) return launch_pdl(fp8_quantize_kernel<__half>, grid, dim3(256), 0, st, a);
  return launch_pdl(fp8_quantize_kernel<float>, grid, dim3(256), 0, st, a);
}

}  // namespace muon
