// block_norm.cuh -- what the kernels of the norms around a block share: sums and blocks of the widest rows, entry points.
#pragma once
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "row_ring.cuh"
#include "train_ops.h"

namespace muon {

// ---- a block of 128 columns to a warp: the widest rows
// Rows of any alignment: lane l holds columns l, l + 32, l + 64 and l + 96 of a block, so that a warp's accesses are
// 32 neighbours whatever the row's first address, and a block's largest magnitude is one reduction of the warp.
template <typename T>
__device__ __forceinline__ float load_or(const void* p, long long i, bool in, float other) {
  return in ? to_f32(static_cast<const T*>(p)[i]) : other;
}
__device__ __forceinline__ float load_weight(const void* w, int dt, int col, bool in) {
  if (!w) return 1.f;
  if (dt == MUON_FP32) return load_or<float>(w, col, in, 0.f);
  return dt == MUON_BF16 ? load_or<__nv_bfloat16>(w, col, in, 0.f) : load_or<__half>(w, col, in, 0.f);
}

// n weights from `col` on, the rest 0; ANYWHERE: their address allows no vector accesses.
template <typename T, bool ANYWHERE>
__device__ __forceinline__ void load_weights(const void* w, int dt, int col, int n, float (&v)[16 / sizeof(T)]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  if constexpr (ANYWHERE) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = i < n ? load_weight(w, dt, col + i, true) : 0.f;
  } else {
    load_weight_piece<E>(w, dt, col, n, v);
  }
}

// Block kb of a row in 8 bits.  All lanes call; v is 0 past the last column.
__device__ __forceinline__ void store_block8(const muon_fp8_out& o, int fmt, long long row, long long rows, int cols, int kb,
                                             const float (&v)[4]) {
  uint8_t* data = static_cast<uint8_t*>(o.data) + row * o.ld;
  uint8_t* scale = static_cast<uint8_t*>(o.scale);
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, abs_bits(v[j]));
  const uint32_t byte = fp8_scale_byte(__reduce_max_sync(0xffffffffu, m), fmt ? 15 : 8);
  const float inv = fp8_inverse_scale(byte);
  const int lane = threadIdx.x % 32, end = (cols + 15) & ~15;
  const uint32_t four = fmt ? fp8_pack4<true>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv)
                            : fp8_pack4<false>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (kb * 128 + lane + 32 * j < end) data[kb * 128 + lane + 32 * j] = static_cast<uint8_t>(four >> (8 * j));
  if (lane == 0) {
    const long long rows4 = (rows + 3) & ~3LL;
    scale[fp8_scale_offset(kb, row, rows4)] = static_cast<uint8_t>(byte);
    if (row == rows - 1)
      for (long long r = rows; r < rows4; ++r) scale[fp8_scale_offset(kb, r, rows4)] = 127;
  }
}
// The scale words' blocks past the last column.
__device__ __forceinline__ void pad_blocks8(const muon_fp8_out& o, long long row, long long rows, int cols) {
  uint8_t* scale = static_cast<uint8_t*>(o.scale);
  const long long rows4 = (rows + 3) & ~3LL;
  for (int kb = (cols + 127) / 128 + threadIdx.x; kb < (cols + 511) / 512 * 4; kb += blockDim.x) {
    scale[fp8_scale_offset(kb, row, rows4)] = 127;
    if (row == rows - 1)
      for (long long r = rows; r < rows4; ++r) scale[fp8_scale_offset(kb, r, rows4)] = 127;
  }
}

// Sums over a CTA of W warps; every thread gets them.  `sh` alternates between two buffers: one barrier each.
template <int W, int N>
__device__ __forceinline__ void cta_sums(float (&v)[N], float (*sh)[N][W], int turn) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) sh[turn & 1][n][threadIdx.x / 32] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = sh[turn & 1][n][threadIdx.x % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  }
}

// Kernels compiled in block_norm_rows.cu and block_norm_grad_rows.cu, for T and rows that start on 16 bytes or ANYWHERE.
template <typename T, bool ANYWHERE>
cudaError_t launch_block_norm_rows(const muon_block_norm_args& a, int sms, cudaStream_t st);
// *ctas: the rows of `partial` that the kernel writes.
template <typename T, bool ANYWHERE>
cudaError_t launch_block_norm_grad_rows(const muon_block_norm_grad_args& a, float* partial, int sms, int* ctas, cudaStream_t st);

}  // namespace muon
