// row_ring.cuh -- pieces of the norm kernels: a ring of rows in shared memory that each thread fills for itself, sums over
// the threads of a row, the row's factor.
#pragma once
#include <cuda_runtime.h>

#include <mutex>

#include "fp8.cuh"
#include "ptx.cuh"

namespace muon {

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {  // the rest of 16 is zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}

// E elements of 16 bytes: a thread's piece of a row.
template <typename T>
__device__ __forceinline__ void unpack_piece(const uint4& w, float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(w, v, T());
  } else {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
}
// n of the elements exist.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int n, const float (&v)[16 / sizeof(T)]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  union {
    uint4 w;
    T e[E];
  } u;
#pragma unroll
  for (int i = 0; i < E; ++i) u.e[i] = from_f32<T>(v[i]);
  if (n == E) {
    *reinterpret_cast<uint4*>(p) = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) p[i] = u.e[i];
  }
}
template <int E>
__device__ __forceinline__ void load_weight_piece(const void* w, int dt, int col, int n, float (&v)[E]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 1.f;
  } else if (dt == MUON_FP32) {
    const float* p = static_cast<const float*>(w) + col;
    if (n == E) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const float4 f = reinterpret_cast<const float4*>(p)[q];
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = i < n ? p[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      v[i] = i >= n               ? 0.f
             : dt == MUON_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(w)[col + i])
                               : to_f32(static_cast<const __half*>(w)[col + i]);
  }
}

// A thread's slots: S rows of NA arrays of C pieces; thread-private.
template <typename T, int TH, int C, int S, int NA>
struct Ring {
  static constexpr int BYTES = S * NA * C * TH * 16;
  uint8_t* base;
  __device__ __forceinline__ uint8_t* at(int slot, int arr, int c) const {
    return base + (((slot * NA + arr) * C + c) * TH + static_cast<int>(threadIdx.x)) * 16;
  }
  // Piece c of a row: the 16 bytes at src, `bytes` of which exist (the rest reads as 0).
  __device__ __forceinline__ void fetch(int slot, int arr, int c, const T* src, int bytes) const {
    copy16(smem_u32(at(slot, arr, c)), src, bytes);
  }
  __device__ __forceinline__ void read(int slot, int arr, int c, float (&v)[16 / sizeof(T)]) const {
    unpack_piece<T>(*reinterpret_cast<const uint4*>(at(slot, arr, c)), v);
  }
};

// Sum over the G threads of a row, one barrier: `sh` alternates between two buffers.
template <int G, int TH>
__device__ __forceinline__ float ring_sum(float v, float (*sh)[TH / 32], int turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 32) return v;
  if ((threadIdx.x & 31) == 0) sh[turn & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  constexpr int W = G / 32;  // added as a tree: each of the last additions rounds the whole
  float s = sh[turn & 1][(threadIdx.x / G) * W + (threadIdx.x & (W - 1))];
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// 1 / sqrt(sum / cols + eps), the quotient and the root corrected by a step of Newton's:
// y goes on to 8 bits, and an error common to a row moves all its values that lie near the middle of two.
__device__ __forceinline__ float row_rstd(float sum, float cols, float inv_cols, float eps) {
  const float q = sum * inv_cols;
  const float m = (isfinite(q) ? fmaf(fmaf(-q, cols, sum), inv_cols, q) : q) + eps;
  const float r = rsqrtf(m);
  const float better = fmaf(0.5f * r, fmaf(-(m * r), r, 1.f), r);
  return isfinite(better) ? better : r;  // of a sum of 0 (without eps), infinity or NaN
}

// A kernel's limit of dynamic shared memory, raised once per device.
template <typename F>
inline cudaError_t smem_limit(F kernel, int bytes, bool (&done)[64]) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

// Sums over the threads of a row: G threads of each of the CL CTAs of a cluster (CL = 1: of a CTA that holds TH / G rows).  One
// barrier; the shared memory alternates between two buffers.
template <int G, int TH, int CL>
struct RowSum {
  static constexpr int WARPS = TH / 32, W = G < 32 ? 1 : G / 32;
  static_assert(CL == 1 || (G == TH && (CL * WARPS <= 32 || CL * WARPS % 32 == 0)), "rows of whole CTAs");
  float v[2][CL * WARPS];
  __device__ __forceinline__ float operator()(float s, int turn) {
#pragma unroll
    for (int o = G < 32 ? G / 2 : 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (G <= 32 && CL == 1) return s;
    float(&b)[CL * WARPS] = v[turn & 1];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if constexpr (CL == 1) {
      if (lane == 0) b[warp] = s;
      __syncthreads();
      s = b[(threadIdx.x / G) * W + (threadIdx.x & (W - 1))];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);  // a tree: each of the last additions rounds the whole
    } else {
      if (lane < CL) st_shared_cluster(mapa_cluster(&b[cluster_ctarank() * WARPS + warp], lane), __float_as_int(s));  // a lane to a CTA
      __syncwarp();
      cluster_sync();
      s = lane < CL * WARPS ? b[lane] : 0.f;
#pragma unroll
      for (int k = 32; k < CL * WARPS; k += 32) s += b[k + lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    return s;
  }
};

// Three sums of each of ROWS rows at once: they part company as the lanes that hold them halve, so that a quarter of a warp
// (or half warp) ends with one of them; half of the instructions of three sums in all lanes.
template <int G, int TH, int CL, int ROWS>
struct RowSums3 {
  static constexpr int WARPS = TH / 32, W = G < 32 ? 1 : G / 32, LANES = G < 32 ? G : 32, Q = LANES / 4;
  static_assert(CL == 1 || (G == TH && CL <= Q), "rows of whole CTAs");
  alignas(16) float v[2][ROWS][3][CL * WARPS];
  static __device__ __forceinline__ float quarter(float f) {
#pragma unroll
    for (int o = Q / 2; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
    return f;
  }
  __device__ __forceinline__ void operator()(float (&s)[ROWS][3], int turn) {
    const int lane = threadIdx.x % LANES, at = lane % Q;  // lanes of quarter 0: the first sum, 1 and 3: the second, 2: the third
    const bool up = lane & (2 * Q), odd = lane & Q, one = lane / Q < 3;
    const int warp = threadIdx.x / 32, sum = odd ? 1 : up ? 2 : 0;
    float f[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const float k = (up ? s[r][2] : s[r][0]) + __shfl_xor_sync(0xffffffffu, up ? s[r][0] : s[r][2], 2 * Q);
      const float m = s[r][1] + __shfl_xor_sync(0xffffffffu, s[r][1], 2 * Q);
      f[r] = quarter((odd ? m : k) + __shfl_xor_sync(0xffffffffu, odd ? k : m, Q));
    }
    if constexpr (G > 32 || CL > 1) {
      float(&b)[ROWS][3][CL * WARPS] = v[turn & 1];
      if constexpr (CL == 1) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          if (at == 0 && one) b[r][sum][warp] = f[r];
        __syncthreads();
        const int first = (threadIdx.x / G) * W;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          f[r] = at < W ? b[r][sum][first + at] : 0.f;
#pragma unroll
          for (int k = Q; k < W; k += Q) f[r] += b[r][sum][first + k + at];
        }
      } else {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          if (at < CL && one)  // a lane to a CTA of the cluster
            st_shared_cluster(mapa_cluster(&b[r][sum][cluster_ctarank() * WARPS + warp], at), __float_as_int(f[r]));
        __syncwarp();
        cluster_sync();
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          f[r] = 0.f;
#pragma unroll
          for (int k = 0; k < CL * WARPS; k += 4 * Q) {
            const float4 p = k + 4 * at < CL * WARPS ? *reinterpret_cast<const float4*>(&b[r][sum][k + 4 * at]) : make_float4(0.f, 0.f, 0.f, 0.f);
            f[r] += (p.x + p.y) + (p.z + p.w);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) f[r] = quarter(f[r]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int n = 0; n < 3; ++n) s[r][n] = __shfl_sync(0xffffffffu, f[r], n * Q, LANES);
  }
};

// Clusters of a kernel that run at the same time, asked for once per device (0: not asked yet).
template <typename F>
inline cudaError_t resident_clusters(F kernel, int threads, int smem, int cluster, int (&known)[64], int* count) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[dev] = n;
  }
  *count = known[dev];
  return cudaSuccess;
}

}  // namespace muon
