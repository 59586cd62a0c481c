// clip.cu -- the global norm of a list of gradients, and the gradients scaled to it.
//
//   N = sqrt(sum_i sum_j g_ij^2)      c = min(1, max_norm / (N + eps))      out = round(g c)
//
// Two launches.  The first strides a fixed grid over chunks of 8192 elements of
// the listed tensors (binary search over the chunk offsets) and leaves one partial
// sum per CTA; which CTA sums which elements in which order is fixed, so the norm
// has the same bits every time.  The second has every CTA add the partial sums (at
// most a few thousand) in order and scale its chunks.  Without a pass over memory in
// between, the floor is one read and one write of every gradient; reading them twice
// is what the norm's dependence costs, less what the second pass finds in the 126 MB
// L2: it runs the chunks in the reverse order.
//
// Sums: fp32 per thread, 64 bits across threads.  Squares that leave fp32's range
// (a CTA's sum that is not finite, or below 2^-100) are summed again, scaled by
// 2^-80 or 2^100, so the norm of finite gradients is right over the whole range.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

template <int MAX>
struct ClipArgs {
  int count;
  int chunks;           // of this launch
  int first;            // start[] of the first tensor: 0
  int nparts;           // partial sums over all launches
  float max_norm, eps;
  double* partial;
  float* norm;
  long long numel[MAX];
  const void* g[MAX];
  void* out[MAX];
  int start[MAX];       // first chunk of each tensor
  unsigned char dt[MAX];  // dtype, | 16: 16-byte aligned
};

template <int MAX>
__device__ __forceinline__ int clip_tensor(const ClipArgs<MAX>& a, int chunk) {
  int lo = 0, hi = a.count - 1;  // last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.start[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of (x s)^2 over elements e0 .. e0 + kClipChunk of a tensor, this thread's part.
template <typename T>
__device__ __forceinline__ void clip_sum_chunk(const T* g, long long e0, long long n, bool aligned, float s,
                                               float (&acc)[4]) {
#pragma unroll
  for (int u = 0; u < kClipChunk / (8 * 256); ++u) {
    const long long e = e0 + (u * 256 + threadIdx.x) * 8;
    if (e < n) {
      float v[8];
      load8(g + e, static_cast<int>(min(n - e, 8LL)), aligned && e + 8 <= n, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = v[i] * s;
        acc[i & 3] = fmaf(x, x, acc[i & 3]);
      }
    }
  }
}

template <int MAX>
__device__ __forceinline__ float clip_thread_sum(const ClipArgs<MAX>& a, float s) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int t = clip_tensor(a, c);
    const long long e0 = static_cast<long long>(c - a.start[t]) * kClipChunk, n = a.numel[t];
    const bool al = a.dt[t] & 16;
    switch (a.dt[t] & 15) {
      case MUON_BF16: clip_sum_chunk(static_cast<const __nv_bfloat16*>(a.g[t]), e0, n, al, s, acc); break;
      case MUON_FP16: clip_sum_chunk(static_cast<const __half*>(a.g[t]), e0, n, al, s, acc); break;
      default: clip_sum_chunk(static_cast<const float*>(a.g[t]), e0, n, al, s, acc); break;
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Sum over the 256 threads, in 64 bits and a fixed order; every thread gets it.
__device__ __forceinline__ double clip_block_sum(double v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += sh[w];
  return s;
}

template <int MAX>
__global__ void __launch_bounds__(256) clip_norm_kernel(const __grid_constant__ ClipArgs<MAX> a) {
  __shared__ double sh[8];
  pdl_launch_dependents();
  pdl_wait();
  double sum = clip_block_sum(static_cast<double>(clip_thread_sum(a, 1.f)), sh);
  if (!(sum < 3e38)) sum = clip_block_sum(static_cast<double>(clip_thread_sum(a, 0x1p-80f)), sh) * 0x1p160;
  else if (sum < 0x1p-100) sum = clip_block_sum(static_cast<double>(clip_thread_sum(a, 0x1p100f)), sh) * 0x1p-200;
  if (threadIdx.x == 0) a.partial[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void clip_scale_chunk(const T* g, T* out, long long e0, long long n, bool aligned, float c) {
#pragma unroll
  for (int u = 0; u < kClipChunk / (8 * 256); ++u) {
    const long long e = e0 + (u * 256 + threadIdx.x) * 8;
    if (e < n) {
      const int k = static_cast<int>(min(n - e, 8LL));
      const bool full = aligned && e + 8 <= n;
      float v[8];
      load8(g + e, k, full, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= c;
      store8(out + e, k, full, v);
    }
  }
}

template <int MAX>
__global__ void __launch_bounds__(256) clip_scale_kernel(const __grid_constant__ ClipArgs<MAX> a) {
  __shared__ double sh[8];
  pdl_launch_dependents();
  pdl_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += 256) s += a.partial[i];
  const float norm = static_cast<float>(sqrt(clip_block_sum(s, sh)));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
  float c = a.max_norm / (norm + a.eps);
  if (c > 1.f) c = 1.f;  // NaN stays
  for (int k = blockIdx.x; k < a.chunks; k += gridDim.x) {
    const int chunk = a.chunks - 1 - k;
    const int t = clip_tensor(a, chunk);
    if (c == 1.f && a.g[t] == a.out[t]) continue;
    const long long e0 = static_cast<long long>(chunk - a.start[t]) * kClipChunk, n = a.numel[t];
    const bool al = a.dt[t] & 16;
    switch (a.dt[t] & 15) {
      case MUON_BF16:
        clip_scale_chunk(static_cast<const __nv_bfloat16*>(a.g[t]), static_cast<__nv_bfloat16*>(a.out[t]), e0, n, al, c);
        break;
      case MUON_FP16:
        clip_scale_chunk(static_cast<const __half*>(a.g[t]), static_cast<__half*>(a.out[t]), e0, n, al, c);
        break;
      default:
        clip_scale_chunk(static_cast<const float*>(a.g[t]), static_cast<float*>(a.out[t]), e0, n, al, c);
        break;
    }
  }
}

// Fills the argument block with tensors [c0, c0 + n).
template <int MAX>
static void clip_fill(ClipArgs<MAX>& a, const void* const* grads, void* const* out, const int64_t* numel,
                      const int32_t* dts, int c0, int n) {
  int chunk = 0;
  a.count = n;
  for (int i = 0; i < n; ++i) {
    const int k = c0 + i;
    a.numel[i] = numel[k];
    a.g[i] = grads[k];
    a.out[i] = out ? out[k] : nullptr;
    a.start[i] = chunk;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(grads[k]) | (out ? reinterpret_cast<uintptr_t>(out[k]) : 0);
    a.dt[i] = static_cast<unsigned char>(dts[k] | (bits % 16 == 0 ? 16 : 0));
    chunk += static_cast<int>((numel[k] + kClipChunk - 1) / kClipChunk);
  }
  a.chunks = chunk;
}

template <int MAX>
static cudaError_t run_clip(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dts,
                            int count, float max_norm, float eps, double* partial, int grid, float* norm,
                            cudaStream_t st) {
  ClipArgs<MAX> a;
  a.first = 0;
  a.max_norm = max_norm;
  a.eps = eps;
  int parts = 0;
  for (int c0 = 0; c0 < count; c0 += MAX) {
    clip_fill(a, grads, out, numel, dts, c0, std::min(MAX, count - c0));
    a.partial = partial + parts;
    const int g = std::max(1, std::min(grid, a.chunks));
    const cudaError_t e = launch_pdl(clip_norm_kernel<MAX>, dim3(g), dim3(256), 0, st, a);
    if (e != cudaSuccess) return e;
    parts += g;
  }
  a.nparts = parts;
  a.partial = partial;
  const int step = out ? MAX : count;  // without outputs one CTA turns the partial sums into the norm
  for (int c0 = 0; c0 < count || c0 == 0; c0 += std::max(step, 1)) {
    if (out) clip_fill(a, grads, out, numel, dts, c0, std::min(MAX, count - c0));
    else a.chunks = 0;
    a.norm = c0 == 0 ? norm : nullptr;
    const int g = std::max(1, std::min(grid, a.chunks));
    const cudaError_t e = launch_pdl(clip_scale_kernel<MAX>, dim3(g), dim3(256), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_clip(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dts, int count,
                        float max_norm, float eps, double* partial, int grid, float* norm, cudaStream_t st) {
  static_assert(sizeof(ClipArgs<kClipLarge>) <= 32000, "kernel parameter space");
  if (count <= kClipSmall)
    return run_clip<kClipSmall>(grads, out, numel, dts, count, max_norm, eps, partial, grid, norm, st);
  return run_clip<kClipLarge>(grads, out, numel, dts, count, max_norm, eps, partial, grid, norm, st);
}

}  // namespace muon
