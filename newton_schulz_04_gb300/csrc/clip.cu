// clip.cu -- the global norm of a list of gradients, and the gradients scaled to it.
//
//   N = sqrt(sum_i sum_j g_ij^2)      c = min(1, max_norm / (N + eps))      out = round(g c)
//
// Two launches.  The first gives every CTA of a fixed grid a contiguous run of the
// listed tensors' 32 KB chunks and leaves one partial sum per CTA; which CTA sums
// which elements in which order is fixed, so the norm has the same bits every
// time.  The second has every CTA add the partial sums (608, in order) and scale its
// run.  Bound by memory: the norm's dependence costs a second read of the gradients
// that the floor (one read, one write) does not have, less what that read finds in the
// 126 MB L2: each CTA scales its run backwards, from what it read last, and reads and
// writes with the evict-first policy so as not to push out what is still to be read.
// A CTA's first chunk is on its way while it adds the partial sums.
//
// Sums: fp32 within a warp, 64 bits across.  Squares that leave fp32's range
// (a CTA's sum that is not finite, or below 2^-100) are summed again, scaled by
// 2^-80 or 2^100, so the norm of finite gradients is right over the whole range.
#include <cuda_runtime.h>

#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

// The last chunks of each run are read to stay in L2 for the scaling kernel (608
// runs x 4 x 32 KB = 80 MB), the ones before them as evict-first: 235M bf16 values take 223
// instead of 229 us (218 with the sums below in fp32 within a warp: 6.5 TB/s over the three passes).
// Of a 100 MB list 60 MB are then found in L2 (46 us).  16 KB chunks on more CTAs: 48 and 223 us.
constexpr int kClipStay = 4;
constexpr int kClipParts = 8;  // 16-byte parts of a chunk per thread
static_assert(kClipChunkBytes == kClipParts * 16 * 256, "one chunk is a CTA's pass");

template <int MAX>
struct ClipArgs {
  int count;
  int chunks;           // of this launch
  int nparts;           // partial sums over all launches
  float max_norm, eps;
  double* partial;
  float* norm;
  long long numel[MAX];
  const void* g[MAX];
  void* out[MAX];
  int start[MAX + 1];   // first chunk of each tensor; start[count] = chunks
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
// Chunks [lo, hi) of this CTA.
template <int MAX>
__device__ __forceinline__ int2 clip_run(const ClipArgs<MAX>& a) {
  const long long n = a.chunks;
  return make_int2(static_cast<int>(n * blockIdx.x / gridDim.x), static_cast<int>(n * (blockIdx.x + 1) / gridDim.x));
}

__device__ __forceinline__ void clip_unpack(const uint4& w, float (&v)[8], __nv_bfloat16 t) { unpack8(w, v, t); }
__device__ __forceinline__ void clip_unpack(const uint4& w, float (&v)[8], __half t) { unpack8(w, v, t); }
__device__ __forceinline__ void clip_unpack(const uint4& w, float (&v)[4], float) {
  v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y), v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ uint4 clip_pack(const float (&v)[4], float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <typename T>
__device__ __forceinline__ uint4 clip_pack(const float (&v)[8], T) {
  union {
    uint4 w;
    T e[8];
  } u;
#pragma unroll
  for (int i = 0; i < 8; ++i) u.e[i] = from_f32<T>(v[i]);
  return u.w;
}

// This thread's part of sum (x s)^2 over the chunk of n elements at g.
template <typename T>
__device__ __forceinline__ void clip_sum_chunk(const T* g, int n, bool aligned, float s, bool stay,
                                               float (&acc)[4]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));  // elements of a part
  if (aligned && n == kClipChunkBytes / static_cast<int>(sizeof(T))) {
    uint4 w[kClipParts];
#pragma unroll
    for (int u = 0; u < kClipParts; ++u) {
      const uint4* q = reinterpret_cast<const uint4*>(g) + u * 256 + threadIdx.x;
      w[u] = stay ? *q : __ldcs(q);
    }
#pragma unroll
    for (int u = 0; u < kClipParts; ++u) {
      float v[E];
      clip_unpack(w[u], v, T());
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float x = v[i] * s;
        acc[i & 3] = fmaf(x, x, acc[i & 3]);
      }
    }
  } else {
    for (int i = threadIdx.x; i < n; i += 256) {
      const float x = to_f32(g[i]) * s;
      acc[0] = fmaf(x, x, acc[0]);
    }
  }
}

template <int MAX>
__device__ __forceinline__ float clip_thread_sum(const ClipArgs<MAX>& a, float s) {
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int2 run = clip_run(a);
  int t = clip_tensor(a, run.x);
  for (int c = run.x; c < run.y; ++c) {
    while (a.start[t + 1] <= c) ++t;
    const bool al = a.dt[t] & 16, wide = (a.dt[t] & 15) == MUON_FP32;
    const int per = kClipChunkBytes / (wide ? 4 : 2);
    const long long e0 = static_cast<long long>(c - a.start[t]) * per;
    const int n = static_cast<int>(min(a.numel[t] - e0, static_cast<long long>(per)));
    const bool stay = c >= run.y - kClipStay;
    switch (a.dt[t] & 15) {
      case MUON_BF16: clip_sum_chunk(static_cast<const __nv_bfloat16*>(a.g[t]) + e0, n, al, s, stay, acc); break;
      case MUON_FP16: clip_sum_chunk(static_cast<const __half*>(a.g[t]) + e0, n, al, s, stay, acc); break;
      default: clip_sum_chunk(static_cast<const float*>(a.g[t]) + e0, n, al, s, stay, acc); break;
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// Sum over the 256 threads in a fixed order, in fp32 within a warp and 64 bits across (64-bit
// additions run at a small fraction of the fp32 rate); every thread gets it.
__device__ __forceinline__ double clip_block_sum(float v, double* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = static_cast<double>(v);
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = sh[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += sh[w];
    sh[8] = s;
  }
  __syncthreads();
  return sh[8];
}

template <int MAX>
__global__ void __launch_bounds__(256, kClipCtasPerSm) clip_norm_kernel(const __grid_constant__ ClipArgs<MAX> a) {
  __shared__ double sh[9];
  pdl_wait();
  pdl_launch_dependents();
  double sum = clip_block_sum(clip_thread_sum(a, 1.f), sh);
  if (!(sum < 3e38)) sum = clip_block_sum(clip_thread_sum(a, 0x1p-80f), sh) * 0x1p160;
  else if (sum < 0x1p-100) sum = clip_block_sum(clip_thread_sum(a, 0x1p100f), sh) * 0x1p-200;
  if (threadIdx.x == 0) a.partial[blockIdx.x] = sum;
}

// out = round(g c) for a chunk of n elements; `factor` gives c, after this thread's loads are on their way.
template <typename T, typename F>
__device__ __forceinline__ void clip_scale_chunk(const T* g, T* out, int n, bool aligned, const F& factor) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  if (aligned && n == kClipChunkBytes / static_cast<int>(sizeof(T))) {
    uint4 w[kClipParts];
#pragma unroll
    for (int u = 0; u < kClipParts; ++u) w[u] = __ldcs(reinterpret_cast<const uint4*>(g) + u * 256 + threadIdx.x);
    const float c = factor();
    if (c == 1.f && g == out) return;
#pragma unroll
    for (int u = 0; u < kClipParts; ++u) {
      float v[E];
      clip_unpack(w[u], v, T());
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] *= c;
      __stcs(reinterpret_cast<uint4*>(out) + u * 256 + threadIdx.x, clip_pack(v, T()));
    }
  } else {
    const float c = factor();
    if (c == 1.f && g == out) return;
    for (int i = threadIdx.x; i < n; i += 256) out[i] = from_f32<T>(to_f32(g[i]) * c);
  }
}

template <int MAX>
__global__ void __launch_bounds__(256, kClipCtasPerSm) clip_scale_kernel(const __grid_constant__ ClipArgs<MAX> a) {
  __shared__ float factor_sh;
  pdl_launch_dependents();
  // Before the first read of a gradient: only this wait makes what ran before the sums' kernel visible here.  With the
  // first chunk read ahead of it, 16 x 32 K fp32 took 4.7 instead of 5.4 us and the larger lists the same.
  pdl_wait();
  float c = 0.f;
  bool known = false;
  // The factor, on first use: one warp of every CTA adds the partial sums.
  const auto factor = [&]() -> float {
    if (!known) {
      known = true;
      if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < a.nparts; i += 32) s += __ldcg(a.partial + i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // within fp32's normal range its root is as exact, and much faster
        const float norm = s > 1e-30 && s < 3e38 ? sqrtf(static_cast<float>(s)) : static_cast<float>(sqrt(s));
        if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
        float f = a.max_norm / (norm + a.eps);
        if (f > 1.f) f = 1.f;  // NaN stays
        if (threadIdx.x == 0) factor_sh = f;
      }
      __syncthreads();
      c = factor_sh;
    }
    return c;
  };
  const int2 run = clip_run(a);
  int t = clip_tensor(a, max(run.y - 1, 0));
  for (int k = run.y - 1; k >= run.x; --k) {
    while (a.start[t] > k) --t;
    if (known && c == 1.f && a.g[t] == a.out[t]) continue;
    const bool al = a.dt[t] & 16, wide = (a.dt[t] & 15) == MUON_FP32;
    const int per = kClipChunkBytes / (wide ? 4 : 2);
    const long long e0 = static_cast<long long>(k - a.start[t]) * per;
    const int n = static_cast<int>(min(a.numel[t] - e0, static_cast<long long>(per)));
    switch (a.dt[t] & 15) {
      case MUON_BF16:
        clip_scale_chunk(static_cast<const __nv_bfloat16*>(a.g[t]) + e0, static_cast<__nv_bfloat16*>(a.out[t]) + e0, n, al,
                         factor);
        break;
      case MUON_FP16:
        clip_scale_chunk(static_cast<const __half*>(a.g[t]) + e0, static_cast<__half*>(a.out[t]) + e0, n, al, factor);
        break;
      default:
        clip_scale_chunk(static_cast<const float*>(a.g[t]) + e0, static_cast<float*>(a.out[t]) + e0, n, al, factor);
        break;
    }
  }
  factor();  // a CTA without chunks (the norm alone) gets here first
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
    const long long per = kClipChunkBytes / dtype_bytes(dts[k]);
    chunk += static_cast<int>((numel[k] + per - 1) / per);
  }
  a.start[n] = chunk;
  a.chunks = chunk;
}

template <int MAX>
static cudaError_t run_clip(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dts,
                            int count, float max_norm, float eps, double* partial, int grid, float* norm,
                            cudaStream_t st) {
  ClipArgs<MAX> a;
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
    else a.count = a.chunks = 0;
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
