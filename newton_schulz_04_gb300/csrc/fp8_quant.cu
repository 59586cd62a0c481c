// fp8_quant.cu -- bf16 / fp16 / fp32 matrices to 8 bits with power-of-two scales, along rows, along columns, or both.
//
//   e = the smallest exponent with  largest |x| of the block <= top 2^e        q = round8(x 2^-e)
//
// Blocks are 1 x 128 along the axis that the product sums over, or 128 x 128.
// `q` keeps x's orientation (blocks along its columns); `qt` is x transposed
// (blocks along x's rows), what a weight gradient reads, where the summed axis is
// the tokens.  One pass over x writes both: 2 + 1 + 1 bytes per bf16 element.  A CTA
// takes a 128 x 128 tile, each thread 8 x 8 of it in registers (16-bit types as
// loaded, two to a register, with maxima of packed halves); row maxima are four
// shuffles, column maxima and the transposed bytes go through 16 KB of shared memory
// (8-byte slots swizzled, so both the writes by column and the reads by row are free
// of bank conflicts).  A square block's bytes are the same both ways and are only
// transposed, four by four.  Bound by memory and, close behind, by the conversions: 4096 x
// 14336 bf16 takes 39 us (6.0 TB/s); with values unpacked to fp32, formats chosen at run
// time and every byte converted twice it took 106.
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

// 16-bit magnitudes compare as whole numbers, two to a word.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// fp32 bits of a 16-bit magnitude
__device__ __forceinline__ uint32_t wide_bits(uint32_t h, __nv_bfloat16) { return h << 16; }
__device__ __forceinline__ uint32_t wide_bits(uint32_t h, __half) {
  return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}
__device__ __forceinline__ float2 two_f32(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 two_f32(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The 8 x 8 elements of a thread.  16-bit types stay packed as they were loaded
// (32 registers instead of 64).
template <typename T>
struct Piece {
  static constexpr int W = static_cast<int>(sizeof(T)) * 2;  // words of 8 elements
  uint32_t w[8][W];
  __device__ __forceinline__ void load(int i, const T* p, int n, bool full) {
    if (full) {
#pragma unroll
      for (int q = 0; q < W / 4; ++q) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[q];
        w[i][4 * q] = x.x, w[i][4 * q + 1] = x.y, w[i][4 * q + 2] = x.z, w[i][4 * q + 3] = x.w;
      }
    } else {
      union {
        T e[8];
        uint32_t u[W];
      } x;
#pragma unroll
      for (int q = 0; q < W; ++q) x.u[q] = 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) x.e[j] = p[j];
#pragma unroll
      for (int q = 0; q < W; ++q) w[i][q] = x.u[q];
    }
  }
  __device__ __forceinline__ float2 pair(int i, int q) const {  // elements 2 q, 2 q + 1 of row i
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[i][2 * q]), __uint_as_float(w[i][2 * q + 1]));
    else return two_f32(w[i][q], T());
  }
  __device__ __forceinline__ float at(int i, int j) const {
    const float2 f = pair(i, j >> 1);
    return j & 1 ? f.y : f.x;
  }
};

template <typename T, bool E5M2, bool SQUARE>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : SQUARE ? 3 : 2) fp8_quantize_kernel(const Fp8QuantArgs a) {
  constexpr int W = Piece<T>::W;
  __shared__ uint2 tile[128][16];  // transposed bytes: [column][8-row slot, swizzled]
  __shared__ __align__(16) uint32_t cmax[8][16][W];  // column maxima of each warp's 16 rows
  pdl_launch_dependents();
  pdl_wait();
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // 8 columns, 8 rows of this thread
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long kbc = blockIdx.x, kbr = blockIdx.y;  // column block, row block of the tile
  const long long c0 = kbc * 128 + cg * 8, r0 = kbr * 128 + rg * 8;
  constexpr int top = E5M2 ? 15 : 8;
  Piece<T> x;
  const int nc = static_cast<int>(max(0LL, min(8LL, a.cols - c0)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = r0 + i < a.rows;
    const T* p = static_cast<const T*>(a.x) + (in ? (r0 + i) * a.ldx + (nc ? c0 : 0) : 0);
    x.load(i, p, in ? nc : 0, in && nc == 8 && a.vec);
  }
  // maxima as fp32 bits of the rows, and of the columns as stored (packed pairs, or fp32 bits)
  uint32_t rm[8], cw[W];
#pragma unroll
  for (int q = 0; q < W; ++q) cw[q] = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m = 0u;
#pragma unroll
    for (int q = 0; q < W; ++q) {
      if constexpr (sizeof(T) == 4) {
        const uint32_t b = x.w[i][q] & 0x7fffffffu;
        m = max(m, b);
        cw[q] = max(cw[q], b);
      } else {
        const uint32_t b = x.w[i][q] & 0x7fff7fffu;
        m = max_u16x2(m, b);
        cw[q] = max_u16x2(cw[q], b);
      }
    }
    rm[i] = m;
  }
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // two rows to a word
      uint32_t m = max_u16x2(__byte_perm(rm[i], rm[i + 1], 0x5410), __byte_perm(rm[i], rm[i + 1], 0x7632));
      if (a.q && !SQUARE) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
      rm[i] = wide_bits(m & 0xffffu, T());
      rm[i + 1] = wide_bits(m >> 16, T());
    }
  } else if (a.q && !SQUARE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) rm[i] = max(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
  }
  uint32_t one = 0u;  // the square block's scale byte
  if (SQUARE) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t* sq = &cmax[0][0][0];
    if (lane == 0) sq[warp] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, sq[w]);
    one = fp8_scale_byte(m, top);
  }
  uint2 o[8];  // 8-bit rows
  if (a.q || SQUARE) {
    const long long rows4 = (a.rows + 3) & ~3LL, kend = (a.cols + 511) / 512 * 4;
    const int rows_here = static_cast<int>(max(0LL, min(8LL, a.rows - r0)));
    const int pads_here = static_cast<int>(max(0LL, min(8LL, rows4 - r0)));
    const bool last = c0 - cg * 8 + 128 >= a.cols;
    uint8_t* q = a.q + r0 * a.ldq + c0;
    uint8_t* qs = a.qs + fp8_scale_offset(kbc, r0, rows4);
    uint8_t* qs_pad = last && cg > 0 && cg < 4 && kbc + cg < kend ? a.qs + fp8_scale_offset(kbc + cg, r0, rows4) : nullptr;
    const bool in = c0 < ((a.cols + 15) & ~15LL);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = i >= rows_here ? 127u : SQUARE ? one : fp8_scale_byte(rm[i], top);
      const float inv = fp8_inverse_scale(byte);
      const float2 f0 = x.pair(i, 0), f1 = x.pair(i, 1), f2 = x.pair(i, 2), f3 = x.pair(i, 3);
      o[i] = make_uint2(fp8_pack4<E5M2>(f0.x * inv, f0.y * inv, f1.x * inv, f1.y * inv),
                        fp8_pack4<E5M2>(f2.x * inv, f2.y * inv, f3.x * inv, f3.y * inv));
      if (a.q) {
        if (in && i < rows_here) *reinterpret_cast<uint2*>(q) = o[i];
        q += a.ldq;
        if (cg == 0 && i < pads_here) qs[4 * i] = static_cast<uint8_t>(byte);
        if (qs_pad && i < pads_here) qs_pad[4 * i] = 127;
      }
    }
  }
  if (a.qt) {
    if (!SQUARE) {
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, cw[q], 16);
        cw[q] = sizeof(T) == 2 ? max_u16x2(cw[q], other) : max(cw[q], other);
      }
      if (lane < 16) {
#pragma unroll
        for (int q = 0; q < W; q += 4)
          *reinterpret_cast<uint4*>(&cmax[warp][cg][q]) = make_uint4(cw[q], cw[q + 1], cw[q + 2], cw[q + 3]);
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w)
#pragma unroll
        for (int q = 0; q < W; q += 4) {
          const uint4 o = *reinterpret_cast<const uint4*>(&cmax[w][cg][q]);
          const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) cw[q + k] = sizeof(T) == 2 ? max_u16x2(cw[q + k], v[k]) : max(cw[q + k], v[k]);
        }
    }
    const long long cols4 = (a.cols + 3) & ~3LL, kend = (a.rows + 511) / 512 * 4;
    const bool last = (kbr + 1) * 128 >= a.rows;
    const int pads_here = static_cast<int>(max(0LL, min(8LL, cols4 - c0)));
    uint8_t* qs = a.qts + fp8_scale_offset(kbr, c0, cols4);
    uint8_t* qs_pad = last && rg > 0 && rg < 4 && kbr + rg < kend ? a.qts + fp8_scale_offset(kbr + rg, c0, cols4) : nullptr;
    if (SQUARE) {  // the same bytes, transposed four by four
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // columns 4 h .. 4 h + 3
        uint32_t t[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // rows 4 k .. 4 k + 3
          const uint32_t w0 = h ? o[4 * k].y : o[4 * k].x, w1 = h ? o[4 * k + 1].y : o[4 * k + 1].x;
          const uint32_t w2 = h ? o[4 * k + 2].y : o[4 * k + 2].x, w3 = h ? o[4 * k + 3].y : o[4 * k + 3].x;
          const uint32_t a0 = __byte_perm(w0, w1, 0x5140), a1 = __byte_perm(w0, w1, 0x7362);
          const uint32_t b0 = __byte_perm(w2, w3, 0x5140), b1 = __byte_perm(w2, w3, 0x7362);
          t[k][0] = __byte_perm(a0, b0, 0x5410);
          t[k][1] = __byte_perm(a0, b0, 0x7632);
          t[k][2] = __byte_perm(a1, b1, 0x5410);
          t[k][3] = __byte_perm(a1, b1, 0x7632);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) tile[cg * 8 + 4 * h + j][rg ^ cg] = make_uint2(t[0][j], t[1][j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t byte = j >= nc ? 127u : one;
      if (!SQUARE) {
        uint32_t m;
        if constexpr (sizeof(T) == 2) m = wide_bits(j & 1 ? cw[j >> 1] >> 16 : cw[j >> 1] & 0xffffu, T());
        else m = cw[j];
        byte = fp8_scale_byte(m, top);  // 127 past the last column, where all is 0
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = x.at(i, j);
        tile[cg * 8 + j][rg ^ cg] = fp8_pack8<E5M2>(u, fp8_inverse_scale(byte));
      }
      if (rg == 0 && j < pads_here) qs[4 * j] = static_cast<uint8_t>(byte);
      if (qs_pad && j < pads_here) qs_pad[4 * j] = 127;
    }
    __syncthreads();
    // 16 bytes per thread: 8 threads to a row of 128, rows of 16-byte multiples
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int cl = it * 32 + (threadIdx.x >> 3), slot = (threadIdx.x & 7) * 2;
      const long long c = kbc * 128 + cl, r = kbr * 128 + slot * 8;
      if (c < a.cols && r < a.rows) {
        const uint2 lo = tile[cl][slot ^ (cl >> 3)], hi = tile[cl][(slot + 1) ^ (cl >> 3)];
        *reinterpret_cast<uint4*>(a.qt + c * a.ldqt + r) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

template <typename T>
static cudaError_t launch_quantize(const Fp8QuantArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>((a.rows + 127) / 128));
  const auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, a); };
  if (a.fmt) return a.square ? go(fp8_quantize_kernel<T, true, true>) : go(fp8_quantize_kernel<T, true, false>);
  return a.square ? go(fp8_quantize_kernel<T, false, true>) : go(fp8_quantize_kernel<T, false, false>);
}

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dt, cudaStream_t st) {
  if (dt == MUON_BF16) return launch_quantize<__nv_bfloat16>(a, st);
  if (dt == MUON_FP16) return launch_quantize<__half>(a, st);
  return launch_quantize<float>(a, st);
}

}  // namespace muon
