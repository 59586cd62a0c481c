// fp8_transpose.cu -- an 8-bit matrix with scales along its columns as the transposed one, with scales along its rows.
//
//   value = q 2^(s - 127)       s' = the scale byte of the column's 128 values       q' = round8(value 2^(127 - s'))
//
// Values and scales are compared and rescaled as whole numbers: an 8-bit value is a normal fp32 number, and adding s to its
// exponent field gives a 32-bit key that orders magnitudes over the scales' whole range (2^-127 to 2^127 times the type's
// own) and from which subtracting s' leaves the fp32 bits to round.  Scaling by powers of two is exact, so q' differs from
// q only in the exponent, but for values that fall below the type's normal range.
#include <cuda_runtime.h>

#include "block_norm.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace muon {

// A 128 x 128 tile to a CTA of 256 threads, 8 rows x 8 columns to a thread.
template <bool E5M2>
__global__ void __launch_bounds__(256, 2) fp8_transpose_kernel(const Fp8TransposeArgs a) {
  __shared__ uint2 tile[128][16];  // transposed bytes: [column][8-row slot, swizzled]
  __shared__ uint32_t cmax[128];
  constexpr uint32_t bad_from = E5M2 ? 0x04040404u : 0x01010101u;  // added to magnitudes, sets bit 7 of infinities and NaN
  pdl_launch_dependents();
  if (threadIdx.x < 128) cmax[threadIdx.x] = 0u;
  __syncthreads();
  pdl_wait();
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const long long kbc = blockIdx.x, kbr = blockIdx.y, c0 = kbc * 128 + cg * 8, r0 = kbr * 128 + rg * 8;
  const long long rows4 = (a.rows + 3) & ~3LL, cols4 = (a.cols + 3) & ~3LL, kend = (a.rows + 511) / 512 * 4;
  const int nc = static_cast<int>(max(0LL, min(8LL, a.cols - c0)));
  uint2 q[8];
  uint32_t s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long row = r0 + i;
    const int n = row < a.rows ? nc : 0;
    const uint8_t* p = a.q + (n ? row * a.ldq + c0 : 0);
    if (n == 8) {
      q[i] = *reinterpret_cast<const uint2*>(p);
    } else {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
      q[i] = make_uint2(w[0], w[1]);
    }
    s[i] = n ? a.qs[fp8_scale_offset(kbc, row, rows4)] : 0u;
  }
  uint32_t cm[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0u;
  const auto key = [&](int i, int j) {  // exponent field plus scale, fraction; 0 for 0
    const uint32_t two = (j < 4 ? q[i].x : q[i].y) >> (16 * ((j >> 1) & 1));
    const float2 f = fp8_unpack2<E5M2>(two);
    const uint32_t b = abs_bits(j & 1 ? f.y : f.x);
    return b ? b + (s[i] << 23) : 0u;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = (((q[i].x & 0x7f7f7f7fu) + bad_from) | ((q[i].y & 0x7f7f7f7fu) + bad_from)) & 0x80808080u;
    if (w || s[i] == 255u) {  // the columns' blocks become NaN
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = ((j < 4 ? q[i].x : q[i].y) >> (8 * (j & 3))) & 0x7fu;
        if (j < nc && (s[i] == 255u || b + (bad_from & 0xffu) >= 0x80u)) cm[j] = 0xffffffffu;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], key(i, j));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
    if ((threadIdx.x & 16) == 0) atomicMax(&cmax[cg * 8 + j], cm[j]);
  }
  __syncthreads();
  const bool bottom = (kbr + 1) * 128 >= a.rows;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t m = cmax[cg * 8 + j];
    uint32_t byte = 127u;
    if (m == 0xffffffffu) byte = 255u;
    else if (m) byte = static_cast<uint32_t>(max(static_cast<int>((m + 0x1fffffu) >> 23) - 127 - (E5M2 ? 15 : 8), 0));
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = 4 * h + k;
        // exponents below fp32's end as 0 or subnormal, far below the 8-bit type's smallest value
        const uint32_t b = static_cast<uint32_t>(max(static_cast<int>(key(i, j) - (byte << 23)), 0));
        const uint32_t raw = (j < 4 ? q[i].x : q[i].y) >> (8 * (j & 3));
        v[k] = __uint_as_float(b | (raw & 0x80u) << 24);
      }
      out[h] = byte == 255u ? 0x7f7f7f7fu : fp8_pack4<E5M2>(v[0], v[1], v[2], v[3]);
    }
    tile[cg * 8 + j][rg ^ cg] = make_uint2(out[0], out[1]);
    if (rg == 0 && c0 + j < cols4) {
      a.qts[fp8_scale_offset(kbr, c0 + j, cols4)] = static_cast<uint8_t>(byte);
      if (bottom)
        for (long long kb = kbr + 1; kb < kend; ++kb) a.qts[fp8_scale_offset(kb, c0 + j, cols4)] = 127;
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 4; ++it) {  // 16 bytes per thread, 8 threads to a column
    const int cl = it * 32 + (threadIdx.x >> 3), slot = (threadIdx.x & 7) * 2;
    const long long c = kbc * 128 + cl, r = kbr * 128 + slot * 8;
    if (c < a.cols && r < a.rows) {
      const uint2 lo = tile[cl][slot ^ (cl >> 3)], hi = tile[cl][(slot + 1) ^ (cl >> 3)];
      *reinterpret_cast<uint4*>(a.qt + c * a.ldqt + r) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

cudaError_t launch_fp8_transpose(const Fp8TransposeArgs& a, int fmt, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.cols + 127) / 128), static_cast<unsigned>((a.rows + 127) / 128));
  return fmt ? launch_pdl(fp8_transpose_kernel<true>, grid, dim3(256), 0, st, a)
             : launch_pdl(fp8_transpose_kernel<false>, grid, dim3(256), 0, st, a);
}

}  // namespace muon
