// fp8_transpose.cu -- an 8-bit matrix with scales along its columns as the transposed one, with scales along its rows.
//
//   value = q 2^(s - 127)       s' = the scale byte of the column's 128 values       q' = round8(value 2^(127 - s'))
//
// Values and scales are compared and rescaled as whole numbers: an 8-bit value is a normal fp32 number, and adding s to its
// exponent field gives a 32-bit key that orders magnitudes over the scales' whole range (2^-127 to 2^127 times the type's
// own) and from which subtracting s' leaves the fp32 bits to round.  Scaling by powers of two is exact, so q' differs from
// q only in the exponent, but for values that fall below the type's normal range.
#include <cuda_runtime.h>

#include "kernels.h"
#include "pairs.cuh"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

// A 128 x 128 tile to a CTA of 256 threads: 8 rows x 8 columns to a thread, 16 lanes to a row.
template <bool E5M2>
__global__ void __launch_bounds__(256, 3) fp8_transpose_kernel(const Fp8TransposeArgs a) {
  __shared__ uint2 tile[128][16];  // transposed bytes: [column][8-row slot, swizzled]
  __shared__ uint32_t cmax[128];   // of column 8 g + j at j * 16 + g
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
  uint32_t bad = 0u;  // bit j: column j holds an infinity or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = ((q[i].x & 0x7f7f7f7fu) + bad_from) & 0x80808080u, y = ((q[i].y & 0x7f7f7f7fu) + bad_from) & 0x80808080u;
    if ((x | y) || s[i] == 255u) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < nc && (s[i] == 255u || ((j < 4 ? x : y) >> (8 * (j & 3)) & 0x80u))) bad |= 1u << j;
    }
  }
  // Two columns at a time: the signed keys of their 8 rows, 0 for 0.
  const auto keys = [&](int j, int i, int (&k)[2]) {
    const uint32_t two = (j < 4 ? q[i].x : q[i].y) >> (8 * (j & 2));
    const float2 f = fp8_unpack2<E5M2>(two);
    const uint32_t x = abs_bits(f.x), y = abs_bits(f.y);
    k[0] = x ? static_cast<int>(x + (s[i] << 23)) : 0;
    k[1] = y ? static_cast<int>(y + (s[i] << 23)) : 0;
  };
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint32_t m0 = 0u, m1 = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int k[2];
      keys(j, i, k);
      m0 = max(m0, static_cast<uint32_t>(k[0]));
      m1 = max(m1, static_cast<uint32_t>(k[1]));
    }
    if (bad >> j & 1) m0 = 0xffffffffu;
    if (bad >> j & 2) m1 = 0xffffffffu;
    // the two half-warps hold other rows of the same columns: each takes one of the two on
    const bool up = threadIdx.x & 16;
    const uint32_t m = max(up ? m1 : m0, __shfl_xor_sync(0xffffffffu, up ? m0 : m1, 16));
    atomicMax(&cmax[(j + up) * 16 + cg], m);
  }
  __syncthreads();
  if (threadIdx.x < 128) {  // a scale byte for each column
    const uint32_t m = cmax[threadIdx.x];
    uint32_t byte = 127u;
    if (m == 0xffffffffu) byte = 255u;
    else if (m) byte = static_cast<uint32_t>(max(static_cast<int>((m + 0x1fffffu) >> 23) - 127 - (E5M2 ? 15 : 8), 0));
    cmax[threadIdx.x] = byte;
    const long long c = kbc * 128 + threadIdx.x % 16 * 8 + threadIdx.x / 16;
    if (c < cols4) {
      a.qts[fp8_scale_offset(kbr, c, cols4)] = static_cast<uint8_t>(byte);
      if ((kbr + 1) * 128 >= a.rows)
        for (long long kb = kbr + 1; kb < kend; ++kb) a.qts[fp8_scale_offset(kb, c, cols4)] = 127;
    }
  }
  __syncthreads();
  // computed again: 128 keys do not fit into registers, and the compiler would keep them
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(q[i].x), "+r"(q[i].y), "+r"(s[i]));
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t b0 = cmax[j * 16 + cg], b1 = cmax[(j + 1) * 16 + cg];
    uint32_t out[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[2][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 4 * h + r;
        int k[2];
        keys(j, i, k);
        // exponents below fp32's end as 0 or subnormal, far below the 8-bit type's smallest value
        const uint32_t raw = j < 4 ? q[i].x : q[i].y;
        v[0][r] = __uint_as_float(static_cast<uint32_t>(max(k[0] - static_cast<int>(b0 << 23), 0)) | (raw << (24 - 8 * (j & 3)) & 0x80000000u));
        v[1][r] = __uint_as_float(static_cast<uint32_t>(max(k[1] - static_cast<int>(b1 << 23), 0)) | (raw << (16 - 8 * (j & 3)) & 0x80000000u));
      }
      out[0][h] = b0 == 255u ? 0x7f7f7f7fu : fp8_pack4<E5M2>(v[0][0], v[0][1], v[0][2], v[0][3]);
      out[1][h] = b1 == 255u ? 0x7f7f7f7fu : fp8_pack4<E5M2>(v[1][0], v[1][1], v[1][2], v[1][3]);
    }
    tile[cg * 8 + j][rg ^ cg] = make_uint2(out[0][0], out[0][1]);
    tile[cg * 8 + j + 1][rg ^ cg] = make_uint2(out[1][0], out[1][1]);
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
