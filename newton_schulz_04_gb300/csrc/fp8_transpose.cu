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

// That takes some 20 instructions a value.  Where the scales of a tile's rows lie near enough to its first row's, 16-bit types hold
// every value times 2^(s - first s) exactly, and two at a time take half of them.  The other way, a function of its own that
// costs this one no registers, is for the rest, and for tiles in which some column's largest magnitude is so small that
// its factor leaves the 16-bit type's range.  Where the first row's scale is 1, as that of zeros is, the next other one takes its place.
//
// e4m3 goes through fp16, to and from which the hardware converts: scales 2^14 below the first (values are multiples of 2^-9, fp16's
// of 2^-24) to 2^7 above it (values are at most 448).  e5m2 has fp16's exponents, which leaves no room for scales; its
// bits are those of a bf16 number times 2^-112, and within 2^100 the products stay normal.  What a column's factor below 1
// takes out of the normal range lies far below the 8-bit types' smallest values.
//
// 8192 x 4096 takes 18.9 us from e4m3 (53 % of the copy rate) and 24 from e5m2, and 42 and 45 where every tile turns out to need
// whole numbers: a tile's barriers and its loads are hidden by three others on the SM only, at 63 % of the issue slots.
template <bool E5M2>
struct Pairwise {  // e4m3
  using V = __half2;
  static constexpr int BELOW = 14, ABOVE = 7;                // the first row's scale
  static constexpr uint32_t LEAST = (127u - 6u) << 23;       // fp32 bits of a column's maximum
  static __device__ __forceinline__ V bits(uint32_t w) { return *reinterpret_cast<const V*>(&w); }
  static __device__ __forceinline__ V row_factor(int k) { return bits(((15u + k) << 10) * 0x10001u); }  // 2^k
  static __device__ __forceinline__ uint32_t column_factor(int k) { return (15 + max(-ABOVE, min(14, k))) << 10; }
  static __device__ __forceinline__ V decode(uint32_t two, V f) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
    return __hmul2(bits(h), f);
  }
  static __device__ __forceinline__ uint32_t encode(V v, V f) {
    const V p = __hmul2(v, f);
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&p)));
    return r;
  }
  static __device__ __forceinline__ float2 wide(V v) { return __half22float2(v); }
  static __device__ __forceinline__ bool bad(const uint2&) { return false; }  // a NaN's product is one
};
template <>
struct Pairwise<true> {  // e5m2
  using V = __nv_bfloat162;
  static constexpr int BELOW = 100, ABOVE = 14;
  static constexpr uint32_t LEAST = (127u - 60u) << 23;
  static __device__ __forceinline__ V bits(uint32_t w) { return *reinterpret_cast<const V*>(&w); }
  static __device__ __forceinline__ V row_factor(int k) { return bits(((127u + 112u + k) << 7) * 0x10001u); }  // 2^(112 + k)
  static __device__ __forceinline__ uint32_t column_factor(int k) { return (127 + max(-ABOVE, min(100, k))) << 7; }
  static __device__ __forceinline__ V decode(uint32_t two, V f) {
    const uint32_t t = __byte_perm(two, 0u, 0x1404);
    return __hmul2(bits((t & 0x80008000u) | ((t >> 3) & 0x0fe00fe0u)), f);
  }
  static __device__ __forceinline__ uint32_t encode(V v, V f) {
    const V p = __hmul2(v, f);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&p);
    unsigned short r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(__uint_as_float(w & 0xffff0000u)), "f"(__uint_as_float(w << 16)));
    return r;
  }
  static __device__ __forceinline__ float2 wide(V v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ bool bad(const uint2& q) {  // infinities and NaN have no such bits
    return (((q.x & 0x7f7f7f7fu) + 0x04040404u) | ((q.y & 0x7f7f7f7fu) + 0x04040404u)) & 0x80808080u;
  }
};

// A 128 x 128 tile to a CTA of 256 threads: 8 rows x 8 columns to a thread, 16 lanes to a row.
struct TransposeTile {
  uint2 slot[128][16];     // transposed bytes: [column][8-row slot, swizzled]
  uint32_t column[128];    // of column 8 g + j at j * 16 + g: its maximum
  uint32_t byte[128];      // and its scale byte
};
struct TransposePart {
  long long c0, r0, rows4;
  int nc, nr;              // columns and rows of the thread's that exist
  __device__ __forceinline__ TransposePart(const Fp8TransposeArgs& a)
      : c0(blockIdx.x * 128LL + (threadIdx.x & 15) * 8),
        r0(blockIdx.y * 128LL + (threadIdx.x >> 4) * 8),
        rows4((a.rows + 3) & ~3LL),
        nc(static_cast<int>(max(0LL, min(8LL, a.cols - c0)))),
        nr(static_cast<int>(max(0LL, min(8LL, a.rows - r0)))) {}
  __device__ __forceinline__ void load(const Fp8TransposeArgs& a, uint2 (&q)[8], uint32_t (&s)[8]) const {
    const uint8_t* p = a.q + (nc && nr ? r0 * a.ldq + c0 : 0);
    const uint8_t* ps = a.qs + (nr ? fp8_scale_offset(blockIdx.x, r0, rows4) : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = make_uint2(0u, 0u);
      s[i] = i < nr ? ps[4 * i] : 0u;
      if (i < nr && nc == 8) {
        q[i] = *reinterpret_cast<const uint2*>(p);
      } else if (i < nr) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < nc) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
        q[i] = make_uint2(w[0], w[1]);
      }
      p += a.ldq;
    }
  }
};

// The first scale byte of the tile's rows that is not `base`, or base: a row of zeros has scale 1, which says nothing of the others.
__device__ __forceinline__ uint32_t other_scale(const Fp8TransposeArgs& a, uint32_t base) {
  const long long rows4 = (a.rows + 3) & ~3LL, row0 = blockIdx.y * 128LL;
#pragma unroll 1
  for (int k = 0; k < 128; k += 32) {
    const long long row = row0 + k + threadIdx.x % 32;
    const uint32_t s = row < a.rows ? a.qs[fp8_scale_offset(blockIdx.x, row, rows4)] : base;
    const uint32_t found = __ballot_sync(0xffffffffu, s != base);
    if (found) return __shfl_sync(0xffffffffu, s, __ffs(found) - 1);
  }
  return base;
}

// Any scales: fills the tile and the columns' scale bytes.
template <bool E5M2>
__device__ __noinline__ void transpose_any(const Fp8TransposeArgs& a, TransposeTile& tile) {
  constexpr int TOP = E5M2 ? 15 : 8;
  constexpr uint32_t BAD = E5M2 ? 0x04040404u : 0x01010101u;  // added to magnitudes, sets bit 7 of infinities and NaN
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  const TransposePart part(a);
  uint2 q[8];
  uint32_t s[8];
  if (threadIdx.x < 128) tile.column[threadIdx.x] = 0u;
  __syncthreads();
  part.load(a, q, s);
  uint32_t bad = 0u;  // bit j: column j holds an infinity or NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = ((q[i].x & 0x7f7f7f7fu) + BAD) & 0x80808080u, y = ((q[i].y & 0x7f7f7f7fu) + BAD) & 0x80808080u;
    if ((x | y) || s[i] == 255u) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < part.nc && (s[i] == 255u || ((j < 4 ? x : y) >> (8 * (j & 3)) & 0x80u))) bad |= 1u << j;
    }
  }
  // the keys of two columns of a row, 0 for 0; they pass 2^31
  const auto keys = [&](int j, int i, uint32_t (&k)[2]) {
    const uint32_t two = (j < 4 ? q[i].x : q[i].y) >> (8 * (j & 2));
    const float2 f = fp8_unpack2<E5M2>(two);
    const uint32_t x = abs_bits(f.x), y = abs_bits(f.y);
    k[0] = x ? x + (s[i] << 23) : 0u;
    k[1] = y ? y + (s[i] << 23) : 0u;
  };
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    uint32_t m0 = 0u, m1 = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t k[2];
      keys(j, i, k);
      m0 = max(m0, k[0]);
      m1 = max(m1, k[1]);
    }
    if (bad >> j & 1) m0 = 0xffffffffu;
    if (bad >> j & 2) m1 = 0xffffffffu;
    const bool up = threadIdx.x & 16;  // the half-warps hold other rows of the same columns: each takes one of two on
    const uint32_t m = max(up ? m1 : m0, __shfl_xor_sync(0xffffffffu, up ? m0 : m1, 16));
    atomicMax(&tile.column[(j + up) * 16 + cg], m);
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    const uint32_t m = tile.column[threadIdx.x];
    uint32_t byte = 127u;
    if (m == 0xffffffffu) byte = 255u;
    else if (m) byte = static_cast<uint32_t>(max(static_cast<int>((m + 0x1fffffu) >> 23) - 127 - TOP, 0));
    tile.byte[threadIdx.x] = byte;
  }
  __syncthreads();
  // computed again: 128 keys do not fit into registers, and the compiler would keep them
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(q[i].x), "+r"(q[i].y), "+r"(s[i]));
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t b0 = tile.byte[j * 16 + cg], b1 = tile.byte[(j + 1) * 16 + cg];
    uint32_t out[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float v[2][4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 4 * k + r;
        uint32_t key[2];
        keys(j, i, key);
        // exponents below fp32's end as 0 or subnormal, far below the 8-bit type's smallest value: where a column's scale is above a key
        const uint32_t raw = j < 4 ? q[i].x : q[i].y;
        v[0][r] = __uint_as_float((max(key[0], b0 << 23) - (b0 << 23)) | (raw << (24 - 8 * (j & 3)) & 0x80000000u));
        v[1][r] = __uint_as_float((max(key[1], b1 << 23) - (b1 << 23)) | (raw << (16 - 8 * (j & 3)) & 0x80000000u));
      }
      out[0][k] = b0 == 255u ? 0x7f7f7f7fu : fp8_pack4<E5M2>(v[0][0], v[0][1], v[0][2], v[0][3]);
      out[1][k] = b1 == 255u ? 0x7f7f7f7fu : fp8_pack4<E5M2>(v[1][0], v[1][1], v[1][2], v[1][3]);
    }
    tile.slot[cg * 8 + j][rg ^ cg] = make_uint2(out[0][0], out[0][1]);
    tile.slot[cg * 8 + j + 1][rg ^ cg] = make_uint2(out[1][0], out[1][1]);
  }
}

template <bool E5M2>
__global__ void __launch_bounds__(256, 4) fp8_transpose_kernel(const __grid_constant__ Fp8TransposeArgs a) {
  using Way = Pairwise<E5M2>;
  using V = typename Way::V;
  constexpr int TOP = E5M2 ? 15 : 8;
  __shared__ TransposeTile tile;
  __shared__ uint32_t factor[64];  // of column pair 4 g + k at k * 16 + g: 2^(first s - s')
  pdl_launch_dependents();
  if (threadIdx.x < 128) tile.column[threadIdx.x] = 0u;
  __syncthreads();
  pdl_wait();
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  V h[8][4];
  bool other = false;  // the other way
  uint32_t base = a.qs[fp8_scale_offset(blockIdx.x, blockIdx.y * 128LL, (a.rows + 3) & ~3LL)];
  {
    const TransposePart part(a);
    uint2 q[8];
    uint32_t s[8];
    part.load(a, q, s);
    if (base == 127u) base = other_scale(a, base);  // a row of zeros, perhaps
    V m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = Way::bits(0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = i < part.nr ? static_cast<int>(s[i]) - static_cast<int>(base) : 0;
      const bool zero = ((q[i].x | q[i].y) & 0x7f7f7f7fu) == 0u;  // zeros' scales, which are 1, are as good as any
      other |= (!zero && (d < -Way::BELOW || d > Way::ABOVE)) || s[i] == 255u || Way::bad(q[i]);
      const V f = Way::row_factor(max(-Way::BELOW, min(Way::ABOVE, d)));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[i][k] = Way::decode((k < 2 ? q[i].x : q[i].y) >> (16 * (k & 1)), f);
        m[k] = __hmax2_nan(m[k], __habs2(h[i][k]));
      }
    }
    const bool up = threadIdx.x & 16;  // the half-warps hold other rows of the same columns: each takes two words of four on
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const V keep = up ? m[k + 2] : m[k], give = up ? m[k] : m[k + 2];
      const float2 v = Way::wide(__hmax2_nan(keep, __shfl_xor_sync(0xffffffffu, give, 16)));
      const int j = 2 * k + (up ? 4 : 0);
      atomicMax(&tile.column[j * 16 + cg], abs_bits(v.x));
      atomicMax(&tile.column[(j + 1) * 16 + cg], abs_bits(v.y));
    }
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    const uint32_t mine = tile.column[threadIdx.x];
    other |= mine != 0u && mine < Way::LEAST;
    uint32_t byte = 127u;
    if (mine >= 0x7f800000u) byte = 255u;
    else if (mine) byte = static_cast<uint32_t>(max(static_cast<int>((mine + 0x1fffffu) >> 23) - TOP + static_cast<int>(base) - 127, 0));
    tile.byte[threadIdx.x] = byte;
    const int j = threadIdx.x / 16, g = threadIdx.x % 16;  // the factor of a column of zeros or NaN: any
    reinterpret_cast<unsigned short*>(factor)[((j / 2) * 16 + g) * 2 + (j & 1)] =
        static_cast<unsigned short>(Way::column_factor(static_cast<int>(base) - static_cast<int>(byte)));
  }
  const bool fast = !__syncthreads_or(other);
  if (fast) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint32_t b0 = tile.byte[j * 16 + cg], b1 = tile.byte[(j + 1) * 16 + cg];
      const V f = Way::bits(factor[j / 2 * 16 + cg]);
      uint32_t out[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = Way::encode(h[4 * k + r][j / 2], f);
        const uint32_t lo = __byte_perm(w[0], w[1], 0x5140), hi = __byte_perm(w[2], w[3], 0x5140);
        out[0][k] = b0 == 255u ? 0x7f7f7f7fu : __byte_perm(lo, hi, 0x5410);
        out[1][k] = b1 == 255u ? 0x7f7f7f7fu : __byte_perm(lo, hi, 0x7632);
      }
      tile.slot[cg * 8 + j][rg ^ cg] = make_uint2(out[0][0], out[0][1]);
      tile.slot[cg * 8 + j + 1][rg ^ cg] = make_uint2(out[1][0], out[1][1]);
    }
  } else {
    transpose_any<E5M2>(a, tile);
  }
  const long long cols4 = (a.cols + 3) & ~3LL, kend = (a.rows + 511) / 512 * 4, kbr = blockIdx.y;
  if (threadIdx.x < 128) {
    const long long c = blockIdx.x * 128LL + threadIdx.x % 16 * 8 + threadIdx.x / 16;
    if (c < cols4) {
      a.qts[fp8_scale_offset(kbr, c, cols4)] = static_cast<uint8_t>(tile.byte[threadIdx.x]);
      if ((kbr + 1) * 128 >= a.rows)
        for (long long kb = kbr + 1; kb < kend; ++kb) a.qts[fp8_scale_offset(kb, c, cols4)] = 127;
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 4; ++it) {  // 16 bytes per thread, 8 threads to a column
    const int cl = it * 32 + (threadIdx.x >> 3), slot = (threadIdx.x & 7) * 2;
    const long long c = blockIdx.x * 128LL + cl, r = kbr * 128 + slot * 8;
    if (c < a.cols && r < a.rows) {
      const uint2 lo = tile.slot[cl][slot ^ (cl >> 3)], hi = tile.slot[cl][(slot + 1) ^ (cl >> 3)];
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
