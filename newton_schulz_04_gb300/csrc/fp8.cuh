// fp8.cuh -- the 8-bit format with a power-of-two scale for each block of 128,
// and typed loads / stores of 8 consecutive elements.
//
// A block with largest magnitude A is stored as q = round8(x 2^-e) with the
// smallest e for which A 2^-e is at most the type's largest value, 448 (e4m3)
// or 57344 (e5m2).  Both are 1.75 * 2^k, so e comes from A's bits: its exponent
// minus k, plus one where its fraction is above 1.75.  Scaling by 2^-e is exact
// and no value saturates, so the only rounding is the one to 8 bits.  The scale
// is kept as the byte e + 127 (E8M0), which the tensor core applies itself.  A
// block of zeros has scale 1; one with an infinity or NaN has scale byte 255 and
// NaN elements, so that what reads it sees NaN.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "muon_ns.h"

namespace muon {

constexpr int kFp8Block = 128;

// Scale byte of a block from the largest magnitude's fp32 bits; `top` is 8 (e4m3) or 15 (e5m2).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits, int top) {
  if (amax_bits == 0u) return 127u;
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = static_cast<int>((amax_bits + 0x1fffffu) >> 23) - top;  // biased by 127
  return static_cast<uint32_t>(max(e, 0));
}
// 2^-e of a scale byte (NaN for 255).
__device__ __forceinline__ float fp8_inverse_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}
// Values to 8 bits, round to nearest even; the first in the low byte.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  uint32_t r;
  if (E5M2)
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e5m2x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
template <bool E5M2>
__device__ __forceinline__ uint2 fp8_pack8(const float (&v)[8], float inv) {
  return make_uint2(fp8_pack4<E5M2>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    fp8_pack4<E5M2>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
// What a scale byte stands for: 2^(b - 127), NaN for 255 (2^-127 is subnormal).
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 0x400000u : byte << 23);
}
// The same for reading values back that are used as they are: FLT_MAX and its neighbours are kept as 2^128, which under this
// factor, 2^-24 less for the scales that reach it, is FLT_MAX again.
template <bool E5M2>
__device__ __forceinline__ float fp8_finite_scale_value(uint32_t byte) {
  return byte > 254u - (E5M2 ? 15u : 8u) && byte != 255u ? __uint_as_float((byte << 23) - 1u) : fp8_scale_value(byte);
}
// Two 8-bit values as fp32, exactly; the first is the low byte.  (e5m2 is fp16 without its last 8 bits.)
template <bool E5M2>
__device__ __forceinline__ float2 fp8_unpack2(uint32_t two) {
  uint32_t h;
  if (E5M2) h = __byte_perm(two, 0u, 0x1404);
  else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 fp8_unpack2(uint32_t two, int fmt) {
  return fmt ? fp8_unpack2<true>(two) : fp8_unpack2<false>(two);
}
// Byte offset of the scale of block kb of row r; rows4 = rows rounded up to 4.
__host__ __device__ __forceinline__ long long fp8_scale_offset(long long kb, long long r, long long rows4) {
  return ((kb >> 2) * rows4 + r) * 4 + (kb & 3);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// ---- one element
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// One element of a product: out = round(v + add).
template <typename Args>
__device__ __forceinline__ void fp8_product_out(const Args& a, long long m, long long n, float v) {
  if (a.add) {
    const long long i = m * a.ldadd + n;
    v += a.out_dt == MUON_FP32   ? static_cast<const float*>(a.add)[i]
         : a.out_dt == MUON_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(a.add)[i])
                                 : to_f32(static_cast<const __half*>(a.add)[i]);
  }
  const long long o = m * a.ldc + n;
  if (a.out_dt == MUON_FP32) static_cast<float*>(a.out)[o] = v;
  else if (a.out_dt == MUON_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = from_f32<__nv_bfloat16>(v);
  else static_cast<__half*>(a.out)[o] = from_f32<__half>(v);
}

// ---- 8 consecutive elements; `full`: all in range and 16-byte aligned
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8], __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8], __half) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void load8_full(const T* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v, T());
}
template <>
__device__ __forceinline__ void load8_full<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// n valid elements (0 .. 8); the others are 0.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool full, float (&v)[8]) {
  if (full) {
    load8_full(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8_full(T* p, const float (&v)[8]) {
  union {
    uint4 w;
    T e[8];
  } u;
#pragma unroll
  for (int i = 0; i < 8; ++i) u.e[i] = from_f32<T>(v[i]);
  *reinterpret_cast<uint4*>(p) = u.w;
}
template <>
__device__ __forceinline__ void store8_full<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool full, const float (&v)[8]) {
  if (full) {
    store8_full(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

}  // namespace muon
