// pairs.cuh -- a thread's piece of a row as pairs of fp32 values (sm_100's two-wide FMA, multiplication and addition halve the
// instructions of what is bound by issuing them), and the exchange by which a row's 8-bit copies get their scales.
#pragma once
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "ptx.cuh"
#include "row_ring.cuh"

namespace muon {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ uint32_t pack2(float2 v, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float2 v, __half) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes of T.
template <typename T>
struct Pairs {
  static constexpr int E = 16 / static_cast<int>(sizeof(T)), N = E / 2;
  float2 v[N];
  __device__ __forceinline__ void unpack(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = unpack2(u[i], T());
    } else {
      v[0] = make_float2(__uint_as_float(u[0]), __uint_as_float(u[1]));
      v[1] = make_float2(__uint_as_float(u[2]), __uint_as_float(u[3]));
    }
  }
  // E bytes of 8-bit values
  template <bool E5M2>
  __device__ __forceinline__ void unpack8(const uint8_t* p) {
    uint32_t w[E / 4];
    if constexpr (E == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fp8_unpack2<E5M2>(w[i / 2] >> (16 * (i & 1)));
  }
  __device__ __forceinline__ uint4 packed() const {
    if constexpr (sizeof(T) == 2) return make_uint4(pack2(v[0], T()), pack2(v[1], T()), pack2(v[2], T()), pack2(v[3], T()));
    else return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  }
  // n of the elements exist.
  __device__ __forceinline__ void store(T* p, int n) const {
    if (n == E) {
      *reinterpret_cast<uint4*>(p) = packed();
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (2 * i < n) p[2 * i] = from_f32<T>(v[i].x);
        if (2 * i + 1 < n) p[2 * i + 1] = from_f32<T>(v[i].y);
      }
    }
  }
  // fp32 bits of the largest magnitude; a NaN's are above all others
  __device__ __forceinline__ uint32_t largest() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(v[i].x)), "f"(fabsf(v[i].y)));
    return __float_as_uint(m);
  }
  template <bool E5M2>
  __device__ __forceinline__ void store8(uint8_t* p, float inv) const {
    float2 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = mul2(v[i], both(inv));
    if constexpr (E == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(fp8_pack4<E5M2>(s[0].x, s[0].y, s[1].x, s[1].y),
                                                fp8_pack4<E5M2>(s[2].x, s[2].y, s[3].x, s[3].y));
    } else {
      *reinterpret_cast<uint32_t*>(p) = fp8_pack4<E5M2>(s[0].x, s[0].y, s[1].x, s[1].y);
    }
  }
  __device__ __forceinline__ void store8(uint8_t* p, float inv, int fmt) const {
    if (fmt) store8<true>(p, inv);
    else store8<false>(p, inv);
  }
};

// Pieces that hold every column are summed as pairs, too.
__device__ __forceinline__ float total(float2 v) { return v.x + v.y; }

// exp(-g) of a pair and, of it, the sigmoid 1 / (1 + exp(-g)), 0 at -infinity and from about g = -87 on.  fp32 data takes the
// accurate exponential and quotient, and so does a gate of a whole row, whose error all its elements share; 16-bit data, which
// is rounded by 2^-11 at best, the hardware's: the sigmoid is off by (4 + 1.2 |g|) 2^-23 of the value.
template <typename T>
__device__ __forceinline__ float2 exp_minus2(float2 g) {
  if constexpr (sizeof(T) == 4) {
    return make_float2(expf(-g.x), expf(-g.y));
  } else {
    float2 e = mul2(g, both(-1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    return e;
  }
}
template <typename T>
__device__ __forceinline__ float2 sigmoid_of2(float2 e) {
  e = add2(e, both(1.f));
  if constexpr (sizeof(T) == 4) {
    return make_float2(1.f / e.x, 1.f / e.y);
  } else {
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
    return r;
  }
}
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 g) {
  return sigmoid_of2<T>(exp_minus2<T>(g));
}
// 1 - s for a derivative, which is multiplied by s: as the product, since the difference of an open gate keeps nothing of it.
// Where exp(-g) is infinite s is 0, and this any finite number.
__device__ __forceinline__ float2 shut2(float2 e, float2 s) {
  return mul2(make_float2(fminf(e.x, 3.402823466e38f), fminf(e.y, 3.402823466e38f)), s);
}

// ---- rows that do not start on 16 bytes
// 16 bytes from byte o (0 .. 15, the same in all lanes) of the 32 bytes lo, hi.
__device__ __forceinline__ uint4 window(const uint4& lo, const uint4& hi, int o) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const bool eight = o & 8, four = o & 4;
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = eight ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = four ? w[i + 1] : w[i];
  const int bits = 8 * (o & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                    __funnelshift_r(w[3], w[4], bits));
}
// A matrix whose rows start anywhere: its memory's ends, so that whole 16 bytes are read only where they lie within.
struct Span {
  const uint8_t *from, *to;
  template <typename T>
  static __device__ __forceinline__ Span of(const void* p, long long rows, long long cols, long long ld) {
    const uint8_t* b = static_cast<const uint8_t*>(p);
    return {b, b + ((rows - 1) * ld + cols) * static_cast<long long>(sizeof(T))};
  }
};
// Piece t of a row of `cols` columns, of which `left` = cols - t E (0 or less: none) are there from its first on: from the four
// or five aligned words that it lies in, which neighbouring lanes' loads share in L1.  Loading and using are apart, so that a
// thread's loads are under way together.
template <typename T>
struct LoadAnywhere {
  uint32_t w[5];
  int bits;
  __device__ __forceinline__ void load(const T* row, int t, int left, const Span& s) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    const uint8_t* piece = reinterpret_cast<const uint8_t*>(row) + 16LL * t;
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(piece) & 3);
    const uint8_t* p = piece - odd;
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = 0u;
    bits = 0;
    if (left >= E && p >= s.from && p + 20 <= s.to) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = q[i];
      bits = 8 * odd;
    } else if (left > 0) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i < left) {
          const T v = reinterpret_cast<const T*>(piece)[i];
          if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v);
          else w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(&v)) << (16 * (i & 1));
        }
      }
    }
  }
  __device__ __forceinline__ uint4 get() const {
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
  }
};
// And written, by LANES neighbouring lanes with neighbouring pieces: what a neighbour has of a lane's aligned 16 bytes comes from
// it; the lanes at the ends write the rest themselves.  All lanes of a warp call.
template <typename T, int LANES>
__device__ __forceinline__ void store_anywhere(T* row, int t, int left, const Pairs<T>& v) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15), lane = threadIdx.x % LANES;
  union {
    uint4 w;
    T e[E];
  } u;
  u.w = v.packed();
  const uint4 before = make_uint4(__shfl_up_sync(0xffffffffu, u.w.x, 1, LANES), __shfl_up_sync(0xffffffffu, u.w.y, 1, LANES),
                                  __shfl_up_sync(0xffffffffu, u.w.z, 1, LANES), __shfl_up_sync(0xffffffffu, u.w.w, 1, LANES));
  const int head = E - off / static_cast<int>(sizeof(T));  // elements of the piece in its first 16 aligned bytes
  uint8_t* p = reinterpret_cast<uint8_t*>(row) - off + 16LL * t;
  const bool whole = left >= head && (lane > 0 || off == 0);
  if (whole) *reinterpret_cast<uint4*>(p) = off ? window(before, u.w, 16 - off) : u.w;
  // the rest, a bit for each element: before the first lane's next 16 bytes, behind the last one's, and a row's end
  const uint32_t first = (1u << head) - 1u, there = (1u << max(0, min(E, left))) - 1u;
  const uint32_t rest = there & ((whole ? 0u : first) | (lane == LANES - 1 || left - E < head ? ~first : 0u));
  if (rest) {
    row += t * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (rest >> i & 1u) row[i] = u.e[i];
  }
}

// A warp's slot of one array and piece in a ring, for rows that start anywhere: the 16 aligned bytes of each of a row's LANES
// lanes and one more, from which a lane takes its own by `window`.  The warp is synchronised before it reads and before
// it fetches into the same slot again.
template <int LANES>
constexpr int kWarpSlot = 32 / LANES * (LANES + 1) * 16;
template <typename T, int LANES>
__device__ __forceinline__ void fetch_anywhere(uint8_t* slot, const T* row, int t, int cols, const uint8_t* from) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15), lane = threadIdx.x % LANES;
  slot += (threadIdx.x % 32 / LANES * (LANES + 1) + lane) * 16;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(row) - off + 16LL * t;
  const int there = cols * static_cast<int>(sizeof(T)) + off - 16 * t;  // bytes to the row's end
  if (p < from && there > 0) {  // the matrix begins within these 16 bytes
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int at = i * static_cast<int>(sizeof(T));
      reinterpret_cast<T*>(slot)[i] = at >= off && at < there ? *reinterpret_cast<const T*>(p + at) : from_f32<T>(0.f);
    }
  } else if (there > 0) {
    copy16(smem_u32(slot), p, min(16, there));
  } else {
    *reinterpret_cast<uint4*>(slot) = make_uint4(0u, 0u, 0u, 0u);
  }
  if (lane == LANES - 1) {
    if (there > 16) copy16(smem_u32(slot + 16), p + 16, min(16, there - 16));
    else *reinterpret_cast<uint4*>(slot + 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}
// off: the row's address modulo 16.  By WORDS, four lanes of which share a bank, or as two accesses of 16 bytes and the choice
// among their words, which takes twice the instructions and less than half of shared memory's time: the norms, which read
// three arrays and are bound by issuing, are 10 us of 33.5M elements faster with the first, their gradient, which reads
// five, 14 with the second.
template <int LANES, bool WORDS>
__device__ __forceinline__ uint4 read_anywhere(const uint8_t* slot, int off) {
  slot += (threadIdx.x % 32 / LANES * (LANES + 1) + threadIdx.x % LANES) * 16;
  if constexpr (WORDS) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(slot + (off & 12));
    const int bits = 8 * (off & 3);
    const uint32_t w[5] = {q[0], q[1], q[2], q[3], off & 3 ? q[4] : 0u};
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
  } else {
    return window(reinterpret_cast<const uint4*>(slot)[0], reinterpret_cast<const uint4*>(slot)[1], off);
  }
}

// The fp32 bits of two magnitudes, a in the lower half, as words of 16 bits that order them and give the same scale bytes: the
// upper bits, rounded up.  A scale byte is the exponent field of bits + 0x1fffff, and the only border within a binade,
// 0x600000, is a multiple of 2^16.  Finite magnitudes stay below infinity: those above 0x7f7f0000 have the byte of 0x7f7f0000.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  constexpr uint32_t LAST = 0x7f7fffffu;  // FLT_MAX; infinity and NaN are above it and stay as they are
  return __byte_perm(max(__viaddmin_u32(a, 0xffffu, LAST), a), max(__viaddmin_u32(b, 0xffffu, LAST), b), 0x7632);
}
// The same of 16-bit types' values, none of which lies between 0x7f7f0000 and infinity.
__device__ __forceinline__ uint32_t upper_halves16(uint32_t a, uint32_t b) { return __byte_perm(a + 0xffffu, b + 0xffffu, 0x7632); }

// Scales of up to four matrices' blocks, whose 128 columns lie in LANES = 16 or 32 neighbouring lanes.  The largest
// magnitudes travel two to a word.  A quarter of the lanes ends up with one matrix each, computes its byte, keeps it and hands
// the others its inverse: a third of the instructions of four exchanges in all lanes.  INPUTS16: the last two hold a 16-bit type's
// values.
template <int LANES, bool INPUTS16>
struct Scales4 {
  static constexpr int Q = LANES / 4;
  uint32_t byte;   // of matrix (lane / Q) % 4
  float inv[4];
  static __device__ __forceinline__ int mine() { return (threadIdx.x / Q) % 4; }
  // m: fp32 bits of the lane's largest magnitudes; top: 8 or 15 for the matrix mine() says
  __device__ __forceinline__ Scales4(const uint32_t (&m)[4], int top) {
    const int lane = threadIdx.x % 32;
    const uint32_t ab = upper_halves(m[0], m[1]), cd = INPUTS16 ? upper_halves16(m[2], m[3]) : upper_halves(m[2], m[3]);
    const bool up = lane & (2 * Q);
    uint32_t w = __vmaxu2(up ? cd : ab, __shfl_xor_sync(0xffffffffu, up ? ab : cd, 2 * Q));
#pragma unroll
    for (int o = Q; o > 0; o >>= 1) w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, o));
    byte = fp8_scale_byte(lane & Q ? w & 0xffff0000u : w << 16, top);
    const float mine_inv = fp8_inverse_scale(byte);
#pragma unroll
    for (int k = 0; k < 4; ++k) inv[k] = __shfl_sync(0xffffffffu, mine_inv, (lane & ~(LANES - 1)) + k * Q);
  }
};

}  // namespace muon
