// fp8_few.cu -- the 8-bit product C = A B^T (+ D) of at most 8 rows of A: single tokens and small batches.
//
// The formula is fp8_gemm.cu's, but every byte of B serves a few products only: the bytes of B bound it, and
// tiles of 256 rows of B on pairs of SMs leave most of the GPU idle where B is small.  Here a CTA takes 16 rows of B and its
// warps a part of K each, straight from memory to registers: no tensor map, cluster or TMEM to set up.
// mma.m16n8k16 multiplies the values as fp16, which holds every 8-bit value exactly, with sums in
// fp32; a block of 128 of K is summed from zero and added to the row's sum times 2^(ea + eb).  Any order of
// K within a block will do as long as both operands have the same, so a thread loads 16
// consecutive bytes of a row and takes them as four fragments' pairs.  The warps' sums are added up in
// their order: the same bits every time.
//
// Taken while all CTAs are resident at once, two of 8 warps on an SM with 111 registers a thread.  Device times in us, this
// kernel and fp8_gemm.cu's, one token: 300 x 4096 2.8 and 5.0; 1024 x 4096 3.0 and 5.0; 2500 x 2500 3.7 and
// 6.5; 4096 x 4096 5.4 (3.1 TB/s, 4.2 with B partly in L2) and 7.3; 4096 x 14336 13.6 (4.3 TB/s) and 15.0; 256 x
// 65536 23.8 and 25.0; 4864 x 512 1.9 and 3.3; 4864 x 14336 15.0 and 15.9, with 8 rows 15.0 and 16.3.  Beyond,
// stepping over the tiles: 6144 x 4096 8.3 and 8.1; 8192 x 8192 15.5 and 14.1; 28672 x 4096 22.1 and 20.8.
// Two blocks of a warp in flight are 64 KB on an SM.  Slower were: the conversion's bits moved by integer
// instructions, 7.9 at 4096 x 4096; four blocks in flight in a ring of cp.async copies, 6.2; the 8-bit
// mma.sync there, 6.1; one chain of eight products a block instead of two of four, 5.6.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

struct FewArgs {
  const uint8_t *x, *w;    // [m][ldx], [n][ldw]
  const uint8_t *sx, *sw;  // scale bytes
  long long ldx, ldw, sx_rows, sw_rows, n, k;
  int m, kblocks, per_warp;  // blocks of 128 of K, and of a warp
  const void* add;
  void* out;
  long long ldadd, ldc;
  int out_dt;
};

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// The first `left` of 16 bytes, the rest 0; nothing past them is read.
__device__ __noinline__ uint4 load_part(const uint8_t* p, int left) {
  uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < left) v[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// Four 8-bit values to two pairs of fp16.
template <bool E5M2>
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (E5M2)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e5m2x2 %0, l;\n\tcvt.rn.f16x2.e5m2x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// v 2^(e - 254), e the sum of two scale bytes, with two factors: the product of the scales may leave fp32's range
// where the result does not.  NaN if one of them is.
__device__ __forceinline__ float scaled(float v, uint32_t a, uint32_t b) {
  const int e = static_cast<int>(a + b) - 254, h = e >> 1;
  const float r = v * __uint_as_float(static_cast<uint32_t>(h + 127) << 23) *
                  __uint_as_float(static_cast<uint32_t>(e - h + 127) << 23);
  return a == 255u || b == 255u ? __uint_as_float(0x7fffffffu) : r;
}

// What a thread holds of a block of K: 2 x 16 bytes of rows g and g + 8 of B and of row g of A, and
// the scale bytes of its four sums.
struct FewBlock {
  uint4 w[2][2], x[2];
  uint32_t sw[2], sx[2];
};

template <bool A5, bool B5>
__global__ void __launch_bounds__(512, 1) fp8_few_kernel(const FewArgs a) {
  __shared__ float sums[16][8 * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warps = blockDim.x >> 5;
  const int kb0 = warp * a.per_warp, blocks = max(0, min(a.kblocks - kb0, a.per_warp));
  const long long n0 = blockIdx.x * 16LL, r0 = min(n0 + g, a.n - 1), r1 = min(n0 + g + 8, a.n - 1);
  // a thread without a row of A reads none, one without a sum of A's rows takes the first's scale
  const bool token = g < a.m;
  const uint8_t *p0 = a.w + r0 * a.ldw, *p1 = a.w + r1 * a.ldw, *px = a.x + (token ? g : 0) * a.ldx;
  const uint8_t *s0 = a.sw + r0 * 4, *s1 = a.sw + r1 * 4;
  const uint8_t *sx0 = a.sx + (2 * t < a.m ? 8 * t : 0), *sx1 = a.sx + (2 * t + 1 < a.m ? 8 * t + 4 : 0);
  pdl_wait();
  pdl_launch_dependents();

  auto load = [&](int j, FewBlock& f) {
    if (j >= blocks) return;
    const long long kb = kb0 + j;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const long long at = kb * 128 + q * 64 + t * 16;
      if (at + 16 <= a.k) {
        f.w[q][0] = load_once(p0 + at);
        f.w[q][1] = load_once(p1 + at);
        f.x[q] = token ? __ldg(reinterpret_cast<const uint4*>(px + at)) : make_uint4(0, 0, 0, 0);
      } else {
        const int some = static_cast<int>(max(0LL, a.k - at));
        f.w[q][0] = load_part(p0 + at, some);
        f.w[q][1] = load_part(p1 + at, some);
        f.x[q] = load_part(px + at, token ? some : 0);
      }
    }
    const long long gw = (kb >> 2) * (a.sw_rows * 4) + (kb & 3), gx = (kb >> 2) * (a.sx_rows * 4) + (kb & 3);
    f.sw[0] = __ldg(s0 + gw);
    f.sw[1] = __ldg(s1 + gw);
    f.sx[0] = __ldg(sx0 + gx);
    f.sx[1] = __ldg(sx1 + gx);
  };
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto use = [&](const FewBlock& f) {
    float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of four
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t w0[4] = {f.w[q][0].x, f.w[q][0].y, f.w[q][0].z, f.w[q][0].w};
        const uint32_t w1[4] = {f.w[q][1].x, f.w[q][1].y, f.w[q][1].z, f.w[q][1].w};
        const uint32_t x[4] = {f.x[q].x, f.x[q].y, f.x[q].z, f.x[q].w};
        uint32_t a0, a1, a2, a3, b0, b1;
        to_f16<B5>(w0[i], a0, a2);
        to_f16<B5>(w1[i], a1, a3);
        to_f16<A5>(x[i], b0, b1);
        mma_f16(d[q], a0, a1, a2, a3, b0, b1);
      }
    }
    // 2^(e - 254) is a normal number for e in 128 .. 254, and no sum with a NaN's 255 is among them
    const uint32_t e[4] = {f.sw[0] + f.sx[0], f.sw[0] + f.sx[1], f.sw[1] + f.sx[0], f.sw[1] + f.sx[1]};
    const uint32_t least = min(min(e[0], e[1]), min(e[2], e[3])), most = max(max(e[0], e[1]), max(e[2], e[3]));
    if (least >= 128u && most <= 254u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(d[0][i] + d[1][i], __uint_as_float((e[i] - 127u) << 23), acc[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += scaled(d[0][i] + d[1][i], f.sw[i >> 1], f.sx[i & 1]);
    }
  };

  FewBlock f0, f1;  // the next block's loads are on their way while one is used
  load(0, f0);
  load(1, f1);
  for (int j = 0; j < blocks; j += 2) {
    use(f0);
    load(j + 2, f0);
    if (j + 1 < blocks) use(f1);
    load(j + 3, f1);
  }
  // The warps' sums, added up in their order
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[warp][(2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[i];
  __syncthreads();
  const int m = threadIdx.x >> 4;
  const long long n = n0 + (threadIdx.x & 15);
  if (m < a.m && n < a.n) {
    float v = 0.f;
    for (int p = 0; p < warps; ++p) v += sums[p][threadIdx.x];
    fp8_product_out(a, m, n, v);
  }
}

bool fp8_few_rows(const Fp8GemmDesc& d, int sms) { return d.m <= 8 && d.n <= 32LL * sms; }

cudaError_t launch_fp8_few(const Fp8GemmDesc& d, int sms, cudaStream_t st) {
  FewArgs a;
  a.x = static_cast<const uint8_t*>(d.a), a.w = static_cast<const uint8_t*>(d.b);
  a.sx = static_cast<const uint8_t*>(d.a_scale), a.sw = static_cast<const uint8_t*>(d.b_scale);
  a.ldx = d.lda, a.ldw = d.ldb, a.sx_rows = (d.m + 3) & ~3LL, a.sw_rows = (d.n + 3) & ~3LL, a.n = d.n, a.k = d.k;
  a.m = static_cast<int>(d.m), a.kblocks = static_cast<int>((d.k + 127) / 128);
  a.add = d.add, a.out = d.out, a.ldadd = d.ldadd, a.ldc = d.ldc, a.out_dt = d.out_dt;
  const long long tiles = (d.n + 15) / 16;
  const int warps = tiles <= sms ? 16 : 8;  // 1024 x 4096: 3.1 us, with 8 warps 3.3
  a.per_warp = (a.kblocks + warps - 1) / warps;
  const dim3 grid(static_cast<unsigned>(tiles)), block(32 * warps);
  if (d.a_fmt == MUON_E5M2)
    return d.b_fmt == MUON_E5M2 ? launch_pdl(fp8_few_kernel<true, true>, grid, block, 0, st, a)
                                : launch_pdl(fp8_few_kernel<true, false>, grid, block, 0, st, a);
  return d.b_fmt == MUON_E5M2 ? launch_pdl(fp8_few_kernel<false, true>, grid, block, 0, st, a)
                              : launch_pdl(fp8_few_kernel<false, false>, grid, block, 0, st, a);
}

}  // namespace muon
