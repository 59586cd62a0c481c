// fp8_gemm.cu -- C = A B^T (+ D) of 8-bit operands with a power-of-two scale for each row and block of 128 of K.
//
//   C[m][n] = round( sum_k a[m][k] 2^ea[m][k/128] b[n][k] 2^eb[n][k/128]  + D[m][n] )
//
// One form serves a layer's three products: the forward pass (A tokens, B the
// weight), the data gradient (B the weight's transposed copy) and the weight
// gradient (both operands laid out along the tokens).
//
// tcgen05.mma kind::mxf8f6f4 multiplies every 32 of K by a scale byte (E8M0) of the
// row of A and the row of B, taken from TMEM, and accumulates in fp32 over all of K.
// A block of 128 is four such steps that name the same byte, so one 32-bit TMEM
// column serves 512 of K, which is how the scales are kept in memory: words of four
// blocks, rows side by side.
//
// A persistent grid of CTA pairs (clusters of two) works through output tiles of
// 256 rows of B by T rows of A (T a multiple of 32, at most 224), one pair MMA of
// M = 256, N = T per 32 of K: the rows of B (output columns) are the MMA's M, so
// that the 32 lanes of a TMEM row group are 32 consecutive elements of C's row.
// Every store of a warp is then one contiguous segment whatever C's alignment or
// stride, with no staging.  Each CTA loads its 128 rows of B and half of the T rows of A.
//
// TMEM (512 columns): two accumulators of 224, so the epilogue of one tile overlaps
// the next main loop, and four sets of scales (4 + 7 columns each).
//
// Warp roles (480 threads):
//   warp 0       TMA producer: stages of 128 of K (one swizzled 128-byte box per operand)
//   warp 1       TMEM allocation; the leader's lane 0 issues the MMAs
//   warps 2..5   scales: every warp stores the words of all rows of the tile to its
//                own quarter of TMEM's lanes (the MMA reads a copy in each quarter),
//                up to four 512-deep groups ahead of the MMAs
//   warps 6..13  epilogue: two warps per lane quarter, alternating 32-column chunks
//   warp 14      fetches the words to shared memory, up to eight groups ahead: behind a
//                queue of TMA loads a fetch takes 1500 to 2500 cycles, and one that
//                was issued a group (1792 cycles) ahead held the MMAs up at every
//                other stage (18 us more at 8192 x 14336 x 4096)
//
// 8192 x 14336 x 4096 takes 270 us in short bursts, 322 to 326 in long runs under the 1.4 kW limit.  Times that
// comments here give for it are of bursts, and differences that a step made when it was taken.
//
// At most 8 rows of A with a B that small tiles cover at once have a kernel of their own (fp8_few.cu).
// When there are too few tiles to fill the GPU, 2 or 4 pairs of one cluster share a tile of
// at most 64 rows of A, each with its part of K.  Every pair sends the others their
// share of the tile's rows of A through distributed shared memory and adds up its own, in
// the order of the parts: no workspace, no second launch, the same bits every time.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "train_ops.h"

namespace muon {

// A kernel that gives up on a wait records it here (muon_fp8_status takes it).
static __device__ int g_fp8_status;
static __device__ int g_fp8_taken;
__global__ void fp8_take_status_kernel() { g_fp8_taken = atomicExch(&g_fp8_status, 0); }

// Three shapes of the kernel, by the tile's rows of A.
//   BIG    224: single blocks of K in a ring of 7, taken two at a time by the MMAs (against
//          3 stages of two blocks 10 us less at 8192 x 14336 x 4096)
//   MID    96 to 192: a pair of blocks' MMAs are shorter than two waits and two commits, so
//          stages of two blocks (2048^3: 11 us, in single blocks 12.5)
//   SMALL  32 and 64: smaller boxes, and room for the split of K
enum F8Kind : int { F8_BIG, F8_MID, F8_SMALL };
template <F8Kind KIND>
struct F8Cfg {
  static constexpr int BN = 128;                 // rows of B per CTA (256 per pair)
  static constexpr int TMAX = KIND == F8_BIG ? 224 : KIND == F8_MID ? 192 : 64;  // rows of A per tile
  static constexpr int KB = 128;                 // K per block: one 128-byte swizzled row of 8-bit values
  static constexpr int KPS = KIND == F8_BIG ? 1 : 2;  // blocks per stage
  static constexpr int STAGES = KIND == F8_BIG ? 7 : KIND == F8_MID ? 3 : 4;
  static constexpr int B_BOX = BN * KB;
  static constexpr int A_BOX = TMAX / 2 * KB;
  static constexpr int STAGE = KPS * (B_BOX + A_BOX);
  static constexpr int EPI_WARP = 6, EPI_WARPS = 8, LOAD_WARP = EPI_WARP + EPI_WARPS;
  static constexpr int THREADS = 32 * (LOAD_WARP + 1);
  static constexpr int SETS = 4;                     // groups of scales in TMEM
  static constexpr int SLOTS = 8;                    // and in shared memory
  static constexpr int SCALE_SLOT = (BN + 256) * 4;  // read in 32-row pieces, up to 256 rows of A
  static constexpr int BAR_BYTES = 512;
  // Split K: the parts' sums of this pair's share of the tile, [parts][T / parts][128] fp32
  static constexpr int RECV = KIND == F8_SMALL ? TMAX * BN * 4 : 0;
  static constexpr int SMEM = STAGES * STAGE + SLOTS * SCALE_SLOT + BAR_BYTES + 1024 + RECV;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ACC_COLS = TMAX;
  static constexpr uint32_t SCALE_COL = 2 * 224;
  static constexpr uint32_t SET_COLS = 16;  // rows of B in the first 4 columns, of A from the 8th on
  static constexpr uint32_t EPI_ARRIVALS = 2 * EPI_WARPS;
  static constexpr uint32_t SCALE_ARRIVALS = 2 * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(2 * ACC_COLS <= SCALE_COL && SCALE_COL + SETS * SET_COLS <= TMEM_COLS, "TMEM budget");
  static_assert(A_BOX % 1024 == 0 && B_BOX % 1024 == 0 && STAGE % 1024 == 0, "swizzle atoms of 1024 bytes");
};

struct F8Args {
  CUtensorMap ta, tb;   // {128, T / 2} boxes of A, {128, 128} boxes of B
  const uint32_t *sa, *sb;  // scale words [group][rows4]
  long long m, n;
  long long sa_rows, sb_rows;
  int kblocks;          // blocks of 128
  int tail_steps;       // 32-deep MMA steps of the last block
  int tile_m;
  int nI, nJ;           // tiles along n (256) and m
  int splits, gps;      // parts of K (pairs of a cluster), 512-deep groups per part
  int items;            // tiles
  int rgroup;           // tiles along n walked together
  uint32_t idesc;
  const void* add;
  void* out;
  long long ldadd, ldc;
  int out_dt;
  int* status;
};

__device__ __forceinline__ void tma_load_2d_pair(const CUtensorMap* m, uint32_t bar_cluster, void* dst, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}
// 16-byte aligned global -> shared copy of whole 16 bytes, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// D[tmem] (+)= (A scale_a) (B scale_b) over the pair, 32 of K; scales in TMEM, one byte per row and 32 of K.
__device__ __forceinline__ void mma_pair_scaled(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                                uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
// Arrive on a barrier that may be another CTA's, without a release: after a fence at cluster scope (which needs an
// arrive of that scope to count for the other CTA), or where only TMEM is handed over, which tcgen05.wait and the
// tcgen05 fences order.  A release at cluster scope would wait for every access of this thread in flight, 2000
// cycles behind a queue of TMA loads.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p)::"memory");
  return p != 0;
}
// Each thread stores words to consecutive TMEM columns of its own lane.
__device__ __forceinline__ void tmem_st_x4(uint32_t t, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

struct F8Item {
  int i, j;        // tile along n, along m
  int g0, g1;      // 512-deep groups of K
};
__device__ __forceinline__ F8Item decode_item(const F8Args& a, int u, int part) {
  F8Item it;
  // rgroup tile rows of B at a time, so that they stay in L2 while A streams by
  const int per = a.rgroup * a.nJ;
  const int g = u / per, first = g * a.rgroup, gs = min(a.nI - first, a.rgroup), w = u - g * per;
  it.i = first + w % gs;
  it.j = w / gs;
  it.g0 = part * a.gps;
  it.g1 = min((a.kblocks + 3) >> 2, it.g0 + a.gps);
  return it;
}

// p + ld, kept as a step from the last row: computed at once, the 32 addresses take 64 registers.
template <typename P>
__device__ __forceinline__ P* step(P* p, long long ld) {
  p += ld;
  asm volatile("" : "+l"(p));
  return p;
}
__device__ __forceinline__ void tmem_ld_rows(uint32_t t, float (&v)[32]) { tmem_ld_32x32b_x32(t, v); }
__device__ __forceinline__ void tmem_ld_rows(uint32_t t, float (&v)[16]) { tmem_ld_32x32b_x16(t, v); }

// A warp's share of a tile: every other chunk of CH rows of C, one row per register, from
// row m0 on (`rows` of them exist), column n of this lane.  `ready` waits for the accumulator.  The
// first rows to add are on their way before that, the next ones while a chunk is stored
// (the weight gradient of 4096 x 4096 over 8192 tokens, repeated under the power cap: 105 -> 103 us).
template <typename T, bool ADD, typename F>
__device__ __forceinline__ bool epi_tile(const F8Args& a, uint32_t acc, long long m0, int rows, int half, long long n,
                                         const F& ready) {
  constexpr int CH = ADD ? 16 : 32;
  const bool in = n < a.n;
  int c = half * CH;
  T x[ADD ? CH : 1];
  const T* d = static_cast<const T*>(a.add) + (ADD ? (m0 + c) * a.ldadd + n : 0);
  const auto fetch = [&](int left) {
    if (in) {
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        if (u < left) x[ADD ? u : 0] = *d;
        d = step(d, a.ldadd);
      }
      d += CH * a.ldadd;
    }
  };
  if (ADD) fetch(rows - c);
  if (!ready()) return false;
  T* o = static_cast<T*>(a.out) + (m0 + c) * a.ldc + n;
  for (; c < rows; c += 2 * CH) {
    float v[CH];
    tmem_ld_rows(acc + c, v);
    if (in) {
      if (ADD) {
#pragma unroll
        for (int u = 0; u < CH; ++u)
          if (c + u < rows) v[u] += to_f32(x[ADD ? u : 0]);
        fetch(rows - c - 2 * CH);
      }
#pragma unroll
      for (int u = 0; u < CH; ++u) {
        if (c + u < rows) *o = from_f32<T>(v[u]);
        o = step(o, a.ldc);
      }
      o += CH * a.ldc;
    }
    __syncwarp();
  }
  return true;
}
template <typename T, typename F>
__device__ __forceinline__ bool epi_tile(const F8Args& a, uint32_t acc, long long m0, int rows, int half, long long n,
                                         const F& ready) {
  return a.add ? epi_tile<T, true>(a, acc, m0, rows, half, n, ready) : epi_tile<T, false>(a, acc, m0, rows, half, n, ready);
}
template <F8Kind KIND, bool SPLIT>
__global__ void __launch_bounds__(F8Cfg<KIND>::THREADS, 1) fp8_gemm_kernel(const __grid_constant__ F8Args a) {
  using C = F8Cfg<KIND>;
  constexpr int STAGES = C::STAGES;
  static_assert(KIND == F8_SMALL || !SPLIT, "only small tiles are split");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tiles = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* scales = tiles + STAGES * C::STAGE;  // [SLOTS] words of the rows of B, then of A
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::SLOTS * C::SCALE_SLOT);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;   // [2] accumulator complete
  uint64_t* tempty = tfull + 2;          // [2] accumulator read
  uint64_t* sfull = tempty + 2;          // [SETS] scales of a group in TMEM
  uint64_t* sempty = sfull + C::SETS;    // [SETS] scales read by the group's MMAs
  uint64_t* sload = sempty + C::SETS;    // [SLOTS] scales of a group in shared memory
  uint64_t* sfree = sload + C::SLOTS;    // [SLOTS] and copied on
  uint64_t* joined = sfree + C::SLOTS;   // the other parts' sums have arrived
  uint64_t* drain = joined + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* recv = reinterpret_cast<uint8_t*>(full) + C::BAR_BYTES;
  static_assert(C::BAR_BYTES >= (2 * STAGES + 2 * C::SETS + 2 * C::SLOTS + 6) * 8 + 8, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::EPI_ARRIVALS);
    }
    for (int b = 0; b < C::SETS; ++b) {
      mbar_init(&sfull[b], C::SCALE_ARRIVALS);
      mbar_init(&sempty[b], 1);
    }
    for (int b = 0; b < C::SLOTS; ++b) {
      mbar_init(&sload[b], 1);
      mbar_init(&sfree[b], 4);
    }
    mbar_init(joined, C::EPI_WARPS * a.splits);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.ta);
    tma_prefetch_desc(&a.tb);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  pdl_wait();
  const int crank = static_cast<int>(cluster_ctarank());
  const int rank = crank & 1, part = SPLIT ? crank >> 1 : 0;  // in the pair; the pair's part of K
  const uint32_t leader = static_cast<uint32_t>(crank & ~1);
  const uint16_t pair_mask = static_cast<uint16_t>(0x3 << (crank & ~1));
  const uint32_t tmem = *tmem_slot;
  const int per_cluster = SPLIT ? 2 * a.splits : 2;
  const int cid = blockIdx.x / per_cluster, ncl = gridDim.x / per_cluster;
  const int half = a.tile_m >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      int st = 0;
      bool ok = true;
      for (int t = cid; t < a.items && ok; t += ncl) {
        const F8Item it = decode_item(a, t, part);
        const int nb0 = it.i * 256 + rank * C::BN, ma0 = it.j * a.tile_m + rank * half;
        const int kb1 = min(a.kblocks, it.g1 * 4);
        for (int kb = it.g0 * 4; kb < kb1; kb += C::KPS, ++st) {
          const int s = st % STAGES;
          if (*abort_flag || !mbar_wait(&empty[s], ((st / STAGES) & 1) ^ 1)) {
            ok = false;
            break;
          }
          const int nb = min(C::KPS, kb1 - kb);
          uint8_t* p = tiles + s * C::STAGE;
          const uint32_t fbar = mapa_cluster(&full[s], leader);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * nb * (C::B_BOX + half * C::KB));
          for (int q = 0; q < nb; ++q) {
            tma_load_2d_pair(&a.tb, fbar, p + q * C::B_BOX, (kb + q) * C::KB, nb0);
            tma_load_2d_pair(&a.ta, fbar, p + C::KPS * C::B_BOX + q * C::A_BOX, (kb + q) * C::KB, ma0);
          }
        }
      }
      if (!ok) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
        if (rank == 0)  // copies in flight land before the CTAs exit
          for (int q = st > STAGES ? st - STAGES : 0; q < st; ++q)
            mbar_wait(&full[q % STAGES], (q / STAGES) & 1);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the loop, so that addresses and descriptors stay in
      // uniform registers; one elected lane issues.  An MMA lasts T / 2 cycles: issued by
      // a divergent lane that rebuilt its descriptors, each took longer than that
      // (147 us more at 8192 x 14336 x 4096).
      int st = 0, grp = 0, tile = 0;
      bool ok = true;
      const uint32_t base = smem_u32(tiles);
      // Without a look at the abort flag, which costs as much again: a wait that another role gave up on runs out here too.
      auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity));
      };
      for (int t = cid; t < a.items && ok; t += ncl, ++tile) {
        const F8Item it = decode_item(a, t, part);
        const int abuf = tile & 1;
        if (!warp_wait(&tempty[abuf], ((tile >> 1) & 1) ^ 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + abuf * C::ACC_COLS;
        const int kb0 = it.g0 * 4, kb1 = min(a.kblocks, it.g1 * 4);
        for (int kb = kb0; kb < kb1; kb += 2) {
          // Two blocks at a time, in one stage or two: the waits and commits of one
          // block took longer than its MMAs.
          const bool two = kb + 1 < kb1;
          const int stages = C::KPS == 2 || !two ? 1 : 2;
          const int s0 = st % STAGES, s1 = (st + 1) % STAGES;
          const uint32_t in_group = static_cast<uint32_t>(kb) & 3u;
          if (in_group == 0) {  // a new group of four blocks: its scales
            if (!warp_wait(&sfull[grp % C::SETS], (grp / C::SETS) & 1)) {
              ok = false;
              break;
            }
          }
          if (!warp_wait(&full[s0], (st / STAGES) & 1) ||
              (stages == 2 && !warp_wait(&full[s1], ((st + 1) / STAGES) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t bd0 = make_sdesc(base + s0 * C::STAGE, 16, 1024, 2u);
          const uint64_t bd1 = C::KPS == 2 ? bd0 + C::B_BOX / 16 : make_sdesc(base + s1 * C::STAGE, 16, 1024, 2u);
          const uint64_t ad0 = bd0 + C::KPS * C::B_BOX / 16;
          const uint64_t ad1 = C::KPS == 2 ? ad0 + C::A_BOX / 16 : bd1 + C::B_BOX / 16;
          const uint32_t sc = tmem + C::SCALE_COL + (grp % C::SETS) * C::SET_COLS;
          const uint32_t idesc = a.idesc | (in_group << 29) | (in_group << 4);
          constexpr uint32_t NEXT_SF = (1u << 29) | (1u << 4);
          const bool whole = two && (kb + 2 < a.kblocks || a.tail_steps == 4);
          const bool group_end = in_group == 2 || kb + 2 >= kb1;
          if (elect_one()) {
            if (whole) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_pair_scaled(d, bd0 + kk * 2, ad0 + kk * 2, idesc, sc, sc + 8, kk != 0 || kb != kb0 ? 1u : 0u);
              if (C::KPS == 1) tc_commit_pair(&empty[s0], pair_mask);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_pair_scaled(d, bd1 + kk * 2, ad1 + kk * 2, idesc + NEXT_SF, sc, sc + 8, 1u);
              tc_commit_pair(&empty[C::KPS == 1 ? s1 : s0], pair_mask);
            } else {
              for (int q = 0; q < (two ? 2 : 1); ++q) {
                const int steps = kb + q == a.kblocks - 1 ? a.tail_steps : 4;
                for (int kk = 0; kk < steps; ++kk)
                  mma_pair_scaled(d, (q ? bd1 : bd0) + kk * 2, (q ? ad1 : ad0) + kk * 2, idesc + q * NEXT_SF, sc, sc + 8,
                                  (q | kk) != 0 || kb != kb0 ? 1u : 0u);
                if (C::KPS == 1) tc_commit_pair(&empty[q ? s1 : s0], pair_mask);
              }
              if (C::KPS == 2) tc_commit_pair(&empty[s0], pair_mask);
            }
            if (group_end) tc_commit_pair(&sempty[grp % C::SETS], pair_mask);
            if (kb + 2 >= kb1) tc_commit_pair(&tfull[abuf], pair_mask);
          }
          __syncwarp();
          st += stages;
          if (group_end) ++grp;
        }
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // tcgen05.commit covers the MMAs of the thread that issues it
      if (elect_one()) tc_commit_pair(drain, static_cast<uint16_t>(1u << leader));
      __syncwarp();
      mbar_wait(drain, 0);
    }
  } else if (warp < C::EPI_WARP) {
    // -------------------------------------------------------------- scales
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's quarter of the lanes
    int grp = 0;
    bool ok = true;
    for (int t = cid; t < a.items && ok; t += ncl) {
      const F8Item it = decode_item(a, t, part);
      for (int g = it.g0; g < it.g1; ++g, ++grp) {
        const int slot = grp % C::SLOTS, set = grp % C::SETS;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&sload[slot], (grp / C::SLOTS) & 1));
        if (!ok) break;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(scales + slot * C::SCALE_SLOT) + lane;
        uint32_t wb[4], wa[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) wb[j] = w[j * 32];
#pragma unroll
        for (int j = 0; j < 8; ++j) wa[j] = w[C::BN + j * 32];
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&sempty[set], ((grp / C::SETS) & 1) ^ 1));
        if (!ok) break;
        tc_fence_after();
        const uint32_t sc = tmem + lanes + C::SCALE_COL + set * C::SET_COLS;
        tmem_st_x4(sc, wb);
        tmem_st_x8(sc + 8, wa);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // The slot is free once its words are in TMEM.  An arrive right after the loads overtook them when the
          // epilogue kept the load unit busy, and the next copy into the slot was read by some of the warps.
          mbar_arrive(&sfree[slot]);
          mbar_arrive_relaxed(mapa_cluster(&sfull[set], leader));
        }
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp == C::LOAD_WARP) {
    if (lane == 0) {
      // ------------------------------------------------------- scale fetch
      int grp = 0;
      bool ok = true;
      for (int t = cid; t < a.items && ok; t += ncl) {
        const F8Item it = decode_item(a, t, part);
        const long long n0 = it.i * 256LL + rank * C::BN, m0 = static_cast<long long>(it.j) * a.tile_m;
        const uint32_t nb = static_cast<uint32_t>(max(0LL, min(static_cast<long long>(C::BN), a.sb_rows - n0))) * 4;
        const uint32_t na = static_cast<uint32_t>(min(static_cast<long long>(a.tile_m), a.sa_rows - m0)) * 4;
        for (int g = it.g0; g < it.g1; ++g, ++grp) {
          const int slot = grp % C::SLOTS;
          if (*abort_flag || !mbar_wait(&sfree[slot], ((grp / C::SLOTS) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* p = scales + slot * C::SCALE_SLOT;
          mbar_arrive_expect_tx(&sload[slot], nb + na);
          if (nb) bulk_load(p, a.sb + g * a.sb_rows + n0, nb, &sload[slot]);
          bulk_load(p + C::BN * 4, a.sa + g * a.sa_rows + m0, na, &sload[slot]);
        }
      }
      if (!ok) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // every copy lands before the CTA exits
      for (int q = grp > C::SLOTS ? grp - C::SLOTS : 0; q < grp; ++q) mbar_wait(&sload[q % C::SLOTS], (q / C::SLOTS) & 1);
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3, half_tile = (warp - C::EPI_WARP) >> 2;
    int tile = 0;
    bool ok = true;
    for (int t = cid; t < a.items; t += ncl, ++tile) {
      const F8Item it = decode_item(a, t, part);
      const int abuf = tile & 1;
      const long long n = it.i * 256LL + rank * C::BN + quarter * 32 + lane;
      const long long m0 = static_cast<long long>(it.j) * a.tile_m;
      const int rows = static_cast<int>(min(static_cast<long long>(a.tile_m), a.m - m0));
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter) << 21) + abuf * C::ACC_COLS;
      const auto ready = [&]() -> bool {
        const bool full_now = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&tfull[abuf], (tile >> 1) & 1));
        tc_fence_after();
        return full_now;
      };
      if (SPLIT) {
        // Rows of A p share .. are added up by part p.  One item per cluster: nothing is received twice.
        const int share = a.tile_m / a.splits, shift = __ffs(share) - 1, c = half_tile * 32;  // 8, 16 or 32 rows
        const float* sums = reinterpret_cast<const float*>(recv) + quarter * 32 + lane;  // [part][row][128]
        float v[32];
        ok = ready();
        if (!ok) break;
        if (c < a.tile_m) tmem_ld_32x32b_x32(acc + c, v);
        if (c < a.tile_m) {
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            const float* to = sums + (part * share + ((c + u) & (share - 1))) * C::BN;
            st_shared_cluster(mapa_cluster(to, static_cast<uint32_t>(2 * ((c + u) >> shift) + rank)), __float_as_int(v[u]));
          }
        }
        __syncwarp();
        if (lane == 0) {  // one release for all parts: each waits for the stores in flight
          fence_cluster();
          for (int p = 0; p < a.splits; ++p) mbar_arrive_relaxed(mapa_cluster(joined, static_cast<uint32_t>(2 * p + rank)));
        }
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait_cluster(joined, 0));
        if (!ok) break;
        // not unrolled over all rows: its code then took longer to fetch than to run (19000 cycles)
#pragma unroll 2
        for (int r = half_tile; r < share; r += 2) {
          const long long m = part * share + r;
          if (m < rows && n < a.n) {
            float sum = sums[r * C::BN] + sums[(share + r) * C::BN];
            if (a.splits == 4) sum = (sum + sums[(2 * share + r) * C::BN]) + sums[(3 * share + r) * C::BN];
            fp8_product_out(a, m0 + m, n, sum);
          }
        }
        __syncwarp();
      } else {
        ok = a.out_dt == MUON_FP32   ? epi_tile<float>(a, acc, m0, rows, half_tile, n, ready)
             : a.out_dt == MUON_BF16 ? epi_tile<__nv_bfloat16>(a, acc, m0, rows, half_tile, n, ready)
                                     : epi_tile<__half>(a, acc, m0, rows, half_tile, n, ready);
        if (!ok) break;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(mapa_cluster(&tempty[abuf], leader));
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
    __syncwarp();
  }

  __syncwarp();
  pdl_launch_dependents();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, C::TMEM_COLS);
  }
}

// K = 0: C = D, or zeros.
template <typename T>
__global__ void __launch_bounds__(256) fp8_empty_kernel(long long m, long long n, const T* add, long long ldadd, T* out,
                                                        long long ldc) {
  pdl_launch_dependents();
  pdl_wait();
  const long long total = m * n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = i / n, c = i - r * n;
    out[r * ldc + c] = add ? add[r * ldadd + c] : from_f32<T>(0.f);
  }
}

// ------------------------------------------------------------------ host side
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// [rows][k] bytes, boxes of 128 bytes by `box_rows`; reads past k or the last row give 0.
static bool byte_map(CUtensorMap* m, const void* base, long long k, long long rows, long long ld, int box_rows) {
  const auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch configuration: clusters of `parts` pairs.
struct Fp8Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  Fp8Launch(F8Kind kind, int parts, int clusters, cudaStream_t st, bool pdl) {
    cfg.gridDim = dim3(2 * parts * clusters);
    cfg.blockDim = dim3(F8Cfg<F8_BIG>::THREADS);
    cfg.dynamicSmemBytes = kind == F8_BIG ? F8Cfg<F8_BIG>::SMEM : kind == F8_MID ? F8Cfg<F8_MID>::SMEM : F8Cfg<F8_SMALL>::SMEM;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
  }
};

cudaError_t fp8_status_address(int** p) { return cudaGetSymbolAddress(reinterpret_cast<void**>(p), g_fp8_status); }

// Read and cleared in one atomic step, after the stream's work: what a kernel on another stream records meanwhile is
// in this answer or in the next.  One caller at a time, for the word that carries the answer.
cudaError_t fp8_take_status(cudaStream_t st, int* word) {
  static std::mutex mu;
  std::lock_guard<std::mutex> lk(mu);
  fp8_take_status_kernel<<<1, 1, 0, st>>>();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(word, g_fp8_taken, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  const cudaError_t done = cudaStreamSynchronize(st);
  return e != cudaSuccess ? e : done;
}

// Clusters of 1, 2 and 4 pairs that can be resident at once; with the kernels' shared-memory limits, once per device.
struct Fp8Clusters {
  int of[3];
  int* status;  // g_fp8_status on that device
};
static cudaError_t fp8_clusters(int sms, Fp8Clusters* out) {
  static std::mutex mu;
  static Fp8Clusters cached[64];
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!done[dev]) {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaFuncSetAttribute(fp8_gemm_kernel<F8_BIG, false>, attr, F8Cfg<F8_BIG>::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_gemm_kernel<F8_MID, false>, attr, F8Cfg<F8_MID>::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_gemm_kernel<F8_SMALL, false>, attr, F8Cfg<F8_SMALL>::SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fp8_gemm_kernel<F8_SMALL, true>, attr, F8Cfg<F8_SMALL>::SMEM);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 3; ++i) {
      const int parts = 1 << i, most = sms / (2 * parts);
      Fp8Launch l(i ? F8_SMALL : F8_BIG, parts, std::max(most, 1), nullptr, false);
      int n = 0;
      e = i ? cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<F8_SMALL, true>, &l.cfg)
            : cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<F8_BIG, false>, &l.cfg);
      if (e != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = i ? 0 : most;  // no clusters of that size: K is not split so far
      }
      cached[dev].of[i] = std::min(n, most);
    }
    e = fp8_status_address(&cached[dev].status);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  *out = cached[dev];
  return cudaSuccess;
}

// The tile of tokens and the parts of K with the least estimated time, in SM cycles.  As measured over T of 32 to 224
// and 1, 2 and 4 parts: a block of K takes the longest of its MMAs (2 T), its loads ((128 + T / 2)
// rows of 128 bytes at 64 bytes a cycle: 256 + T) and the handling of a stage (313); a tile some 2000 cycles to
// fill and drain the pipeline; joining parts 85 T.  K is split only where every tile has a cluster of
// its own.  A tile of 32 rows of A by 4096 x 4096 takes 7.0 us on two parts (32 clusters; of four parts 15
// fit) and 7.9 unsplit, by 1024 x 4096 5.4 on four and 7.9; 512 x 4096 x 4096 10.3 with T = 128, 14.9 with 64, 12.7 with 224.
static Fp8Plan fp8_plan(long long m, long long n, long long k, const Fp8Clusters& fit) {
  const long long groups = (k + 511) / 512, nI = (n + 255) / 256;
  Fp8Plan best = {32, 1, static_cast<int>(groups)};
  double best_time = 1e300;
  for (int t = 32; t <= F8Cfg<F8_BIG>::TMAX; t += 32) {
    const long long tiles = nI * ((m + t - 1) / t);
    const double block = std::max({2.0 * t, 256.0 + t, 313.0});
    for (int i = 0; i < 3; ++i) {
      const long long parts = 1 << i, gps = (groups + parts - 1) / parts;
      if (i && (t > F8Cfg<F8_SMALL>::TMAX || tiles > fit.of[i] || (groups + gps - 1) / gps != parts)) break;
      const double waves = static_cast<double>((tiles + fit.of[i] - 1) / std::max(1, fit.of[i]));
      const double time = waves * (gps * 4 * block + 2000.0) + (i ? 85.0 * t : 0.0);
      if (time < best_time) {
        best_time = time;
        best = {t, static_cast<int>(parts), static_cast<int>(gps)};
      }
    }
    if (t >= m) break;
  }
  return best;
}

template <typename T>
static cudaError_t launch_empty(const Fp8GemmDesc& d, int sms, cudaStream_t st) {
  const long long want = (d.m * d.n + 255) / 256;
  return launch_pdl(fp8_empty_kernel<T>, dim3(static_cast<unsigned>(std::min<long long>(want, 8LL * sms))), dim3(256), 0, st,
                    d.m, d.n, static_cast<const T*>(d.add), d.ldadd, static_cast<T*>(d.out), d.ldc);
}

cudaError_t launch_fp8_gemm(const Fp8GemmDesc& d, int sms, cudaStream_t st, const char** why) {
  using C = F8Cfg<F8_BIG>;
  *why = nullptr;
  if (d.k == 0)
    return d.out_dt == MUON_FP32   ? launch_empty<float>(d, sms, st)
           : d.out_dt == MUON_BF16 ? launch_empty<__nv_bfloat16>(d, sms, st)
                                   : launch_empty<__half>(d, sms, st);
  if (fp8_few_rows(d, sms)) return launch_fp8_few(d, sms, st);
  Fp8Clusters fit;
  cudaError_t e = fp8_clusters(sms, &fit);
  if (e != cudaSuccess) return e;
  const Fp8Plan p = fp8_plan(d.m, d.n, d.k, fit);
  F8Args a;
  if (!byte_map(&a.ta, d.a, d.k, d.m, d.lda, p.tile_m / 2) || !byte_map(&a.tb, d.b, d.k, d.n, d.ldb, C::BN)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  a.sa = static_cast<const uint32_t*>(d.a_scale);
  a.sb = static_cast<const uint32_t*>(d.b_scale);
  a.m = d.m;
  a.n = d.n;
  a.sa_rows = (d.m + 3) & ~3LL;
  a.sb_rows = (d.n + 3) & ~3LL;
  a.kblocks = static_cast<int>((d.k + 127) / 128);
  a.tail_steps = static_cast<int>((d.k - (a.kblocks - 1) * 128LL + 31) / 32);
  a.tile_m = p.tile_m;
  a.nI = static_cast<int>((d.n + 255) / 256);
  a.nJ = static_cast<int>((d.m + p.tile_m - 1) / p.tile_m);
  a.splits = p.splits;
  a.gps = p.groups_per_split;
  const long long items = static_cast<long long>(a.nI) * a.nJ;
  if (items > 0x3fffffffLL) {
    *why = "too many tiles";
    return cudaErrorInvalidValue;
  }
  a.items = static_cast<int>(items);
  // as many 256-row panels of B as fit 32 MB of the 126 MB L2, at least 4
  a.rgroup = static_cast<int>(std::min<long long>(a.nI, std::max<long long>(4, (32LL << 20) / (256 * d.k))));
  // instruction descriptor: A (the kernel's B) and B formats, N >> 3, E8M0 scales, M >> 4 with M = 256
  a.idesc = (static_cast<uint32_t>(d.b_fmt) << 7) | (static_cast<uint32_t>(d.a_fmt) << 10) |
            (static_cast<uint32_t>(p.tile_m >> 3) << 17) | (1u << 23) | (16u << 24);
  a.add = d.add;
  a.out = d.out;
  a.ldadd = d.ldadd;
  a.ldc = d.ldc;
  a.out_dt = d.out_dt;
  a.status = fit.status;
  const F8Kind kind = p.tile_m <= F8Cfg<F8_SMALL>::TMAX ? F8_SMALL : p.tile_m <= F8Cfg<F8_MID>::TMAX ? F8_MID : F8_BIG;
  Fp8Launch l(kind, p.splits, p.splits > 1 ? a.items : std::min(a.items, fit.of[0]), st, true);
  return p.splits > 1       ? cudaLaunchKernelEx(&l.cfg, fp8_gemm_kernel<F8_SMALL, true>, a)
         : kind == F8_SMALL ? cudaLaunchKernelEx(&l.cfg, fp8_gemm_kernel<F8_SMALL, false>, a)
         : kind == F8_MID   ? cudaLaunchKernelEx(&l.cfg, fp8_gemm_kernel<F8_MID, false>, a)
                            : cudaLaunchKernelEx(&l.cfg, fp8_gemm_kernel<F8_BIG, false>, a);
}

}  // namespace muon
