// train_ops.h -- internal interface of the operators around the update: gradient
// clipping, the RMS norm, 8-bit quantisation and the 8-bit product; the norms around a
// block, the gated activation and the transposition of 8-bit matrices.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "muon_ns.h"

namespace muon {

// engine.cu
muon_status fail(muon_status s, const char* fmt, ...);
void clear_error();
int device_sms(int* major, int* minor, muon_status* st);

inline int dtype_bytes(int dt) { return dt == MUON_FP32 ? 4 : 2; }

// ---- clip.cu
// Tensors per launch: two sizes of the argument block, so that a short list
// does not pay for copying the long one (29 bytes per tensor, 32 KB at most).
constexpr int kClipSmall = 64, kClipLarge = 1024;
constexpr int kClipChunkBytes = 32768;  // of one tensor, that a CTA takes at a time
constexpr int kClipCtasPerSm = 4;       // 256-thread CTAs
cudaError_t launch_clip(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dts, int count,
                        float max_norm, float eps, double* partial, int grid, float* norm, cudaStream_t st);

// ---- rms_norm.cu
struct RmsNormArgs {
  const void* x;         // [rows][ldx]
  const void* residual;  // [rows][ldr] or nullptr
  const void* weight;    // [cols] or nullptr (1)
  void* y;               // [rows][ldy] or nullptr
  void* h;               // [rows][ldh] or nullptr
  float* rstd;           // [rows] or nullptr
  uint8_t* q;            // [rows][ldq] or nullptr
  uint8_t* qscale;       // kept scales, with q
  long long ldx, ldr, ldy, ldh, ldq;
  long long rows;
  int cols;
  int weight_dt;
  int fmt;               // 0 e4m3, 1 e5m2
  float eps;
  int vec;               // 1: every row of x, residual, y, h and the weight allow 16-byte accesses
};
cudaError_t launch_rms_norm(const RmsNormArgs& a, int dt, int sms, cudaStream_t st);
struct RmsNormGradArgs {
  const void* dy;        // [rows][lddy]
  const void* h;         // [rows][ldh]
  const void* weight;    // [cols] or nullptr (1)
  const float* rstd;     // [rows]
  const void* dres;      // [rows][lddr] or nullptr
  void* dx;              // [rows][lddx] or nullptr
  float* partial;        // [ctas][cols], or nullptr (no weight gradient)
  float* dweight;        // [cols]
  long long lddy, ldh, lddr, lddx;
  long long rows;
  int cols;
  int weight_dt;
  int vec;
};
// CTAs of the gradient kernel, i.e. rows of `partial`.
int rms_norm_grad_ctas(long long rows, int cols, int dt, int sms);
cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int dt, int sms, cudaStream_t st);

// ---- fp8_quant.cu
struct Fp8QuantArgs {
  const void* x;
  long long ldx, rows, cols;
  int fmt, square, vec;
  uint8_t *q, *qs;       // [rows][ldq] and its scales, or nullptr
  uint8_t *qt, *qts;     // [cols][ldqt] and its scales, or nullptr
  long long ldq, ldqt;
};
cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, int dt, cudaStream_t st);

// ---- block_norm.cu
// vec: every row of the matrices allows 16-byte accesses.
cudaError_t launch_block_norm(const muon_block_norm_args& a, int vec, int sms, cudaStream_t st);
// CTAs or clusters of the gradient kernel at most, each with two rows of `partial` (or nullptr: no gradients of the weights).
int block_norm_grad_parts(long long rows, long long cols, int elem_size, int sms);
cudaError_t launch_block_norm_grad(const muon_block_norm_grad_args& a, float* partial, int vec, int sms, cudaStream_t st);

// ---- gated.cu
cudaError_t launch_gated(const muon_gated_args& a, int vec, cudaStream_t st);
cudaError_t launch_gated_grad(const muon_gated_grad_args& a, int vec, cudaStream_t st);

// ---- fp8_transpose.cu
struct Fp8TransposeArgs {
  const uint8_t *q, *qs;
  long long ldq, rows, cols;
  uint8_t *qt, *qts;
  long long ldqt;
};
cudaError_t launch_fp8_transpose(const Fp8TransposeArgs& a, int fmt, cudaStream_t st);

// ---- fp8_gemm.cu
struct Fp8GemmDesc {
  const void *a, *b;               // [m][lda], [n][ldb] 8-bit
  const void *a_scale, *b_scale;   // [ceil(k / 512)][rows up to 4][4]
  long long lda, ldb, m, n, k;
  int a_fmt, b_fmt;
  const void* add;                 // [m][ldadd] of the output's type, or nullptr
  void* out;                       // [m][ldc]
  long long ldadd, ldc;
  int out_dt;
};
// Tile of tokens and parts of the k axis for a problem (see fp8_gemm.cu).
struct Fp8Plan {
  int tile_m;
  int splits;
  int groups_per_split;  // 512-deep groups of k
};
cudaError_t launch_fp8_gemm(const Fp8GemmDesc& d, int sms, cudaStream_t st, const char** why);
// The kernel for a few rows of a (fp8_few.cu), and whether it is the one to take.
bool fp8_few_rows(const Fp8GemmDesc& d, int sms);
cudaError_t launch_fp8_few(const Fp8GemmDesc& d, int sms, cudaStream_t st);
// Address of the 8-bit product's status word (device memory of the library).
cudaError_t fp8_status_address(int** p);
// Synchronises the stream; *word is the status word's value, which is 0 from then on.
cudaError_t fp8_take_status(cudaStream_t st, int* word);

}  // namespace muon
