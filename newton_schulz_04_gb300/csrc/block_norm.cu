// block_norm.cu -- the norms around a block: bf16 rows, and the choice by type.
#include "block_norm_rows.cuh"

namespace muon {

// the other types are compiled in files of their own
extern template cudaError_t launch_block_norm_rows<__half>(const muon_block_norm_args&, int, int, cudaStream_t);
extern template cudaError_t launch_block_norm_rows<float>(const muon_block_norm_args&, int, int, cudaStream_t);

cudaError_t launch_block_norm(const muon_block_norm_args& a, int vec, int sms, cudaStream_t st) {
  if (a.dt == MUON_BF16) return launch_block_norm_rows<__nv_bfloat16>(a, vec, sms, st);
  return a.dt == MUON_FP16 ? launch_block_norm_rows<__half>(a, vec, sms, st) : launch_block_norm_rows<float>(a, vec, sms, st);
}

}  // namespace muon
