// block_norm.cu -- the norms around a block: the choice by type and alignment.
#include "block_norm.cuh"

namespace muon {

cudaError_t launch_block_norm(const muon_block_norm_args& a, int vec, int sms, cudaStream_t st) {
  const auto go = [&](auto t) {
    using T = decltype(t);
    return vec ? launch_block_norm_rows<T, false>(a, sms, st) : launch_block_norm_rows<T, true>(a, sms, st);
  };
  return a.dt == MUON_BF16 ? go(__nv_bfloat16()) : a.dt == MUON_FP16 ? go(__half()) : go(float());
}

}  // namespace muon
