// block_norm_fp32.cu -- the norms around a block: fp32 rows.
#include "block_norm_rows.cuh"

namespace muon {

template cudaError_t launch_block_norm_rows<float>(const muon_block_norm_args&, int, int, cudaStream_t);

}  // namespace muon
