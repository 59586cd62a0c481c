// block_norm_fp16.cu -- the norms around a block: fp16 rows.
#include "block_norm_rows.cuh"

namespace muon {

template cudaError_t launch_block_norm_rows<__half>(const muon_block_norm_args&, int, int, cudaStream_t);

}  // namespace muon
