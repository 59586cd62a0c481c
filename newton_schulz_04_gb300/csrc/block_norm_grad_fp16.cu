// block_norm_grad_fp16.cu -- gradient of the norms around a block: fp16 rows.
#include "block_norm_grad.cuh"

namespace muon {

template cudaError_t launch_block_norm_grad_rows<__half>(const muon_block_norm_grad_args&, float*, int, int, int*, cudaStream_t);

}  // namespace muon
