// block_norm_grad_fp32.cu -- gradient of the norms around a block: fp32 rows.
#include "block_norm_grad.cuh"

namespace muon {

template cudaError_t launch_block_norm_grad_rows<float>(const muon_block_norm_grad_args&, float*, int, int, int*, cudaStream_t);

}  // namespace muon
