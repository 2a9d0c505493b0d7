// 8-bit split-kernel instantiations for head_dim 64.
#include "pda_quant.cuh"

namespace pda {

const void* quant_fn_d64(const QuantForm& form) { return quant_fn<64>(form); }

cudaError_t launch_quant_d64(const QuantForm& form, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_quant_of<64>(form, p, grid, smem, stream);
}

}  // namespace pda
