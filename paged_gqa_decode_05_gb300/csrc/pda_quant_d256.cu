// 8-bit split-kernel instantiations for head_dim 256.
#include "pda_quant.cuh"

namespace pda {

const void* quant_fn_d256(int format, int n_tiles, bool multi) { return quant_fn<256>(format, n_tiles, multi); }

cudaError_t launch_quant_d256(int format, int n_tiles, bool multi, const QuantParams& p, int grid, size_t smem,
                            cudaStream_t stream) {
    return launch_quant_of<256>(format, n_tiles, multi, p, grid, smem, stream);
}

}  // namespace pda
