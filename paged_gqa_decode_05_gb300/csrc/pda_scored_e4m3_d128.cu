// Scored split kernels over e4m3 caches for head_dim 128.
#include "pda_scored.cuh"

namespace pda {

ScoredShape scored_shape_e4m3_d128(const ScoredForm& f) { return scored_shape_quant<128, kE4m3>(f); }
cudaError_t launch_scored_e4m3_d128(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_scored_quant<128, kE4m3>(f, p, grid, smem, stream);
}

}  // namespace pda
