// Scored split kernels over bf16 caches for head_dim 64.
#include "pda_scored.cuh"

namespace pda {

ScoredShape scored_shape_bf16_d64(const ScoredForm& f) { return scored_shape_bf16<64>(f); }
cudaError_t launch_scored_bf16_d64(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_scored_bf16<64>(f, p, grid, smem, stream);
}

}  // namespace pda
