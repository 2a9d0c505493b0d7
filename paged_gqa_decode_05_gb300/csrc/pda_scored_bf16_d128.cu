// Scored split kernels over bf16 caches for head_dim 128.
#include "pda_scored.cuh"

namespace pda {

ScoredShape scored_shape_bf16_d128(const ScoredForm& f) { return scored_shape_bf16<128>(f); }
cudaError_t launch_scored_bf16_d128(const ScoredForm& f, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_scored_bf16<128>(f, p, grid, smem, stream);
}

}  // namespace pda
