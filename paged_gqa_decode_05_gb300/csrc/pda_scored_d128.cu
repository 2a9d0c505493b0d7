// kScored instances for head_dim 128.
#include "pda_scored.cuh"

namespace pda {

ScoredShape scored_shape_d128(int st, int format, bool fine) { return scored_shape_of<128>(st, format, fine); }
cudaError_t launch_scored_d128(int st, int format, bool fine, const QuantParams& p, int grid, size_t smem, cudaStream_t stream) {
    return launch_scored_of<128>(st, format, fine, p, grid, smem, stream);
}

}  // namespace pda
