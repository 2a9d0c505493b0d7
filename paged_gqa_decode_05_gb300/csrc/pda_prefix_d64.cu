// The shared-prefix kernel for head_dim 64.
#include "pda_prefix.cuh"

namespace pda {

PrefixShape prefix_shape_d64(int format) { return prefix_shape_of<64>(format); }
cudaError_t launch_prefix_d64(int format, const PrefixParams& p, int ctas, cudaStream_t stream) {
    return launch_prefix_of<64>(format, p, ctas, stream);
}

}  // namespace pda
