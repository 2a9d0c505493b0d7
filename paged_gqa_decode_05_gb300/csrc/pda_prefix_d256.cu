// The shared-prefix kernel for head_dim 256.
#include "pda_prefix.cuh"

namespace pda {

PrefixShape prefix_shape_d256(int format) { return prefix_shape_of<256>(format); }
cudaError_t launch_prefix_d256(int format, const PrefixParams& p, int ctas, cudaStream_t stream) {
    return launch_prefix_of<256>(format, p, ctas, stream);
}

}  // namespace pda
