// The shared-prefix kernel for head_dim 128.
#include "pda_prefix.cuh"

namespace pda {

PrefixShape prefix_shape_d128(int format) { return prefix_shape_of<128>(format); }
cudaError_t launch_prefix_d128(int format, const PrefixParams& p, int ctas, cudaStream_t stream) {
    return launch_prefix_of<128>(format, p, ctas, stream);
}

}  // namespace pda
