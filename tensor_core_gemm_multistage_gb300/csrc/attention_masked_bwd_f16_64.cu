// attention_masked_bwd_f16_64.cu - gradients of masked attention for f16 operands, head_dim 64.
#include "attention_masked_bwd.cuh"

namespace gsr {

cudaError_t launch_masked_bwd_f16_64(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    return launch_bwd_type<__half, 64>(tm, p, stream);
}

}  // namespace gsr
