// attention_masked_bwd_f16_128.cu - gradients of masked attention for f16 operands, head_dim 128.
#include "attention_masked_bwd.cuh"

namespace gsr {

cudaError_t launch_masked_bwd_f16_128(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    return launch_bwd_type<__half, 128>(tm, p, stream);
}

}  // namespace gsr
