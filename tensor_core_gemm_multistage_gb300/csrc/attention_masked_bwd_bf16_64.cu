// attention_masked_bwd_bf16_64.cu - gradients of masked attention for bf16 operands, head_dim 64.
#include "attention_masked_bwd.cuh"

namespace gsr {

cudaError_t launch_masked_bwd_bf16_64(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    return launch_bwd_type<__nv_bfloat16, 64>(tm, p, stream);
}

}  // namespace gsr
