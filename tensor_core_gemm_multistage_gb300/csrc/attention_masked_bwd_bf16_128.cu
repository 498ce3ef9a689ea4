// attention_masked_bwd_bf16_128.cu - gradients of masked attention for bf16 operands, head_dim 128.
#include "attention_masked_bwd.cuh"

namespace gsr {

cudaError_t launch_masked_bwd_bf16_128(const MaskedBwdMaps& tm, const MaskedBwdParams& p, cudaStream_t stream) {
    return launch_bwd_type<__nv_bfloat16, 128>(tm, p, stream);
}

}  // namespace gsr
