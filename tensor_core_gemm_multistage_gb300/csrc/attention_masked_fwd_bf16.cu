// attention_masked_fwd_bf16.cu - masked attention forward for bf16 operands.
#include "attention_masked_fwd.cuh"

namespace gsr {

cudaError_t launch_masked_fwd_bf16(const MaskedFwdMaps& tm, const MaskedFwdParams& p, int D, cudaStream_t stream) {
    return D == 64 ? launch_masked_type<__nv_bfloat16, 64>(tm, p, stream) : launch_masked_type<__nv_bfloat16, 128>(tm, p, stream);
}

}  // namespace gsr
