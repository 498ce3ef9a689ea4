// attention_masked_fwd_f16.cu - masked attention forward for f16 operands.
#include "attention_masked_fwd.cuh"

namespace gsr {

cudaError_t launch_masked_fwd_f16(const MaskedFwdMaps& tm, const MaskedFwdParams& p, int D, cudaStream_t stream) {
    return D == 64 ? launch_masked_type<__half, 64>(tm, p, stream) : launch_masked_type<__half, 128>(tm, p, stream);
}

}  // namespace gsr
