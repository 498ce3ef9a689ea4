// attention_tree4_bf16.cu - attention over a cache of 4 bits, bfloat16.
#include "attention_tree4.cuh"

namespace gsr {

cudaError_t launch_tree4_bf16(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream) { return launch_tree4_type<__nv_bfloat16>(p, split, stream); }

}  // namespace gsr
