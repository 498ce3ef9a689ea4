// attention_tree4_f16.cu - attention over a cache of 4 bits, float16.
#include "attention_tree4.cuh"

namespace gsr {

cudaError_t launch_tree4_f16(const Tree4Params& p, const Tree4Split& split, cudaStream_t stream) { return launch_tree4_type<__half>(p, split, stream); }

}  // namespace gsr
