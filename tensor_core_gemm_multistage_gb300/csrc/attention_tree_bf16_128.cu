// attention_tree_bf16_128.cu - tree attention over a paged cache for bf16 operands, head_dim 128.
#include "attention_tree.cuh"

namespace gsr {

cudaError_t launch_tree_bf16_128(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream) {
    return launch_tree_type<__nv_bfloat16, 128>(tm, p, grid, stream);
}

}  // namespace gsr
