// attention_tree_f16_64.cu - tree attention over a paged cache for f16 operands, head_dim 64.
#include "attention_tree.cuh"

namespace gsr {

cudaError_t launch_tree_f16_64(const TreeMaps& tm, const TreeParams& p, int grid, cudaStream_t stream) {
    return launch_tree_type<__half, 64>(tm, p, grid, stream);
}

}  // namespace gsr
