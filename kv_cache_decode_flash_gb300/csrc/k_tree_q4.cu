// k_tree_q4.cu - the tree attention over q8_0 K and q4_0 V rows (tree_kernel.cuh).
#include "tree_kernel.cuh"

namespace kvc {
cudaError_t launch_tree_q4(const BlockParams &p, const TreeMaps &t, cudaStream_t st) {
    return tree_pick<128, KVC_Q8_0, KVC_Q4_0>(p, t, st);
}
} // namespace kvc
