// k_tree_q8.cu - the tree attention over q8_0 rows (tree_kernel.cuh).
#include "tree_kernel.cuh"

namespace kvc {
cudaError_t launch_tree_q8(const BlockParams &p, const TreeMaps &t, cudaStream_t st) {
    return p.D == 64 ? tree_pick<64, KVC_Q8_0, KVC_Q8_0>(p, t, st) : tree_pick<128, KVC_Q8_0, KVC_Q8_0>(p, t, st);
}
} // namespace kvc
