// k_tree_f16.cu - the tree attention over f16 rows (tree_kernel.cuh).
#include "tree_kernel.cuh"

namespace kvc {
cudaError_t launch_tree_f16(const BlockParams &p, const TreeMaps &t, cudaStream_t st) {
    return p.D == 64 ? tree_pick<64, KVC_F16, KVC_F16>(p, t, st) : tree_pick<128, KVC_F16, KVC_F16>(p, t, st);
}
} // namespace kvc
