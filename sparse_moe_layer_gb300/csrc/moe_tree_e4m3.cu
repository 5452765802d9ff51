// Attention of drafted tokens over e4m3 caches (a unit of its own, so that the builds run side by side).
#include "moe_tree.cuh"

namespace moe {

cudaError_t launch_tree_e4m3(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p, const TreePlan& w,
                             cudaStream_t st) {
    return launch_tree_d<kKvE4m3>(tmK, tmV, p, w, st);
}

}  // namespace moe
