// Attention of drafted tokens over fp16 caches (a unit of its own, so that the builds run side by side).
#include "moe_tree.cuh"

namespace moe {

cudaError_t launch_tree_fp16(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p, const TreePlan& w,
                             cudaStream_t st) {
    return launch_tree_d<kKvFp16>(tmK, tmV, p, w, st);
}

}  // namespace moe
