// Tree attention, f16 queries.
#include "tree_dispatch.cuh"

namespace da {

cudaError_t launch_tree_f16(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, const TreeSpace& space,
                            cudaStream_t stream) {
  return launch_tree_as<__half>(l, head_dim, e4m3, ctas, space, stream);
}

}  // namespace da
