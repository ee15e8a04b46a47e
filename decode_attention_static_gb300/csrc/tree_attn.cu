// Attention of several new tokens of each sequence over a paged cache: the
// workspace, the tensor maps and the choice of instance.
#include <stdint.h>

#include <algorithm>

#include "decode_attn.h"
#include "launch.h"
#include "tree_attn.cuh"

namespace da {

namespace {

constexpr int kMaxCtas = 256;
constexpr int kMeetBytes = kCounterBytes + kMaxCtas * (int)sizeof(TreeMeet);
static_assert(kMaxCtas <= kMaxCounterGroups && kMeetBytes % 16 == 0, "layout of the workspace");

int tree_ctas(int sms) { return std::min(sms, kMaxCtas); }

}  // namespace

size_t tree_workspace_bytes(int sms, int group, int head_dim) {
  return kMeetBytes + (size_t)tree_ctas(sms) * 2 * tree_slot_floats(head_dim) * sizeof(float);
}

cudaError_t launch_tree(const TreeParams& p, int dtype, int head_dim, bool e4m3, int sms, cudaStream_t stream) {
  TreeLaunch l = {};
  l.p = p;
  if (!e4m3) {
    const int64_t rows = (int64_t)p.num_pages * p.n_kv_head * p.page_rows;
    const int box = std::min(p.page_rows, kTreeTile);
    if (!encode_rows_map(&l.k_map, p.k, dtype, rows, head_dim, box) ||
        !encode_rows_map(&l.v_map, p.v, dtype, rows, head_dim, box))
      return cudaErrorInvalidValue;
  }
  uint8_t* const at = static_cast<uint8_t*>(p.workspace);
  const TreeSpace space = {reinterpret_cast<unsigned*>(at), reinterpret_cast<TreeMeet*>(at + kCounterBytes),
                           reinterpret_cast<float*>(at + kMeetBytes)};
  const int ctas = tree_ctas(sms);
  return dtype == DA_F16 ? launch_tree_f16(l, head_dim, e4m3, ctas, space, stream)
                         : launch_tree_bf16(l, head_dim, e4m3, ctas, space, stream);
}

}  // namespace da
