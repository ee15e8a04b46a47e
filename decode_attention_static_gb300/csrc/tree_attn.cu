// Attention of several new tokens of each sequence over a paged cache: the join
// of units that several CTAs took, the workspace, and the choice of instance.
//
// The join is a kernel of its own: the parts of a unit are up to 256 rows of
// fp32 each, which the last CTA to arrive would read alone; here 8 CTAs a unit
// do, 32 rows each. It waits for the first kernel by programmatic dependent
// launch.
#include <stdint.h>

#include <algorithm>

#include "decode_attn.h"
#include "launch.h"
#include "tree_attn.cuh"

namespace da {

namespace {

constexpr int kMaxCtas = 256;
constexpr int kJoinBytes = kMaxCtas * (int)sizeof(TreeJoin);
constexpr int kJoinThreads = 256;

int tree_ctas(int sms) { return std::min(sms, kMaxCtas); }

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
    tree_join_kernel(const TreeJoin* joins, const float* partials, uint8_t* out_bytes, int n_head, int group) {
  pdl_wait();
  pdl_trigger();
  const TreeJoin j = joins[blockIdx.x];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, row = blockIdx.y * 32 + lane;
  if (blockIdx.y * 32 >= (unsigned)j.rows || row >= j.rows) return;
  // the first CTA's part is its second state, the others' their first
  auto slot = [&](int c) {
    return partials + ((int64_t)c * 2 + (c == (int)blockIdx.x ? 1 : 0)) * tree_slot_floats(D);
  };
  auto state = [&](int c) { return reinterpret_cast<const float4*>(slot(c) + kTreeUnitRows * D)[row]; };
  float m = -INFINITY, ml = -INFINITY;
  for (int c = blockIdx.x; c <= j.last; ++c) {
    const float4 s = state(c);
    m = fmaxf(m, s.x);
    ml = fmaxf(ml, s.y);
  }
  const float m0 = m == -INFINITY ? 0.f : m, ml0 = ml == -INFINITY ? 0.f : ml;
  float l = 0.f;
  constexpr int kEach = D / 32;  // groups of four columns of a thread
  float4 acc[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = blockIdx.x; c <= j.last; ++c) {
    const float4 s = state(c);
    const float w = fast_exp2(s.x - m0);
    l += s.z * fast_exp2(s.y - ml0);
    const float4* const o = reinterpret_cast<const float4*>(slot(c)) + (row / kTreeTile) * (D / 4) * kTreeTile + row % kTreeTile;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const float4 x = o[(warp + 8 * k) * kTreeTile];
      acc[k].x = fmaf(x.x, w, acc[k].x);
      acc[k].y = fmaf(x.y, w, acc[k].y);
      acc[k].z = fmaf(x.z, w, acc[k].z);
      acc[k].w = fmaf(x.w, w, acc[k].w);
    }
  }
  const float inv = l == 0.f ? 0.f : fast_exp2(m0 - ml0) / l;
  uint16_t* const out = reinterpret_cast<uint16_t*>(out_bytes) +
                        ((int64_t)(j.token0 + row / group) * n_head + j.g * group + row % group) * D;
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    *reinterpret_cast<uint2*>(out + 4 * (warp + 8 * k)) =
        make_uint2(pack2<Storage<T>::kBf16>(acc[k].x * inv, acc[k].y * inv),
                   pack2<Storage<T>::kBf16>(acc[k].z * inv, acc[k].w * inv));
}

template <typename T, int D>
cudaError_t launch_join(const TreeLaunch& l, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, kTreeUnitRows / 32);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D>, static_cast<const TreeJoin*>(l.p.workspace),
                            reinterpret_cast<const float*>(static_cast<const uint8_t*>(l.p.workspace) + kJoinBytes),
                            l.p.out, l.p.n_head, l.p.group);
}

}  // namespace

size_t tree_workspace_bytes(int sms, int group, int head_dim) {
  return kJoinBytes + (size_t)tree_ctas(sms) * 2 * tree_slot_floats(head_dim) * sizeof(float);
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
  TreeJoin* const joins = static_cast<TreeJoin*>(p.workspace);
  float* const partials = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kJoinBytes);
  const int ctas = tree_ctas(sms);
  const cudaError_t e = dtype == DA_F16 ? launch_tree_f16(l, head_dim, e4m3, ctas, joins, partials, stream)
                                        : launch_tree_bf16(l, head_dim, e4m3, ctas, joins, partials, stream);
  if (e != cudaSuccess) return e;
  if (dtype == DA_F16)
    return head_dim == 128 ? launch_join<__half, 128>(l, ctas, stream) : launch_join<__half, 64>(l, ctas, stream);
  return head_dim == 128 ? launch_join<__nv_bfloat16, 128>(l, ctas, stream)
                         : launch_join<__nv_bfloat16, 64>(l, ctas, stream);
}

}  // namespace da
