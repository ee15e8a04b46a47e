// Attention of several new tokens of each sequence over a paged cache.
//
// One CTA for each (token, KV head), one thread for each column: a tile of D
// rows is scored a row a thread, weighted a column a thread.
#include <stdint.h>

#include "common.cuh"
#include "decode_attn.h"
#include "tree_params.h"

namespace da {

namespace {

// Tokens and rows of sequence b: 0 to be skipped, 1 valid, -1 NaN rows.
__device__ __forceinline__ int tree_sequence(const TreeParams& p, int b, int* first, int* count, int* rows,
                                             int* errors) {
  int a = b, n = 1;
  if (p.start) {
    a = p.start[b];
    const int e = p.start[b + 1];
    if (a < 0 || e < a || e > p.tokens) {
      *errors |= kErrTokens;
      return 0;
    }
    n = e - a;
  }
  *first = a;
  *count = n;
  if (n == 0) return 0;
  if (n > kTreeMaxTokens || (p.mask && n > 64 * p.mask_words)) {
    *errors |= kErrTokens;
    return -1;
  }
  *rows = p.kv_len[b];
  if (*rows < n || *rows > p.max_pages << p.page_shift) {
    *errors |= kErrKvLen;
    return -1;
  }
  return 1;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h)).x;
}

template <typename T, bool EIGHT>
__global__ void tree_simple_kernel(const TreeParams p, int D) {
  __shared__ float q[128], x[128], scale_v[128];
  __shared__ float red[4];
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, h = blockIdx.y, g = h / p.group, d = threadIdx.x;
  int b = t, first = 0, count = 0, rows = 0, errors = 0;
  if (p.start) {
    for (b = 0; b < p.B; ++b) {
      const int s = p.start[b], e = p.start[b + 1];
      if (s >= 0 && e <= p.tokens && t >= s && t < e) break;
    }
  }
  const int64_t at = ((int64_t)t * p.n_head + h) * D + d;
  int state = b < p.B ? tree_sequence(p, b, &first, &count, &rows, &errors) : 0;
  if (t == 0 && h == 0) {
    for (int i = d; i < p.B; i += D) {
      int f, c, r;
      tree_sequence(p, i, &f, &c, &r, &errors);
    }
  }
  const int32_t* table = p.table + (int64_t)b * p.max_pages;
  if (state == 1) {
    for (int j = 0; j < (rows + p.page_rows - 1) >> p.page_shift; ++j)
      if (table[j] < 0 || table[j] >= p.num_pages) state = -1, errors |= kErrPage;
  }
  if (errors && p.err_flag) atomicOr(p.err_flag, errors);
  if (state == 0) return;
  T* out = reinterpret_cast<T*>(p.out) + at;
  if (state < 0) {
    reinterpret_cast<uint16_t*>(p.out)[at] = Storage<T>::kNaN;
    return;
  }
  q[d] = to_f32(reinterpret_cast<const T*>(p.q)[at]);
  const int base = rows - count, me = t - first;
  auto seen = [&](int j) {
    if (j < base) return j < rows;
    if (j >= rows) return false;
    const int i = j - base;
    return p.mask ? (p.mask[(int64_t)t * p.mask_words + i / 64] >> (i % 64) & 1) != 0 : i <= me;
  };
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 < rows; j0 += D) {
    __syncthreads();
    const int j = j0 + d;
    float s = -INFINITY;
    if (seen(j)) {
      const int id = table[j >> p.page_shift];
      const int64_t block = (int64_t)id * p.n_kv_head + g;
      const int64_t row = (block * p.page_rows + (j & (p.page_rows - 1))) * D;
      s = 0.f;
      for (int e = 0; e < D; ++e)
        s += q[e] * (EIGHT ? e4m3_f32(p.k[row + e]) : to_f32(reinterpret_cast<const T*>(p.k)[row + e]));
      if (EIGHT) s *= p.k_scale[block];
      if (EIGHT) scale_v[d] = p.v_scale[block];
      s *= p.qscale;
    }
    float top = s;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (d % 32 == 0) red[d / 32] = top;
    __syncthreads();
    top = m;
    for (int w = 0; w < D / 32; ++w) top = fmaxf(top, red[w]);
    const float ref = top == -INFINITY ? 0.f : top;
    x[d] = seen(j) ? exp2f(s - ref) : -1.f;
    __syncthreads();
    const float keep = exp2f(m - ref);
    acc *= keep;
    l *= keep;
    m = top;
    for (int r = 0; r < D && j0 + r < rows; ++r) {
      if (x[r] == -1.f) continue;
      const int jr = j0 + r;
      const int64_t block = (int64_t)table[jr >> p.page_shift] * p.n_kv_head + g;
      const int64_t row = (block * p.page_rows + (jr & (p.page_rows - 1))) * D + d;
      l += x[r];
      acc += x[r] * (EIGHT ? e4m3_f32(p.v[row]) * scale_v[r] : to_f32(reinterpret_cast<const T*>(p.v)[row]));
    }
  }
  *reinterpret_cast<uint16_t*>(out) = Storage<T>::round(l == 0.f ? 0.f : acc / l);
}

}  // namespace

size_t tree_workspace_bytes(int sms, int group, int head_dim) { return 16; }

cudaError_t launch_tree(const TreeParams& p, int dtype, int head_dim, bool e4m3, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.tokens, p.n_head);
  cfg.blockDim = dim3(head_dim);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (dtype == DA_F16)
    return e4m3 ? cudaLaunchKernelEx(&cfg, tree_simple_kernel<__half, true>, p, head_dim)
                : cudaLaunchKernelEx(&cfg, tree_simple_kernel<__half, false>, p, head_dim);
  return e4m3 ? cudaLaunchKernelEx(&cfg, tree_simple_kernel<__nv_bfloat16, true>, p, head_dim)
              : cudaLaunchKernelEx(&cfg, tree_simple_kernel<__nv_bfloat16, false>, p, head_dim);
}

}  // namespace da
