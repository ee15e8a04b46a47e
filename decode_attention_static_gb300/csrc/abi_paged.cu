// C ABI of the paged-cache and sliding-window operators: argument validation
// and the launches on the caller's stream. Nothing here allocates or
// synchronises.
#include <stdint.h>

#include "cache_params.h"
#include "decode_attn.h"
#include "launch.h"
#include "tree_params.h"

namespace da {

cudaError_t launch_cache_attn(const CacheAttnParams& p, int dtype, int head_dim, bool e4m3, int sms,
                              cudaStream_t stream) {
  return dtype == DA_F16 ? launch_cache_attn_f16(p, head_dim, e4m3, sms, stream)
                         : launch_cache_attn_bf16(p, head_dim, e4m3, sms, stream);
}

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Sizes that the attention entry points share.
int check_heads(int B, int n_head, int n_kv_head, int head_dim, int dtype) {
  if (dtype != DA_F16 && dtype != DA_BF16) return DA_ERR_DTYPE;
  if (B < 0 || n_head < 1 || n_kv_head < 1 || head_dim < 1) return DA_ERR_SHAPE;
  if (n_head % n_kv_head != 0 || B > kMaxBatch || n_kv_head > kMaxBatch) return DA_ERR_SHAPE;
  if (!decode_supported(head_dim, n_head / n_kv_head)) return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

int check_pages(int num_pages, int page_size, int max_pages) {
  if (num_pages < 1 || page_size < 1 || max_pages < 1) return DA_ERR_SHAPE;
  if (page_size < kMinPageSize || page_size > kMaxPageSize || (page_size & (page_size - 1)) != 0)
    return DA_ERR_UNSUPPORTED;
  // row numbers are 32-bit, with room for a tile past the last one
  if ((int64_t)max_pages * page_size > INT32_MAX - 2 * kMaxPageSize) return DA_ERR_SHAPE;
  return DA_OK;
}

int run_attention(CacheAttnParams p, int head_dim, bool e4m3, float scale, void* workspace, size_t workspace_bytes,
                  int dtype, void* stream) {
  // the kernel numbers the 16-row tiles of a CTA's share (at least 1 / 128 of
  // all) in 32 bits
  if ((int64_t)p.B * p.n_kv_head * ((int64_t)p.max_len / 16 + 32) >= (1ll << 37)) return DA_ERR_SHAPE;
  if (!p.q || !p.k || !p.v || !p.kv_len || !p.out) return DA_ERR_NULL;
  if (p.out == p.q) return DA_ERR_SHAPE;  // CTAs read q while others write out
  if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.out, 16)) return DA_ERR_ALIGN;
  if (!aligned(p.kv_len, 4) || !aligned(p.table, 4) || !aligned(p.k_scale, 4) || !aligned(p.v_scale, 4) ||
      !aligned(p.err_flag, 4))
    return DA_ERR_ALIGN;
  int sms = 0;
  if (current_device_sms(&sms) != cudaSuccess) return DA_ERR_CUDA;
  const size_t need = cache_attn_workspace_bytes(sms, p.group, head_dim);
  if (!workspace || workspace_bytes < need) return DA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return DA_ERR_ALIGN;
  p.counters = static_cast<unsigned int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  p.qscale = scale * kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!record_timing_before(st)) return DA_ERR_CUDA;
  if (launch_cache_attn(p, dtype, head_dim, e4m3, sms, st) != cudaSuccess) return DA_ERR_CUDA;
  if (!record_timing_after(st)) return DA_ERR_CUDA;
  return DA_OK;
}

int paged_attention(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                    const float* v_scale, bool e4m3, const int32_t* page_table, const int32_t* kv_len, int B,
                    int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int window,
                    int sinks, float scale, void* out, void* workspace, size_t workspace_bytes, int dtype,
                    int32_t* err_flag, void* stream) {
  int rc = check_heads(B, n_head, n_kv_head, head_dim, dtype);
  if (rc == DA_OK) rc = check_pages(num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return DA_ERR_SHAPE;
  if (B == 0) return DA_OK;
  if (!page_table || (e4m3 && (!k_scale || !v_scale))) return DA_ERR_NULL;
  CacheAttnParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_pages);
  p.v = static_cast<const uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.kv_len = kv_len;
  p.B = B;
  p.n_head = n_head;
  p.n_kv_head = n_kv_head;
  p.group = n_head / n_kv_head;
  p.num_pages = num_pages;
  p.page_rows = page_size;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  p.max_len = max_pages * page_size;
  p.window = window;
  p.sinks = sinks;
  p.out = static_cast<uint8_t*>(out);
  p.err_flag = err_flag;
  return run_attention(p, head_dim, e4m3, scale, workspace, workspace_bytes, dtype, stream);
}

// Rotary positions of their own (kvcache_append_paged_axes).
struct Turns {
  const int32_t* rows;
  const int32_t* axis;
  int axes;
};

int append_paged(void* k_pages, void* v_pages, float* k_scale, float* v_scale, bool e4m3, const void* k_new,
                 const void* v_new, const void* q, void* q_out, const float* rope_cos, const float* rope_sin,
                 int rope_rows, const int32_t* page_table, const int32_t* position_ids, const int32_t* token_start,
                 int B, int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size,
                 int max_pages, int dtype, int32_t* err_flag, void* stream, const Turns* turns = nullptr) {
  if (dtype != DA_F16 && dtype != DA_BF16) return DA_ERR_DTYPE;
  if (B < 0 || tokens < 0 || n_kv_head < 1 || head_dim < 1) return DA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return DA_ERR_UNSUPPORTED;
  const int rc = check_pages(num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (token_start ? B == 0 && tokens > 0 : tokens != B) return DA_ERR_SHAPE;
  if (q && n_head < 1) return DA_ERR_SHAPE;
  if (turns && (turns->axes < 1 || turns->axes > kMaxRopeAxes)) return DA_ERR_SHAPE;
  if (B == 0 || tokens == 0) return DA_OK;
  if (turns && (!turns->rows || !rope_cos)) return DA_ERR_NULL;
  if (turns && (!aligned(turns->rows, 4) || !aligned(turns->axis, 16))) return DA_ERR_ALIGN;
  if (!k_pages || !v_pages || !k_new || !v_new || !page_table || !position_ids) return DA_ERR_NULL;
  if (e4m3 && (!k_scale || !v_scale)) return DA_ERR_NULL;
  if ((rope_cos != nullptr) != (rope_sin != nullptr)) return DA_ERR_NULL;
  if (q && (!q_out || !rope_cos)) return DA_ERR_NULL;
  if (rope_cos && rope_rows < 1) return DA_ERR_SHAPE;
  if (k_pages == v_pages || (e4m3 && k_scale == v_scale)) return DA_ERR_SHAPE;  // K and V need arrays of their own
  const void* wide[] = {k_pages, v_pages, k_new, v_new, q, q ? q_out : nullptr, rope_cos, rope_sin};
  for (const void* w : wide)
    if (!aligned(w, 16)) return DA_ERR_ALIGN;
  const void* words[] = {page_table, position_ids, token_start, k_scale, v_scale, err_flag};
  for (const void* w : words)
    if (!aligned(w, 4)) return DA_ERR_ALIGN;
  AppendPagedParams p = {};
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_new = static_cast<const uint8_t*>(k_new);
  p.v_new = static_cast<const uint8_t*>(v_new);
  p.q = static_cast<const uint8_t*>(q);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.cos = rope_cos;
  p.sin = rope_sin;
  p.table = page_table;
  p.pos = position_ids;
  p.start = token_start;
  p.B = B;
  p.tokens = tokens;
  p.n_head = n_head;
  p.n_kv_head = n_kv_head;
  p.head_dim = head_dim;
  p.num_pages = num_pages;
  p.page_rows = page_size;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  p.limit = max_pages * page_size;
  if (turns) {
    p.turn = turns->rows;
    p.axis = turns->axis;
    p.axes = turns->axes;
    p.rope_rows = rope_rows;
  } else if (rope_cos && rope_rows < p.limit) {
    p.limit = rope_rows;
  }
  p.err_flag = err_flag;
  int sms = 0;
  if (current_device_sms(&sms) != cudaSuccess) return DA_ERR_CUDA;
  return launch_append_paged(p, dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

int tree_attention(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                   const float* v_scale, bool e4m3, const int32_t* page_table, const int32_t* kv_len,
                   const int32_t* token_start, const int64_t* tree_mask, int mask_words, int B, int tokens, int n_head,
                   int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, float scale, void* out,
                   void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag, void* stream) {
  int rc = check_heads(B, n_head, n_kv_head, head_dim, dtype);
  if (rc == DA_OK) rc = check_pages(num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (tokens < 0 || (token_start ? B == 0 && tokens > 0 : tokens != B)) return DA_ERR_SHAPE;
  if (tree_mask && (mask_words < 1 || mask_words > kTreeMaxWords)) return DA_ERR_SHAPE;
  // tokens and rows of pools are 32-bit coordinates of tensor copies, tiles are numbered in 32 bits
  if ((int64_t)num_pages * n_kv_head * page_size > INT32_MAX) return DA_ERR_SHAPE;
  if ((int64_t)B * n_kv_head * (kTreeMaxTokens * (n_head / n_kv_head) / 256) *
          (((int64_t)max_pages * page_size + 127) / 128 + 8) > INT32_MAX)
    return DA_ERR_SHAPE;
  if (B == 0 || tokens == 0) return DA_OK;
  if (!q || !k_pages || !v_pages || !page_table || !kv_len || !out || (e4m3 && (!k_scale || !v_scale)))
    return DA_ERR_NULL;
  if (out == q) return DA_ERR_SHAPE;  // CTAs read q while others write out
  for (const void* w : {q, k_pages, v_pages, static_cast<const void*>(out)})
    if (!aligned(w, 16)) return DA_ERR_ALIGN;
  for (const void* w : {static_cast<const void*>(page_table), static_cast<const void*>(kv_len),
                        static_cast<const void*>(token_start), static_cast<const void*>(k_scale),
                        static_cast<const void*>(v_scale), static_cast<const void*>(err_flag)})
    if (!aligned(w, 4)) return DA_ERR_ALIGN;
  if (!aligned(tree_mask, 8)) return DA_ERR_ALIGN;
  int sms = 0;
  if (current_device_sms(&sms) != cudaSuccess) return DA_ERR_CUDA;
  if (!workspace || workspace_bytes < tree_workspace_bytes(sms, n_head / n_kv_head, head_dim)) return DA_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return DA_ERR_ALIGN;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), out0 = reinterpret_cast<uintptr_t>(out);
  const uint64_t bytes = (uint64_t)tokens * n_head * head_dim * 2;
  if (out0 < q0 + bytes && q0 < out0 + bytes) return DA_ERR_SHAPE;  // nor any part of it
  TreeParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_pages);
  p.v = static_cast<const uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.kv_len = kv_len;
  p.start = token_start;
  p.mask = reinterpret_cast<const uint64_t*>(tree_mask);
  p.mask_words = mask_words;
  p.B = B;
  p.tokens = tokens;
  p.n_head = n_head;
  p.n_kv_head = n_kv_head;
  p.group = n_head / n_kv_head;
  p.num_pages = num_pages;
  p.page_rows = page_size;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  p.qscale = scale * kLog2e;
  p.out = static_cast<uint8_t*>(out);
  p.workspace = workspace;
  p.err_flag = err_flag;
  p.skip_slot = skipped_slot();
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!record_timing_before(st)) return DA_ERR_CUDA;
  if (launch_tree(p, dtype, head_dim, e4m3, sms, st) != cudaSuccess) return DA_ERR_CUDA;
  if (!record_timing_after(st)) return DA_ERR_CUDA;
  return DA_OK;
}

}  // namespace

size_t cache_attn_workspace_bytes(int sms, int group, int head_dim) {
  return kCounterBytes + (size_t)cache_attn_ctas(sms) * 2 * cache_attn_slot_floats(group, head_dim) * sizeof(float);
}

}  // namespace da

extern "C" {

size_t decode_attn_paged_workspace_size(int n_head, int n_kv_head, int head_dim) {
  if (da::check_heads(1, n_head, n_kv_head, head_dim, DA_F16) != DA_OK) return (size_t)-1;
  int sms = 0;
  if (da::current_device_sms(&sms) != cudaSuccess) return (size_t)-1;
  return da::cache_attn_workspace_bytes(sms, n_head / n_kv_head, head_dim);
}

int decode_attn_paged_fwd(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                          const int32_t* kv_len, int B, int n_head, int n_kv_head, int head_dim, int num_pages,
                          int page_size, int max_pages, int window, int sinks, float scale, void* out,
                          void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag, void* stream) {
  return da::paged_attention(q, k_pages, v_pages, nullptr, nullptr, false, page_table, kv_len, B, n_head, n_kv_head,
                             head_dim, num_pages, page_size, max_pages, window, sinks, scale, out, workspace,
                             workspace_bytes, dtype, err_flag, stream);
}

int decode_attn_paged_q8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                             const float* v_scale, const int32_t* page_table, const int32_t* kv_len, int B,
                             int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages,
                             int window, int sinks, float scale, void* out, void* workspace, size_t workspace_bytes,
                             int dtype, int32_t* err_flag, void* stream) {
  return da::paged_attention(q, k_pages, v_pages, k_scale, v_scale, true, page_table, kv_len, B, n_head, n_kv_head,
                             head_dim, num_pages, page_size, max_pages, window, sinks, scale, out, workspace,
                             workspace_bytes, dtype, err_flag, stream);
}

int decode_attn_window_fwd(const void* q, const void* k_cache, const void* v_cache, const int32_t* kv_len, int B,
                           int n_head, int n_kv_head, int head_dim, int capacity, int window, int sinks, float scale,
                           void* out, void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag,
                           void* stream) {
  const int rc = da::check_heads(B, n_head, n_kv_head, head_dim, dtype);
  if (rc != DA_OK) return rc;
  if (capacity < 1 || capacity > INT32_MAX - 2 * da::kMaxPageSize || window < 1 || sinks < 0) return DA_ERR_SHAPE;
  if (B == 0) return DA_OK;
  da::CacheAttnParams p = {};
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.kv_len = kv_len;
  p.B = B;
  p.n_head = n_head;
  p.n_kv_head = n_kv_head;
  p.group = n_head / n_kv_head;
  p.num_pages = B;
  p.page_rows = capacity;
  p.page_shift = 31;  // every row is in the sequence's one page
  p.max_pages = 1;
  p.max_len = capacity;
  p.window = window;
  p.sinks = sinks;
  p.out = static_cast<uint8_t*>(out);
  p.err_flag = err_flag;
  return da::run_attention(p, head_dim, false, scale, workspace, workspace_bytes, dtype, stream);
}

int kvcache_append_paged(void* k_pages, void* v_pages, const void* k_new, const void* v_new, const void* q,
                         void* q_out, const float* rope_cos, const float* rope_sin, int rope_rows,
                         const int32_t* page_table, const int32_t* position_ids, const int32_t* token_start, int B,
                         int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size,
                         int max_pages, int dtype, int32_t* err_flag, void* stream) {
  return da::append_paged(k_pages, v_pages, nullptr, nullptr, false, k_new, v_new, q, q_out, rope_cos, rope_sin,
                          rope_rows, page_table, position_ids, token_start, B, tokens, n_head, n_kv_head, head_dim,
                          num_pages, page_size, max_pages, dtype, err_flag, stream);
}

int kvcache_append_paged_q8(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const void* k_new,
                            const void* v_new, const void* q, void* q_out, const float* rope_cos,
                            const float* rope_sin, int rope_rows, const int32_t* page_table,
                            const int32_t* position_ids, const int32_t* token_start, int B, int tokens, int n_head,
                            int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int dtype,
                            int32_t* err_flag, void* stream) {
  return da::append_paged(k_pages, v_pages, k_scale, v_scale, true, k_new, v_new, q, q_out, rope_cos, rope_sin,
                          rope_rows, page_table, position_ids, token_start, B, tokens, n_head, n_kv_head, head_dim,
                          num_pages, page_size, max_pages, dtype, err_flag, stream);
}

int kvcache_append_paged_axes(void* k_pages, void* v_pages, const void* k_new, const void* v_new, const void* q,
                              void* q_out, const float* rope_cos, const float* rope_sin, int rope_rows,
                              const int32_t* rope_position_ids, const int32_t* rope_axis, int axes,
                              const int32_t* page_table, const int32_t* position_ids, const int32_t* token_start,
                              int B, int tokens, int n_head, int n_kv_head, int head_dim, int num_pages,
                              int page_size, int max_pages, int dtype, int32_t* err_flag, void* stream) {
  const da::Turns turns = {rope_position_ids, rope_axis, axes};
  return da::append_paged(k_pages, v_pages, nullptr, nullptr, false, k_new, v_new, q, q_out, rope_cos, rope_sin,
                          rope_rows, page_table, position_ids, token_start, B, tokens, n_head, n_kv_head, head_dim,
                          num_pages, page_size, max_pages, dtype, err_flag, stream, &turns);
}

int kvcache_append_paged_q8_axes(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const void* k_new,
                                 const void* v_new, const void* q, void* q_out, const float* rope_cos,
                                 const float* rope_sin, int rope_rows, const int32_t* rope_position_ids,
                                 const int32_t* rope_axis, int axes, const int32_t* page_table,
                                 const int32_t* position_ids, const int32_t* token_start, int B, int tokens,
                                 int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages,
                                 int dtype, int32_t* err_flag, void* stream) {
  const da::Turns turns = {rope_position_ids, rope_axis, axes};
  return da::append_paged(k_pages, v_pages, k_scale, v_scale, true, k_new, v_new, q, q_out, rope_cos, rope_sin,
                          rope_rows, page_table, position_ids, token_start, B, tokens, n_head, n_kv_head, head_dim,
                          num_pages, page_size, max_pages, dtype, err_flag, stream, &turns);
}

size_t decode_attn_tree_workspace_size(int n_head, int n_kv_head, int head_dim) {
  if (da::check_heads(1, n_head, n_kv_head, head_dim, DA_F16) != DA_OK) return (size_t)-1;
  int sms = 0;
  if (da::current_device_sms(&sms) != cudaSuccess) return (size_t)-1;
  return da::tree_workspace_bytes(sms, n_head / n_kv_head, head_dim);
}

int decode_attn_tree_fwd(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                         const int32_t* kv_len, const int32_t* token_start, const int64_t* tree_mask, int mask_words,
                         int B, int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size,
                         int max_pages, float scale, void* out, void* workspace, size_t workspace_bytes, int dtype,
                         int32_t* err_flag, void* stream) {
  return da::tree_attention(q, k_pages, v_pages, nullptr, nullptr, false, page_table, kv_len, token_start, tree_mask,
                            mask_words, B, tokens, n_head, n_kv_head, head_dim, num_pages, page_size, max_pages, scale,
                            out, workspace, workspace_bytes, dtype, err_flag, stream);
}

int decode_attn_tree_q8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                            const float* v_scale, const int32_t* page_table, const int32_t* kv_len,
                            const int32_t* token_start, const int64_t* tree_mask, int mask_words, int B, int tokens,
                            int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages,
                            float scale, void* out, void* workspace, size_t workspace_bytes, int dtype,
                            int32_t* err_flag, void* stream) {
  return da::tree_attention(q, k_pages, v_pages, k_scale, v_scale, true, page_table, kv_len, token_start, tree_mask,
                            mask_words, B, tokens, n_head, n_kv_head, head_dim, num_pages, page_size, max_pages, scale,
                            out, workspace, workspace_bytes, dtype, err_flag, stream);
}

}  // extern "C"
