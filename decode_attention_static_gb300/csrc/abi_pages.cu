// C ABI of the page operators: argument validation and the launches on the
// caller's stream. Nothing here allocates or synchronises.
#include <stdint.h>

#include "cache_params.h"
#include "decode_attn.h"
#include "page_params.h"

namespace da {

namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? DA_OK : DA_ERR_CUDA; }

int check_page_size(int page_size) {
  if (page_size < 1) return DA_ERR_SHAPE;
  if (page_size < kMinPageSize || page_size > kMaxPageSize || (page_size & (page_size - 1)) != 0)
    return DA_ERR_UNSUPPORTED;
  return DA_OK;
}

int check_table(int B, int num_pages, int page_size, int max_pages) {
  if (B < 0 || B > kMaxBatch || num_pages < 1 || max_pages < 1) return DA_ERR_SHAPE;
  const int rc = check_page_size(page_size);
  if (rc != DA_OK) return rc;
  if ((int64_t)max_pages * page_size > INT32_MAX - 2 * kMaxPageSize) return DA_ERR_SHAPE;
  return DA_OK;
}

int check_pools(const void* k_pages, const void* v_pages, const float* k_scale, const float* v_scale, int layers,
                int num_pages, int n_kv_head, int head_dim) {
  if (layers < 0 || num_pages < 1 || n_kv_head < 1 || n_kv_head > kMaxBatch || head_dim < 1) return DA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return DA_ERR_UNSUPPORTED;
  if (!k_pages || !v_pages || (k_scale != nullptr) != (v_scale != nullptr)) return DA_ERR_NULL;
  if (k_pages == v_pages || (k_scale && k_scale == v_scale)) return DA_ERR_SHAPE;  // K and V need arrays of their own
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return DA_ERR_ALIGN;
  return DA_OK;
}

int compact(void* k_pages, void* v_pages, float* k_scale, float* v_scale, bool e4m3, const int32_t* page_table,
            const int32_t* keep, const int32_t* keep_start, const int32_t* position_ids, int B, int kept, int layers,
            int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int32_t* err_flag,
            void* stream) {
  int rc = check_table(B, num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (kept < 0 || layers < 0 || n_kv_head < 1 || head_dim < 1) return DA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return DA_ERR_UNSUPPORTED;
  if (B == 0 || kept == 0 || layers == 0) return DA_OK;
  if (e4m3 && (!k_scale || !v_scale)) return DA_ERR_NULL;
  rc = check_pools(k_pages, v_pages, k_scale, v_scale, layers, num_pages, n_kv_head, head_dim);
  if (rc != DA_OK) return rc;
  const void* words[] = {page_table, keep, keep_start, position_ids};
  for (const void* w : words) {
    if (!w) return DA_ERR_NULL;
    if (!aligned(w, 4)) return DA_ERR_ALIGN;
  }
  if (!aligned(err_flag, 4)) return DA_ERR_ALIGN;
  MoveParams p = {};
  p.k = static_cast<uint8_t*>(k_pages);
  p.v = static_cast<uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.keep = keep;
  p.start = keep_start;
  p.pos = position_ids;
  p.B = B;
  p.kept = kept;
  p.layers = layers;
  p.n_kv_head = n_kv_head;
  p.num_pages = num_pages;
  p.page_rows = page_size;
  p.page_shift = log2_of(page_size);
  p.max_pages = max_pages;
  p.row_vecs = head_dim * (e4m3 ? 1 : 2) / 16;
  p.err_flag = err_flag;
  // one thread for each column, at most 2^31 - 1 CTAs
  if ((int64_t)B * n_kv_head * 2 * p.row_vecs > (INT64_MAX >> 16) / layers ||
      ((int64_t)B * n_kv_head * 2 * p.row_vecs * layers + 255) / 256 > INT32_MAX)
    return DA_ERR_SHAPE;
  return status_of(launch_compact(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

}  // namespace da

extern "C" {

int kvcache_pool_init(int32_t* pool, int num_pages, void* stream) {
  if (num_pages < 1 || num_pages > da::kPoolMaxPages) return DA_ERR_SHAPE;
  if (!pool) return DA_ERR_NULL;
  if (!da::aligned(pool, 4)) return DA_ERR_ALIGN;
  return da::status_of(da::launch_pool_init(pool, num_pages, static_cast<cudaStream_t>(stream)));
}

int kvcache_resize_paged(int32_t* page_table, const int32_t* held_len, const int32_t* wanted_len, int32_t* pool, int B,
                         int num_pages, int page_size, int max_pages, int32_t* err_flag, void* stream) {
  const int rc = da::check_table(B, num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (num_pages > da::kPoolMaxPages || (int64_t)B * max_pages > INT32_MAX) return DA_ERR_SHAPE;
  if (B == 0) return DA_OK;
  const void* words[] = {page_table, held_len, wanted_len, pool};
  for (const void* w : words) {
    if (!w) return DA_ERR_NULL;
    if (!da::aligned(w, 4)) return DA_ERR_ALIGN;
  }
  if (!da::aligned(err_flag, 4)) return DA_ERR_ALIGN;
  da::PoolParams p = {};
  p.table = page_table;
  p.pool = pool;
  p.a = held_len;
  p.b = wanted_len;
  p.B = p.n = B;
  p.num_pages = num_pages;
  p.page_shift = da::log2_of(page_size);
  p.max_pages = max_pages;
  p.err_flag = err_flag;
  return da::status_of(da::launch_pool_resize(p, static_cast<cudaStream_t>(stream)));
}

int kvcache_fork_paged(int32_t* page_table, int32_t* kv_len, const int32_t* parent, const int32_t* child,
                       int32_t* pool, int32_t* copies, int forks, int B, int num_pages, int page_size, int max_pages,
                       int32_t* err_flag, void* stream) {
  const int rc = da::check_table(B, num_pages, page_size, max_pages);
  if (rc != DA_OK) return rc;
  if (forks < 0 || forks > da::kMaxBatch || num_pages > da::kPoolMaxPages || (int64_t)B * max_pages > INT32_MAX)
    return DA_ERR_SHAPE;
  if (forks == 0) return DA_OK;
  if (B == 0) return DA_ERR_SHAPE;
  const void* words[] = {page_table, kv_len, parent, child, pool, copies};
  for (const void* w : words) {
    if (!w) return DA_ERR_NULL;
    if (!da::aligned(w, 4)) return DA_ERR_ALIGN;
  }
  if (!da::aligned(err_flag, 4)) return DA_ERR_ALIGN;
  da::PoolParams p = {};
  p.table = page_table;
  p.pool = pool;
  p.a = parent;
  p.b = child;
  p.kv_len = kv_len;
  p.copies = copies;
  p.B = B;
  p.n = forks;
  p.num_pages = num_pages;
  p.page_shift = da::log2_of(page_size);
  p.max_pages = max_pages;
  p.err_flag = err_flag;
  return da::status_of(da::launch_pool_fork(p, static_cast<cudaStream_t>(stream)));
}

int kvcache_copy_pages(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int32_t* copies, int n,
                       int layers, int num_pages, int n_kv_head, int page_size, int head_dim, int element_size,
                       int32_t* err_flag, void* stream) {
  if (n < 0 || layers < 0) return DA_ERR_SHAPE;
  int rc = da::check_page_size(page_size);
  if (rc != DA_OK) return rc;
  if (element_size != 1 && element_size != 2) return DA_ERR_DTYPE;
  if (n == 0 || layers == 0) return DA_OK;
  rc = da::check_pools(k_pages, v_pages, k_scale, v_scale, layers, num_pages, n_kv_head, head_dim);
  if (rc != DA_OK) return rc;
  if (!copies) return DA_ERR_NULL;
  if (!da::aligned(copies, 4) || !da::aligned(err_flag, 4)) return DA_ERR_ALIGN;
  if ((int64_t)n * layers > INT32_MAX / (2 * n_kv_head)) return DA_ERR_SHAPE;  // one CTA for each run of rows
  da::MoveParams p = {};
  p.k = static_cast<uint8_t*>(k_pages);
  p.v = static_cast<uint8_t*>(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.copies = copies;
  p.n = n;
  p.layers = layers;
  p.n_kv_head = n_kv_head;
  p.num_pages = num_pages;
  p.page_rows = page_size;
  p.row_vecs = head_dim * element_size / 16;
  p.err_flag = err_flag;
  return da::status_of(da::launch_copy_pages(p, static_cast<cudaStream_t>(stream)));
}

int kvcache_compact_paged(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* keep,
                          const int32_t* keep_start, const int32_t* position_ids, int B, int kept, int layers,
                          int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int32_t* err_flag,
                          void* stream) {
  return da::compact(k_pages, v_pages, nullptr, nullptr, false, page_table, keep, keep_start, position_ids, B, kept,
                     layers, n_kv_head, head_dim, num_pages, page_size, max_pages, err_flag, stream);
}

int kvcache_compact_paged_q8(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int32_t* page_table,
                             const int32_t* keep, const int32_t* keep_start, const int32_t* position_ids, int B,
                             int kept, int layers, int n_kv_head, int head_dim, int num_pages, int page_size,
                             int max_pages, int32_t* err_flag, void* stream) {
  return da::compact(k_pages, v_pages, k_scale, v_scale, true, page_table, keep, keep_start, position_ids, B, kept,
                     layers, n_kv_head, head_dim, num_pages, page_size, max_pages, err_flag, stream);
}

}  // extern "C"
