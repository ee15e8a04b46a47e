// Host-side interface of the page operators: the state of a pool (counts and
// free pages), and the rows and pages that move inside the pools.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace da {

// A table of sequences' pages and the pool's state: pool[0] free pages, from
// pool[kPoolHeader] on the pages' counts, then the list of free pages.
constexpr int kPoolHeader = 4;
constexpr int kPoolMaxPages = 1 << 22;

struct PoolParams {
  int32_t* table;          // [B, max_pages]
  int32_t* pool;
  const int32_t* a;        // resize: held lengths [B]; fork: parents [n]
  const int32_t* b;        // resize: wanted lengths [B]; fork: children [n]
  int32_t* kv_len;         // fork: [B]
  int32_t* copies;         // fork: [3, n]
  int B, n;                // sequences; entries of a and b
  int num_pages, page_shift, max_pages;
  int32_t* err_flag;       // may be null
};

// Rows or pages that move inside the K and V pools of several layers.
struct MoveParams {
  uint8_t* k;              // [layers, num_pages, n_kv_head, page_rows, D]
  uint8_t* v;
  float* k_scale;          // e4m3: [layers, num_pages, n_kv_head] (else null)
  float* v_scale;
  const int32_t* copies;   // copy: [3, n]
  const int32_t* table;    // compact: [B, max_pages]
  const int32_t* keep;     // compact: [kept], packed
  const int32_t* start;    // compact: [B + 1]
  const int32_t* pos;      // compact: [B]
  int n, B, kept;
  int layers, n_kv_head, num_pages, page_rows, page_shift, max_pages;
  int row_vecs;            // 16-byte vectors of a row
  int32_t* err_flag;       // may be null
};

cudaError_t launch_pool_init(int32_t* pool, int num_pages, cudaStream_t stream);
cudaError_t launch_pool_resize(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_pool_fork(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_copy_pages(const MoveParams& p, cudaStream_t stream);
cudaError_t launch_compact(const MoveParams& p, cudaStream_t stream);

}  // namespace da
