// Host-side interface of the attention of several new tokens over a paged cache.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace da {

constexpr int kTreeMaxTokens = 256;
constexpr int kTreeMaxWords = kTreeMaxTokens / 64;

struct TreeParams {
  const uint8_t* q;        // [tokens, n_head, D]
  const uint8_t* k;        // [pages, n_kv_head, page_rows, D]
  const uint8_t* v;
  const float* k_scale;    // 8-bit pages: [pages, n_kv_head] (else null)
  const float* v_scale;
  const int32_t* table;    // [B, max_pages]
  const int32_t* kv_len;   // [B]
  const int32_t* start;    // [B + 1] (null: one token per sequence)
  const uint64_t* mask;    // [tokens, mask_words] (null: a chain)
  int mask_words;
  int B, tokens, n_head, n_kv_head, group;
  int num_pages, page_rows, page_shift, max_pages;
  float qscale;            // softmax scale * log2(e)
  uint8_t* out;            // [tokens, n_head, D]
  void* workspace;
  int32_t* err_flag;       // may be null
  int skip_slot;           // test hook: copy of the first CTA that is left out (< 0: none)
};

size_t tree_workspace_bytes(int sms, int group, int head_dim);
cudaError_t launch_tree(const TreeParams& p, int dtype, int head_dim, bool e4m3, int sms, cudaStream_t stream);

}  // namespace da
