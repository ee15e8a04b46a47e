// Host-side interface of the paged-cache and sliding-window operators.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace da {

// Smallest scale of an 8-bit block is 2^kMinScaleExponent.
constexpr int kMinScaleExponent = -100;
constexpr int kMinPageSize = 16;
constexpr int kMaxPageSize = 256;
// Most sequences, and most KV heads, of an attention call (cache_attn.cuh packs
// a sequence number and a head into 16 bits each).
constexpr int kMaxBatch = 65535;
// Most rotary axes of an append.
constexpr int kMaxRopeAxes = 4;

// Attention over a cache in pages, or (table == nullptr) over a static cache,
// where sequence b is page b of `page_rows` = capacity rows.
struct CacheAttnParams {
  const uint8_t* q;        // [B, n_head, D]
  const uint8_t* k;        // [pages, n_kv_head, page_rows, D]
  const uint8_t* v;
  const float* k_scale;    // 8-bit pages: [pages, n_kv_head] (else null)
  const float* v_scale;
  const int32_t* table;    // [B, max_pages] (null: static cache)
  const int32_t* kv_len;   // [B]
  int B, n_head, n_kv_head, group;
  int num_pages, page_rows, page_shift, max_pages;
  int max_len;             // largest valid kv_len
  int window, sinks;       // window <= 0: every row is visible
  float qscale;            // softmax scale * log2(e)
  uint8_t* out;            // [B, n_head, D]
  unsigned int* counters;
  float* partials;
  int32_t* err_flag;       // may be null
};

// Append of new rows to a paged cache.
struct AppendPagedParams {
  uint8_t* k_pages;        // [num_pages, n_kv_head, page_rows, D]
  uint8_t* v_pages;
  float* k_scale;          // 8-bit pages: [num_pages, n_kv_head] (else null)
  float* v_scale;
  const uint8_t* k_new;    // [tokens, n_kv_head, D]
  const uint8_t* v_new;
  const uint8_t* q;        // [tokens, n_head, D] (null: no query to rotate)
  uint8_t* q_out;
  const float* cos;        // [rope_rows, D] (null: no rotation)
  const float* sin;
  const int32_t* table;    // [B, max_pages]
  const int32_t* pos;      // [B]
  const int32_t* start;    // [B + 1] (null: one token per sequence)
  int B, tokens, n_head, n_kv_head, head_dim;
  int num_pages, page_rows, page_shift, max_pages;
  int limit;               // positions must lie in [0, limit)
  const int32_t* turn;     // rows of the tables: [axes, tokens] (null: a token's row is its position)
  const int32_t* axis;     // [D / 2]: axis of each element pair (null: the first)
  int axes, rope_rows;
  int32_t* err_flag;       // may be null
};

// CTAs of an attention launch: one for each SM, at most 256 (cache_attn.cuh).
inline int cache_attn_ctas(int sms) { return sms < 256 ? sms : 256; }
// Floats of a partial state: acc [group][D], m [group], l [group], in whole
// 16-byte vectors.
__host__ __device__ inline int cache_attn_slot_floats(int group, int head_dim) {
  return group * head_dim + (2 * group + 3) / 4 * 4;
}
// Scratch of the attention: a fixed region of arrival counters (the one of
// the other decode kernels), then two partial states for each CTA.
size_t cache_attn_workspace_bytes(int sms, int group, int head_dim);
cudaError_t launch_cache_attn(const CacheAttnParams& p, int dtype, int head_dim, bool e4m3, int sms,
                              cudaStream_t stream);
cudaError_t launch_cache_attn_f16(const CacheAttnParams& p, int head_dim, bool e4m3, int sms, cudaStream_t stream);
cudaError_t launch_cache_attn_bf16(const CacheAttnParams& p, int head_dim, bool e4m3, int sms, cudaStream_t stream);
cudaError_t launch_append_paged(const AppendPagedParams& p, int dtype, int sms, cudaStream_t stream);

// abi.cu: this host thread's profiling events around a kernel, and the SM
// count of the current device.
bool record_timing_before(cudaStream_t stream);
bool record_timing_after(cudaStream_t stream);
cudaError_t current_device_sms(int* sms);
// abi.cu: the ring slot that this host thread's failure tests leave unfilled (< 0: none).
int skipped_slot();

}  // namespace da
