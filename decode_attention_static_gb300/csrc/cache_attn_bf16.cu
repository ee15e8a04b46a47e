// Paged and sliding-window attention instances for bf16 queries.
#include "cache_attn.cuh"

namespace da {

cudaError_t launch_cache_attn_bf16(const CacheAttnParams& p, int head_dim, bool e4m3, int sms, cudaStream_t stream) {
  return launch_cache_attn_type<__nv_bfloat16>(p, head_dim, e4m3, sms, stream);
}

}  // namespace da
