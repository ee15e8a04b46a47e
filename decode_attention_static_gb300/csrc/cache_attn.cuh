// Decode attention over a paged cache (16-bit or e4m3 pages) or a static
// cache, with an optional sliding window and sinks.
#pragma once

#include "cache_params.h"
#include "common.cuh"

namespace da {

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// One CTA per (KV head, sequence): each warp takes every eighth visible row.
template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(256) cache_attn_kernel(const CacheAttnParams p) {
  constexpr int kWarps = 8, kMaxGroup = 8, kPer = D / 32;
  __shared__ float sm_m[kWarps][kMaxGroup], sm_l[kWarps][kMaxGroup], sm_acc[kWarps][kMaxGroup][D];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int L = p.kv_len[b], G = p.group;
  const bool bad_len = L < 0 || L > p.max_len;
  if (bad_len && threadIdx.x == 0 && g == 0 && p.err_flag) atomicOr(p.err_flag, kErrKvLen);
  const int w0 = (!bad_len && p.window > 0 && L > p.window) ? L - p.window : 0;
  const int s0 = min(p.sinks, w0);
  const int rows = bad_len ? 0 : s0 + (L - w0);
  const T* q = reinterpret_cast<const T*>(p.q) + ((int64_t)b * p.n_head + g * G) * D + lane * kPer;
  float qf[kMaxGroup][kPer], acc[kMaxGroup][kPer], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      qf[h][e] = h < G ? (float)q[h * D + e] : 0.f;
      acc[h][e] = 0.f;
    }
  }
  bool bad_page = false;
  for (int i = warp; i < rows; i += kWarps) {
    const int r = i < s0 ? i : i - s0 + w0;
    int page = b, in = r;
    if (p.table) {
      page = p.table[(int64_t)b * p.max_pages + (r >> p.page_shift)];
      in = r & (p.page_rows - 1);
      if (page < 0 || page >= p.num_pages) {
        bad_page = true;
        break;
      }
    }
    const int64_t at = (((int64_t)page * p.n_kv_head + g) * p.page_rows + in) * D + lane * kPer;
    float kf[kPer], vf[kPer];
    if constexpr (E4M3) {
      const float ks = p.k_scale[(int64_t)page * p.n_kv_head + g], vs = p.v_scale[(int64_t)page * p.n_kv_head + g];
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const float2 a = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.k + at + e));
        const float2 c = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p.v + at + e));
        kf[e] = a.x * ks;
        kf[e + 1] = a.y * ks;
        vf[e] = c.x * vs;
        vf[e + 1] = c.y * vs;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        kf[e] = (float)reinterpret_cast<const T*>(p.k)[at + e];
        vf[e] = (float)reinterpret_cast<const T*>(p.v)[at + e];
      }
    }
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
      if (h >= G) break;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x = fmaf(qf[h][e], kf[e], x);
#pragma unroll
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= p.qscale;
      const float mn = fmaxf(m[h], x), c = exp2f(m[h] - mn), w = exp2f(x - mn);
      m[h] = mn;
      l[h] = l[h] * c + w;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[h][e] = acc[h][e] * c + w * vf[e];
    }
  }
  if (bad_page && p.err_flag) atomicOr(p.err_flag, kErrPage);
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) {
    sm_m[warp][h] = m[h];
    sm_l[warp][h] = bad_page ? NAN : l[h];
#pragma unroll
    for (int e = 0; e < kPer; ++e) sm_acc[warp][h][lane * kPer + e] = acc[h][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += blockDim.x) {
    const int h = i / D, d = i % D;
    float mm = -INFINITY, ll = 0.f, a = 0.f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][h]);
    for (int w = 0; w < kWarps; ++w) {
      const float c = sm_m[w][h] == -INFINITY ? 0.f : exp2f(sm_m[w][h] - mm);
      ll += c * sm_l[w][h];
      a += c * sm_acc[w][h][d];
    }
    for (int w = 0; w < kWarps; ++w)
      if (isnan(sm_l[w][h])) ll = NAN;
    float r = rows > 0 ? a / ll : 0.f;
    if (bad_len) r = NAN;
    reinterpret_cast<uint16_t*>(p.out)[((int64_t)b * p.n_head + g * G) * D + i] = Storage<T>::round(r);
  }
}

template <typename T, bool E4M3, int D>
cudaError_t launch_cache_attn_t(const CacheAttnParams& p, int sms, cudaStream_t stream) {
  (void)sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_kv_head, p.B);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_kernel<T, E4M3, D>, p);
}

template <typename T>
cudaError_t launch_cache_attn_type(const CacheAttnParams& p, int head_dim, bool e4m3, int sms, cudaStream_t stream) {
  if (head_dim == 128)
    return e4m3 ? launch_cache_attn_t<T, true, 128>(p, sms, stream) : launch_cache_attn_t<T, false, 128>(p, sms, stream);
  return e4m3 ? launch_cache_attn_t<T, true, 64>(p, sms, stream) : launch_cache_attn_t<T, false, 64>(p, sms, stream);
}

}  // namespace da
