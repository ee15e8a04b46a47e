// Append of new key and value rows to a paged cache, with the rotary
// embedding of the keys (and of the query) on the way; 16-bit pages, or e4m3
// pages with one power-of-two scale per page and KV head.
//
// Both kernels move each byte once and are bound by HBM for prompts and by
// launch latency for single tokens.
#include "cache_params.h"
#include "common.cuh"
#include "decode_attn.h"

namespace da {
namespace {


constexpr int kThreads = 256;

// New rows of sequence b: first packed token, count and first position.
// False for a sequence whose positions do not all lie in [0, limit) or whose
// token range is not inside the packed tokens.
__device__ __forceinline__ bool sequence_rows(const AppendPagedParams& p, int b, int* first, int* count, int* p0) {
  int a = b, n = 1;
  if (p.start) {
    a = p.start[b];
    const int e = p.start[b + 1];
    if (a < 0 || e < a || e > p.tokens) {
      *count = 0;
      return false;
    }
    n = e - a;
  }
  *first = a;
  *count = n;
  *p0 = p.pos[b];
  return n == 0 || (*p0 >= 0 && *p0 <= p.limit - n);
}

// Sequence that owns packed token t, or -1.
__device__ __forceinline__ int sequence_of(const AppendPagedParams& p, int t) {
  if (!p.start) return t;
  int lo = 0, hi = p.B;  // the last b with start[b] <= t lies in [lo, hi)
  if (t < p.start[0] || t >= p.start[p.B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One 16-byte vector x of the first half of a head and its partner y in the
// second half, rotated in fp32: each product and the sum rounded on their
// own, as in rope_vec8.
template <typename T>
__device__ __forceinline__ void rotate_pair(const uint4& x, const uint4& y, const AppendPagedParams& p, int position,
                                            int c, float (&a)[8], float (&b)[8]) {
  float xf[8], yf[8], c0[8], s0[8], c1[8], s1[8];
  Storage<T>::unpack(x, xf);
  Storage<T>::unpack(y, yf);
  const int D = p.head_dim;
  load_f32x8(p.cos, position, D, 8 * c, c0);
  load_f32x8(p.sin, position, D, 8 * c, s0);
  load_f32x8(p.cos, position, D, D / 2 + 8 * c, c1);
  load_f32x8(p.sin, position, D, D / 2 + 8 * c, s1);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = __fsub_rn(__fmul_rn(xf[e], c0[e]), __fmul_rn(yf[e], s0[e]));
    b[e] = __fadd_rn(__fmul_rn(yf[e], c1[e]), __fmul_rn(xf[e], s1[e]));
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint16_t r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = Storage<T>::round(f[e]);
  return make_uint4((uint32_t)r[0] | ((uint32_t)r[1] << 16), (uint32_t)r[2] | ((uint32_t)r[3] << 16),
                    (uint32_t)r[4] | ((uint32_t)r[5] << 16), (uint32_t)r[6] | ((uint32_t)r[7] << 16));
}

template <typename T>
__device__ __forceinline__ uint4 nan8() {
  const uint32_t n = (uint32_t)Storage<T>::kNaN * 0x10001u;
  return make_uint4(n, n, n, n);
}

// Rotates query head `h` of packed token t into q_out (the D / 16 lanes of a
// head each take vector c and its partner).
template <typename T>
__device__ __forceinline__ void rotate_query(const AppendPagedParams& p, int t, int h, int c, bool ok, int position) {
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2;
  const int64_t at = ((int64_t)t * p.n_head + h) * row_vecs + c;
  uint4* out = reinterpret_cast<uint4*>(p.q_out) + at;
  if (!ok) {
    out[0] = nan8<T>();
    out[half] = nan8<T>();
    return;
  }
  const uint4* in = reinterpret_cast<const uint4*>(p.q) + at;
  float a[8], b[8];
  rotate_pair<T>(in[0], in[half], p, position, c, a, b);
  out[0] = pack8<T>(a);
  out[half] = pack8<T>(b);
}

// 16-bit pages: one group of D / 16 lanes per (token, head), heads in the
// order K, V, q.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_paged_kernel(const AppendPagedParams p) {
  pdl_wait();
  pdl_trigger();
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2;
  const int heads = 2 * p.n_kv_head + (p.q ? p.n_head : 0);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int c = (int)(i % half);
  const int64_t item = i / half;
  const int t = (int)(item / heads);
  int h = (int)(item % heads);
  if (t >= p.tokens) return;
  const int b = sequence_of(p, t);
  if (b < 0) return;
  int first = 0, count = 0, p0 = 0;
  const bool ok = sequence_rows(p, b, &first, &count, &p0) && t >= first && t < first + count;
  if (!ok && h == 0 && c == 0 && p.err_flag) atomicOr(p.err_flag, kErrPosition);
  const int position = p0 + (t - first);
  if (h >= 2 * p.n_kv_head) {
    rotate_query<T>(p, t, h - 2 * p.n_kv_head, c, ok, position);
    return;
  }
  if (!ok) return;
  const int page = p.table[(int64_t)b * p.max_pages + (position >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    if (h == 0 && c == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
    return;
  }
  const bool is_k = h < p.n_kv_head;
  if (!is_k) h -= p.n_kv_head;
  const uint4* in =
      reinterpret_cast<const uint4*>(is_k ? p.k_new : p.v_new) + ((int64_t)t * p.n_kv_head + h) * row_vecs + c;
  const int64_t row = ((int64_t)page * p.n_kv_head + h) * p.page_rows + (position & (p.page_rows - 1));
  uint4* out = reinterpret_cast<uint4*>(is_k ? p.k_pages : p.v_pages) + row * row_vecs + c;
  uint4 x = in[0], y = in[half];
  if (is_k && p.cos) {
    float a[8], bb[8];
    rotate_pair<T>(x, y, p, position, c, a, bb);
    x = pack8<T>(a);
    y = pack8<T>(bb);
  }
  out[0] = x;
  out[half] = y;
}

// Exponent of the smallest power of two s with peak <= 448 s (448 = 1.75 *
// 2^8 is the largest e4m3 value), at least kMinScaleExponent.
__device__ __forceinline__ int scale_exponent(float peak) {
  const uint32_t u = __float_as_uint(peak);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExponent);
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// 8 values over a scale; non-finite ones become the type's NaN (e4m3 has no
// infinities).
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float inv) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fabsf(f[e]) < INFINITY ? f[e] * inv : NAN;
  return make_uint2(to_e4m3x2(x[0], x[1]) | (to_e4m3x2(x[2], x[3]) << 16),
                    to_e4m3x2(x[4], x[5]) | (to_e4m3x2(x[6], x[7]) << 16));
}

__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t v, float ratio) {
  const float2 a = from_e4m3x2(v & 0xffffu), b = from_e4m3x2(v >> 16);
  return to_e4m3x2(a.x * ratio, a.y * ratio) | (to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

__device__ __forceinline__ float finite_peak(float peak, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fabsf(f[e]);
    if (a < INFINITY) peak = fmaxf(peak, a);
  }
  return peak;
}

// e4m3 pages: one CTA per (touched page, KV head, K or V); the CTAs after
// those rotate the query rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) append_paged_q8_kernel(const AppendPagedParams p, int page_tasks) {
  __shared__ int sh[6];
  __shared__ float sh_peak[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2;
  const int units = kThreads / half, unit = threadIdx.x / half, c = threadIdx.x % half;
  const int64_t page_ctas = (int64_t)page_tasks * 2 * p.n_kv_head;
  if (blockIdx.x >= page_ctas) {
    const int64_t item = (blockIdx.x - page_ctas) * units + unit;
    const int t = (int)(item / p.n_head), h = (int)(item % p.n_head);
    if (t >= p.tokens) return;
    const int b = sequence_of(p, t);
    if (b < 0) return;
    int first = 0, count = 0, p0 = 0;
    const bool ok = sequence_rows(p, b, &first, &count, &p0) && t >= first && t < first + count;
    rotate_query<T>(p, t, h, c, ok, p0 + (t - first));
    return;
  }
  const int task = (int)(blockIdx.x / (2 * p.n_kv_head));
  const int g = (int)(blockIdx.x % (2 * p.n_kv_head)) >> 1;
  const bool is_k = (blockIdx.x & 1) == 0;
  if (threadIdx.x < 32) {
    // the task's sequence and page: tasks are the touched pages in sequence order
    int b_found = -1, j = 0, before = 0;
    for (int base = 0; base < p.B && b_found < 0; base += 32) {
      const int b = base + threadIdx.x;
      int pages = 0, first, count, p0;
      if (b < p.B && sequence_rows(p, b, &first, &count, &p0) && count > 0)
        pages = ((p0 + count - 1) >> p.page_shift) - (p0 >> p.page_shift) + 1;
      int sum = pages;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (threadIdx.x >= o) sum += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > task);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b_found = base + src;
        j = task - before - (__shfl_sync(0xffffffffu, sum, src) - __shfl_sync(0xffffffffu, pages, src));
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (threadIdx.x == 0) {
      sh[0] = b_found;
      sh[1] = j;
    }
  }
  if (task == 0 && g == 0 && is_k && p.err_flag) {
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      int first, count, p0;
      if (!sequence_rows(p, b, &first, &count, &p0)) atomicOr(p.err_flag, kErrPosition);
    }
  }
  __syncthreads();
  const int b = sh[0];
  if (b < 0) return;
  int first = 0, count = 0, p0 = 0;
  sequence_rows(p, b, &first, &count, &p0);
  const int j = (p0 >> p.page_shift) + sh[1];
  const int lo = max(p0, j << p.page_shift), hi = min(p0 + count, (j + 1) << p.page_shift);
  const int page = p.table[(int64_t)b * p.max_pages + j];
  if (page < 0 || page >= p.num_pages) {
    if (g == 0 && is_k && threadIdx.x == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
    return;
  }
  const uint4* in = reinterpret_cast<const uint4*>(is_k ? p.k_new : p.v_new);
  const bool rotate = is_k && p.cos;
  float a[8], bb[8], peak = 0.f;
  auto load = [&](int position) {
    const uint4* src = in + ((int64_t)(first + position - p0) * p.n_kv_head + g) * row_vecs + c;
    const uint4 x = src[0], y = src[half];
    if (rotate) {
      rotate_pair<T>(x, y, p, position, c, a, bb);
    } else {
      Storage<T>::unpack(x, a);
      Storage<T>::unpack(y, bb);
    }
  };
  for (int position = lo + unit; position < hi; position += units) {
    load(position);
    peak = finite_peak(finite_peak(peak, a), bb);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  if (threadIdx.x % 32 == 0) sh_peak[threadIdx.x / 32] = peak;
  const int old_rows = lo & (p.page_rows - 1);
  float* scale_at = (is_k ? p.k_scale : p.v_scale) + (int64_t)page * p.n_kv_head + g;
  const float old_scale = old_rows > 0 ? *scale_at : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) peak = fmaxf(peak, sh_peak[w]);
  const float scale = fmaxf(__uint_as_float((uint32_t)(scale_exponent(peak) + 127) << 23), old_scale);
  uint8_t* rows = (is_k ? p.k_pages : p.v_pages) + ((int64_t)page * p.n_kv_head + g) * p.page_rows * p.head_dim;
  if (old_rows > 0 && scale != old_scale) {
    const float ratio = old_scale / scale;
    for (int i = threadIdx.x; i < old_rows * p.head_dim / 16; i += kThreads) {
      uint4* at = reinterpret_cast<uint4*>(rows) + i;
      const uint4 v = *at;
      *at = make_uint4(rescale_e4m3x4(v.x, ratio), rescale_e4m3x4(v.y, ratio), rescale_e4m3x4(v.z, ratio),
                       rescale_e4m3x4(v.w, ratio));
    }
  }
  const float inv = 1.f / scale;
  for (int position = lo + unit; position < hi; position += units) {
    load(position);
    uint2* out = reinterpret_cast<uint2*>(rows + (int64_t)(position & (p.page_rows - 1)) * p.head_dim) + c;
    out[0] = quantise8(a, inv);
    out[half] = quantise8(bb, inv);
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

}  // namespace

cudaError_t launch_append_paged(const AppendPagedParams& p, int dtype, cudaStream_t stream) {
  const int half = p.head_dim / 16;
  int64_t ctas, page_tasks = 0;
  if (p.k_scale) {
    // every sequence touches at most one page more than its rows fill
    page_tasks = p.start ? (int64_t)p.tokens / p.page_rows + 2 * (int64_t)p.B : p.B;
    if (page_tasks > p.tokens) page_tasks = p.tokens;
    const int64_t query_items = p.q ? (int64_t)p.tokens * p.n_head : 0;
    ctas = page_tasks * 2 * p.n_kv_head + (query_items * half + kThreads - 1) / kThreads;
  } else {
    const int64_t items = (int64_t)p.tokens * (2 * p.n_kv_head + (p.q ? p.n_head : 0));
    ctas = (items * half + kThreads - 1) / kThreads;
  }
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.k_scale)
    return dtype == DA_F16 ? cudaLaunchKernelEx(&cfg, append_paged_q8_kernel<__half>, p, (int)page_tasks)
                           : cudaLaunchKernelEx(&cfg, append_paged_q8_kernel<__nv_bfloat16>, p, (int)page_tasks);
  return dtype == DA_F16 ? cudaLaunchKernelEx(&cfg, append_paged_kernel<__half>, p)
                         : cudaLaunchKernelEx(&cfg, append_paged_kernel<__nv_bfloat16>, p);
}

}  // namespace da
