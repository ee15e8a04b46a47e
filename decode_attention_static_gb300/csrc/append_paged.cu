// Append of new key and value rows to a paged cache, with the rotary
// embedding of the keys (and of the query) on the way; 16-bit pages, or e4m3
// pages with one power-of-two scale per page and KV head.
//
// A head of a row is D / 16 lanes ("a unit"), each with a 16-byte vector c of the
// first half and its partner c + D / 16 of the second: a rotation needs no
// other lane. Every byte of q, k_new, v_new and the pages moves once (but for
// the table rows, which come from L1 and L2 after the first head): prompts are
// bound by HBM, single tokens by the chain of dependent loads (sequence,
// position, page). Measured (of the measured 6782 GB/s copy): prompts of 8.8k
// tokens, 8 KV and 32 query heads of 128, fp16, 225 MB in 37.6 us (88%); the
// same heads, 20.8k tokens into 8 bits, 482 MB in 86.5 us (82%; the 30% that are K
// and V take 35 us, bound by the chain of peaks and rounding at two CTAs an SM);
// 8 sequences, one token each, 2.4 us, 64 into 8 bits 2.4 us.
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

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

__device__ __forceinline__ void load_f32x4(const float* from, float (&out)[4]) {
  const uint4 v = ld_global_nc_v4(from);
  out[0] = __uint_as_float(v.x);
  out[1] = __uint_as_float(v.y);
  out[2] = __uint_as_float(v.z);
  out[3] = __uint_as_float(v.w);
}

// Table rows of one token with positions on several axes (AX): element pairs
// (i, i + D / 2) of axis a turn by the table row at[a].
struct TurnRows {
  int at[kMaxRopeAxes];
  // The rows of token t; false when one is not in the tables.
  __device__ __forceinline__ bool load(const AppendPagedParams& p, int t) {
    bool ok = true;
#pragma unroll
    for (int a = 0; a < kMaxRopeAxes; ++a) {
      at[a] = a < p.axes ? p.turn[(int64_t)a * p.tokens + t] : at[0];
      ok = ok && at[a] >= 0 && at[a] < p.rope_rows;
    }
    return ok;
  }
  __device__ __forceinline__ int of(int axis) const {
    int r = at[0];
#pragma unroll
    for (int a = 1; a < kMaxRopeAxes; ++a) r = axis == a ? at[a] : r;
    return r;
  }
};

// Axes of four pairs from pair i on (a multiple of four): an axis outside [0,
// axes) counts as the first (the kernels' first units report it).
__device__ __forceinline__ int4 pair_axes(const AppendPagedParams& p, int i) {
  return p.axis ? __ldg(reinterpret_cast<const int4*>(p.axis + i)) : make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ bool one_axis(const int4& a) { return a.x == a.y && a.x == a.z && a.x == a.w; }

// Four elements at column `col` of a table, for pairs of axes `a`: one vector
// where the pairs share an axis (sections of whole vectors), else gathered (keys
// and values of 27k tokens into 8 bits, us: one axis 48, sections of whole
// vectors 52, sections that end inside vectors 71, interleaved 72; a vector of
// each axis that the pairs have, and its elements of it, spilled: 59, 73, 73, 80).
__device__ __forceinline__ void load_turn4(const float* table, int D, const TurnRows& rows, const int4& a, int col,
                                           float (&out)[4]) {
  if (one_axis(a)) {
    load_f32x4(table + (int64_t)rows.of(a.x) * D + col, out);
  } else {
    out[0] = __ldg(table + (int64_t)rows.of(a.x) * D + col);
    out[1] = __ldg(table + (int64_t)rows.of(a.y) * D + col + 1);
    out[2] = __ldg(table + (int64_t)rows.of(a.z) * D + col + 2);
    out[3] = __ldg(table + (int64_t)rows.of(a.w) * D + col + 3);
  }
}

// The first CTA's threads report axes outside [0, axes).
__device__ __forceinline__ void check_axes(const AppendPagedParams& p) {
  if (blockIdx.x == 0 && p.err_flag && p.axis && (int)threadIdx.x < p.head_dim / 2) {
    const int a = p.axis[threadIdx.x];
    if (a < 0 || a >= p.axes) atomicOr(p.err_flag, kErrPosition);
  }
}

// cos and sin of one row at a lane's two vectors.
struct RopeRow {
  float c0[8], s0[8], c1[8], s1[8];
  __device__ __forceinline__ void load_axes(const AppendPagedParams& p, const TurnRows& rows, int c) {
    const int D = p.head_dim;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const int4 a = pair_axes(p, 8 * c + e);
      load_turn4(p.cos, D, rows, a, 8 * c + e, *reinterpret_cast<float(*)[4]>(c0 + e));
      load_turn4(p.sin, D, rows, a, 8 * c + e, *reinterpret_cast<float(*)[4]>(s0 + e));
      load_turn4(p.cos, D, rows, a, D / 2 + 8 * c + e, *reinterpret_cast<float(*)[4]>(c1 + e));
      load_turn4(p.sin, D, rows, a, D / 2 + 8 * c + e, *reinterpret_cast<float(*)[4]>(s1 + e));
    }
  }
  __device__ __forceinline__ void load(const AppendPagedParams& p, int position, int c) {
    const int D = p.head_dim;
    load_f32x8(p.cos, position, D, 8 * c, c0);
    load_f32x8(p.sin, position, D, 8 * c, s0);
    load_f32x8(p.cos, position, D, D / 2 + 8 * c, c1);
    load_f32x8(p.sin, position, D, D / 2 + 8 * c, s1);
  }
  // The vectors x and y, rotated in fp32: each product and the sum rounded on
  // their own, as in rope_vec8.
  template <typename T>
  __device__ __forceinline__ void rotate(const uint4& x, const uint4& y, float (&a)[8], float (&b)[8]) const {
    float xf[8], yf[8];
    Storage<T>::unpack(x, xf);
    Storage<T>::unpack(y, yf);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = __fsub_rn(__fmul_rn(xf[e], c0[e]), __fmul_rn(yf[e], s0[e]));
      b[e] = __fadd_rn(__fmul_rn(yf[e], c1[e]), __fmul_rn(xf[e], s1[e]));
    }
  }
};

// The same for a row's unpacked vectors of N heads, in place; 4 elements at a
// time, so that few registers hold the table row.
template <bool AX, int N>
__device__ __forceinline__ void rotate_rows(const AppendPagedParams& p, int position, const TurnRows& rows, int c,
                                            float (&a)[N][8], float (&b)[N][8]) {
  const int64_t at = (int64_t)position * p.head_dim + 8 * c;
#pragma unroll
  for (int q = 0; q < 8; q += 4) {
    float c0[4], s0[4], c1[4], s1[4];
    if constexpr (AX) {
      const int D = p.head_dim;
      const int4 axes = pair_axes(p, 8 * c + q);
      load_turn4(p.cos, D, rows, axes, 8 * c + q, c0);
      load_turn4(p.sin, D, rows, axes, 8 * c + q, s0);
      load_turn4(p.cos, D, rows, axes, D / 2 + 8 * c + q, c1);
      load_turn4(p.sin, D, rows, axes, D / 2 + 8 * c + q, s1);
    } else {
      load_f32x4(p.cos + at + q, c0);
      load_f32x4(p.sin + at + q, s0);
      load_f32x4(p.cos + at + p.head_dim / 2 + q, c1);
      load_f32x4(p.sin + at + p.head_dim / 2 + q, s1);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = a[k][q + e], y = b[k][q + e];
        a[k][q + e] = __fsub_rn(__fmul_rn(x, c0[e]), __fmul_rn(y, s0[e]));
        b[k][q + e] = __fadd_rn(__fmul_rn(y, c1[e]), __fmul_rn(x, s1[e]));
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (Storage<T>::kBf16) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
      r[e] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      const __half2 v = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
      r[e] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// One unit of one token: heads h, h + stride, ... of the order K, V, q (from
// `first` on; K and V go to 16-bit pages). kAtOnce heads are loaded before the
// token's place is looked up, and the table row serves all of them.
constexpr int kAtOnce = 6;

template <typename T, bool AX>
__device__ __forceinline__ void move_token(const AppendPagedParams& p, int t, int first, int stride, int c) {
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2, Hkv = p.n_kv_head;
  const int heads = 2 * Hkv + (p.q ? p.n_head : 0);
  RopeRow rope;
  int b = 0, page = 0, position = 0;
  bool ok = false, page_ok = false;
  // AX: the table rows do not depend on the token's place, and are asked for first
  TurnRows rows;
  bool turns_ok = true;
  if constexpr (AX) turns_ok = rows.load(p, t);
  for (int h0 = first, turn = 0; h0 < heads; h0 += kAtOnce * stride, ++turn) {
    // (q may be rotated in place: plain loads, not the read-only path)
    uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int h = h0 + j * stride;
      if (h < heads) {
        const uint8_t* base = h < Hkv ? p.k_new : h < 2 * Hkv ? p.v_new : p.q;
        const int64_t row = h < 2 * Hkv ? (int64_t)t * Hkv + (h < Hkv ? h : h - Hkv)
                                        : (int64_t)t * p.n_head + h - 2 * Hkv;
        const uint4* in = reinterpret_cast<const uint4*>(base) + row * row_vecs;
        x[j] = in[c];
        y[j] = in[c + half];
      }
    }
    if (turn == 0) {
      if constexpr (AX) {
        if (turns_ok) rope.load_axes(p, rows, c);
      }
      b = sequence_of(p, t);
      if (b < 0) return;
      int from = 0, count = 0, p0 = 0;
      ok = sequence_rows(p, b, &from, &count, &p0) && t >= from && t < from + count;
      position = p0 + (t - from);
      ok = ok && turns_ok;
      if (!ok && first == 0 && c == 0 && p.err_flag) atomicOr(p.err_flag, kErrPosition);
      if (ok) {
        if constexpr (!AX) {
          if (p.cos) rope.load(p, position, c);
        }
        page = p.table[(int64_t)b * p.max_pages + (position >> p.page_shift)];
        page_ok = page >= 0 && page < p.num_pages;
        if (!page_ok && first == 0 && c == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int h = h0 + j * stride;
      if (h >= heads) break;
      const bool is_v = h >= Hkv && h < 2 * Hkv;
      if (ok && p.cos && !is_v) {
        float a[8], bb[8];
        rope.rotate<T>(x[j], y[j], a, bb);
        x[j] = pack8<T>(a);
        y[j] = pack8<T>(bb);
      }
      uint4* out;
      if (h >= 2 * Hkv) {
        out = reinterpret_cast<uint4*>(p.q_out) + ((int64_t)t * p.n_head + h - 2 * Hkv) * row_vecs;
        if (!ok) {
          const uint32_t n = (uint32_t)Storage<T>::kNaN * 0x10001u;
          x[j] = y[j] = make_uint4(n, n, n, n);
        }
      } else {
        if (!ok || !page_ok) continue;
        const int64_t row = ((int64_t)page * Hkv + (is_v ? h - Hkv : h)) * p.page_rows + (position & (p.page_rows - 1));
        out = reinterpret_cast<uint4*>(is_v ? p.v_pages : p.k_pages) + row * row_vecs;
      }
      out[c] = x[j];
      out[c + half] = y[j];
    }
  }
}

// 16-bit pages: `stride` units for each token.
template <typename T, bool AX>
__global__ void __launch_bounds__(kThreads, 2) append_paged_kernel(const AppendPagedParams p, int stride) {
  pdl_wait();
  pdl_trigger();
  if constexpr (AX) check_axes(p);
  const int half = p.head_dim / 16;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / half;
  const int64_t t = unit / stride;
  if (t < p.tokens) move_token<T, AX>(p, (int)t, (int)(unit - t * stride), stride, threadIdx.x % half);
}

// Exponent of the smallest power of two s with peak <= 448 s (448 = 1.75 *
// 2^8 is the largest e4m3 value), at least kMinScaleExponent.
__device__ __forceinline__ int scale_exponent(float peak) {
  const uint32_t u = __float_as_uint(peak);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kMinScaleExponent);
}

__device__ __forceinline__ float scale_of(float peak) {
  return __uint_as_float((uint32_t)(scale_exponent(peak) + 127) << 23);
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

// Whether a scale's reciprocal is exact and normal: scales that this call makes
// are powers of two up to 2^120, but a page may come with any other from elsewhere.
__device__ __forceinline__ bool power_of_two(float scale) {
  const uint32_t u = __float_as_uint(scale);
  return (u & 0x7fffffu) == 0 && u < 254u << 23;
}

// 8 values over a scale. NaN becomes the type's NaN by the conversion. CAREFUL:
// infinities, which would be clamped to 448, become NaN too (e4m3 has none), and
// the values are divided; else they are multiplied by the reciprocal of a power
// of two.
template <bool CAREFUL>
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float scale) {
  float x[8];
  const float inv = __uint_as_float((2u * 127 << 23) - __float_as_uint(scale));
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    if constexpr (CAREFUL) {
      x[e] = fabsf(f[e]) == INFINITY ? NAN : f[e] / scale;
      x[e + 1] = fabsf(f[e + 1]) == INFINITY ? NAN : f[e + 1] / scale;
    } else {
      const float2 v = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(inv, inv));
      x[e] = v.x;
      x[e + 1] = v.y;
    }
  }
  return make_uint2(to_e4m3x2(x[0], x[1]) | (to_e4m3x2(x[2], x[3]) << 16),
                    to_e4m3x2(x[4], x[5]) | (to_e4m3x2(x[6], x[7]) << 16));
}

__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t v, float ratio) {
  const float2 a = from_e4m3x2(v & 0xffffu), b = from_e4m3x2(v >> 16);
  return to_e4m3x2(a.x * ratio, a.y * ratio) | (to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

// Rows [0, count) of a page and head to a larger scale, by `threads` threads.
__device__ __forceinline__ void rescale_rows(uint8_t* rows, int bytes, float ratio, int thread, int threads) {
  for (int i = thread; i < bytes / 16; i += threads) {
    uint4* at = reinterpret_cast<uint4*>(rows) + i;
    const uint4 v = *at;
    *at = make_uint4(rescale_e4m3x4(v.x, ratio), rescale_e4m3x4(v.y, ratio), rescale_e4m3x4(v.z, ratio),
                     rescale_e4m3x4(v.w, ratio));
  }
}

// Largest |f| so far; NaN does not count, infinity does.
__device__ __forceinline__ float peak_of(float peak, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(peak) : "f"(f[e]), "f"(f[e + 1]));
  return peak;
}

// The same of the finite values alone: for heads whose peak is infinity.
__device__ __forceinline__ float finite_peak(float peak, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fabsf(f[e]);
    if (a < INFINITY) peak = fmaxf(peak, a);
  }
  return peak;
}

// e4m3 pages, one token for each sequence: one unit for each (sequence, K or V
// head), and `stride` units for the query heads of each token. A unit finds
// its row's peak with shuffles; where a scale grows, its whole warp rounds the
// page's older rows.
template <typename T, bool AX>
__global__ void __launch_bounds__(kThreads)
    append_token_q8_kernel(const AppendPagedParams p, int row_ctas, int stride) {
  pdl_wait();
  pdl_trigger();
  if constexpr (AX) check_axes(p);
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2, Hkv = p.n_kv_head, c = threadIdx.x % half;
  if ((int)blockIdx.x >= row_ctas) {
    const int64_t unit = ((int64_t)(blockIdx.x - row_ctas) * kThreads + threadIdx.x) / half;
    const int64_t t = unit / stride;
    if (t < p.tokens) move_token<T, AX>(p, (int)t, 2 * Hkv + (int)(unit - t * stride), stride, c);
    return;
  }
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / half;
  const int b = (int)min(unit / (2 * Hkv), (int64_t)p.B - 1), hk = (int)(unit % (2 * Hkv));
  const bool live = unit < (int64_t)p.B * 2 * Hkv, is_k = hk < Hkv;
  const int g = is_k ? hk : hk - Hkv;
  const uint4* in = reinterpret_cast<const uint4*>(is_k ? p.k_new : p.v_new) + ((int64_t)b * Hkv + g) * row_vecs + c;
  const uint4 x = in[0], y = in[half];
  const int position = p.pos[b];
  TurnRows turn;
  bool ok = position >= 0 && position < p.limit;
  if constexpr (AX) ok = turn.load(p, b) && ok;
  int page = ok ? p.table[(int64_t)b * p.max_pages + (position >> p.page_shift)] : 0;
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (live && hk == 0 && c == 0 && p.err_flag && !(ok && page_ok)) atomicOr(p.err_flag, ok ? kErrPage : kErrPosition);
  const bool write = live && ok && page_ok;
  if (!write) page = 0;
  float a[8], bb[8];
  if (write && is_k && p.cos) {
    RopeRow rope;
    if constexpr (AX) rope.load_axes(p, turn, c); else rope.load(p, position, c);
    rope.rotate<T>(x, y, a, bb);
  } else {
    Storage<T>::unpack(x, a);
    Storage<T>::unpack(y, bb);
  }
  float peak = peak_of(peak_of(0.f, a), bb);
  for (int o = half / 2; o; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  const bool infinities = peak == INFINITY;
  if (__any_sync(0xffffffffu, infinities)) {
    peak = finite_peak(finite_peak(0.f, a), bb);
    for (int o = half / 2; o; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  }
  const int old_rows = position & (p.page_rows - 1);
  const int64_t block = (int64_t)page * Hkv + g;
  float* scale_at = (is_k ? p.k_scale : p.v_scale) + block;
  const float old_scale = write && old_rows > 0 ? *scale_at : 0.f;
  const float scale = fmaxf(scale_of(peak), old_scale);
  uint8_t* rows = (is_k ? p.k_pages : p.v_pages) + block * p.page_rows * p.head_dim;
  unsigned todo = __ballot_sync(0xffffffffu, write && old_rows > 0 && scale != old_scale && c == 0);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    uint8_t* at = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rows), src));
    const int n = __shfl_sync(0xffffffffu, old_rows, src);
    const float ratio = __shfl_sync(0xffffffffu, old_scale / scale, src);
    rescale_rows(at, n * p.head_dim, ratio, threadIdx.x % 32, 32);
  }
  if (write) {
    uint2* out = reinterpret_cast<uint2*>(rows + (int64_t)old_rows * p.head_dim) + c;
    if (infinities || !power_of_two(scale)) {
      out[0] = quantise8<true>(a, scale);
      out[half] = quantise8<true>(bb, scale);
    } else {
      out[0] = quantise8<false>(a, scale);
      out[half] = quantise8<false>(bb, scale);
    }
    if (c == 0) *scale_at = scale;
  }
}

// e4m3 pages, prompts. An item is a touched page, K or V of it, and a chunk of
// heads; the page CTAs take equal runs of the items' list. A unit takes R rows
// of the page (as many units as the page has rows; where the CTA has more, they
// take further heads) and HC heads of a chunk. A thread's rows of the next item
// are on their way into its own places in shared memory while it finds the
// peaks of this one and rounds it: nothing is waited for but the peaks, once an
// item. Two CTAs of 64 values a thread fill an SM's registers (and spill a little:
// 144 bytes with one row and four heads a unit, 40 with two and two). (21k tokens of 8
// KV and 32 query heads, us: pages of 16 / 64 / 128 86.7 / 86.5 / 88.3; one CTA for
// each page and K or V, with no load ahead of it, 97 / 87 / 93; three CTAs of 32
// values 92 / 101 / 90; the values rotated twice instead of kept 98 / 97 / 102.)
__host__ __device__ constexpr int prompt_heads(int R) { return R >= 4 ? 1 : 4 / R; }
__host__ __device__ constexpr int prompt_smem(int R) { return 2 * kThreads * R * prompt_heads(R) * 32; }
__host__ __device__ constexpr int prompt_ctas(int R) { return R == 8 ? 1 : 2; }  // on an SM

template <typename T, int R, bool AX>
__global__ void __launch_bounds__(kThreads, prompt_ctas(R))
    append_prompt_q8_kernel(const AppendPagedParams p, int page_ctas, int chunks, int stride) {
  constexpr int HC = prompt_heads(R), kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint4 staged[];  // [2][R * HC][2][kThreads]
  __shared__ int64_t sh_items;
  __shared__ int sh[2];
  __shared__ uint32_t sh_peak[2][HC][kWarps];
  pdl_wait();
  pdl_trigger();
  if constexpr (AX) check_axes(p);
  const int row_vecs = p.head_dim / 8, half = row_vecs / 2, Hkv = p.n_kv_head;
  const int units = kThreads / half, unit = threadIdx.x / half, c = threadIdx.x % half;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((int)blockIdx.x >= page_ctas) {
    const int64_t u = (int64_t)(blockIdx.x - page_ctas) * units + unit, t = u / stride;
    if (t < p.tokens) move_token<T, AX>(p, (int)t, 2 * Hkv + (int)(u - t * stride), stride, c);
    return;
  }
  int first = 0, count = 0, p0 = 0;  // new rows of the sequence at hand
  auto pages_of = [&](int b) {
    return b < p.B && sequence_rows(p, b, &first, &count, &p0) && count > 0
               ? ((p0 + count - 1) >> p.page_shift) - (p0 >> p.page_shift) + 1 : 0;
  };
  if (warp == 0) {
    // the touched pages, in sequence order; the sequence and page of the first item
    int64_t items = 0;
    for (int b = lane; b < p.B; b += 32) items += pages_of(b);
#pragma unroll
    for (int o = 16; o; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
    items *= 2 * chunks;
    const int64_t task = items * blockIdx.x / page_ctas / (2 * chunks);
    int64_t before = 0;
    for (int base = 0; base < p.B; base += 32) {
      const int pages = pages_of(base + lane);
      int sum = pages;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (task >= before + sum - pages && task < before + sum) {
        sh[0] = base + lane;
        sh[1] = (int)(task - (before + sum - pages));
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
      if (before > task) break;
    }
    if (lane == 0) sh_items = items;
  }
  if (blockIdx.x == 0 && p.err_flag) {
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
      if (!sequence_rows(p, b, &first, &count, &p0)) atomicOr(p.err_flag, kErrPosition);
    }
  }
  __syncthreads();
  const int64_t begin = sh_items * blockIdx.x / page_ctas;
  int left = (int)(sh_items * (blockIdx.x + 1) / page_ctas - begin);  // items of this CTA
  if (left == 0) return;
  // the next item: chunk `chunk` of V (which) or K of page j of sequence b
  int b = sh[0], chunk = (int)(begin % chunks), which = (int)(begin / chunks % 2);
  pages_of(b);
  int j = (p0 >> p.page_shift) + sh[1];
  // rows of this unit: slot, slot + slots, ...; its heads of a chunk: from
  // (chunk * at_once + unit / slots) * HC on
  const int slots = p.page_rows / R, slot = unit % slots, at_once = units / slots;
  struct Item {
    int row0, lo, hi, page, which, g0;  // first row of the page, rows [lo, hi) of it, first head of the unit
    int token0;                         // AX: the packed token of position 0 would be (rows' turns are looked up by it)
  };
  auto place = [&](int stage, int i, int k, int which) {
    return staged + (((stage * R + i) * HC + k) * 2 + which) * kThreads + threadIdx.x;
  };
  auto fetch = [&](int stage) {
    Item it;
    it.row0 = j << p.page_shift;
    it.lo = max(p0, it.row0);
    it.hi = min(p0 + count, it.row0 + p.page_rows);
    it.which = which;
    it.g0 = (chunk * at_once + unit / slots) * HC;
    if constexpr (AX) it.token0 = first - p0;
    const uint4* in = reinterpret_cast<const uint4*>(which ? p.v_new : p.k_new);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int position = it.row0 + slot + i * slots;
      if (position >= it.lo && position < it.hi) {
        const uint4* src = in + (((int64_t)first + position - p0) * Hkv + it.g0) * row_vecs + c;
#pragma unroll
        for (int k = 0; k < HC; ++k) {
          if (it.g0 + k < Hkv) {
            copy16(smem_addr(place(stage, i, k, 0)), src + k * row_vecs);
            copy16(smem_addr(place(stage, i, k, 1)), src + k * row_vecs + half);
          }
        }
      }
    }
    copy_commit();
    it.page = p.table[(int64_t)b * p.max_pages + j];
    return it;
  };
  auto advance = [&]() {
    if (++chunk < chunks) return;
    chunk = 0;
    which ^= 1;
    if (which) return;
    if (++j <= (p0 + count - 1) >> p.page_shift) return;
    do ++b; while (pages_of(b) == 0 && b < p.B - 1);  // (an item is left, so there is one)
    j = p0 >> p.page_shift;
  };
  const int team = slots * half, team_warps = team / 32, warp0 = warp / team_warps * team_warps;  // (whole warps)
  const int64_t page_bytes = (int64_t)p.page_rows * p.head_dim;
  int turn = 0;  // items rounded: the one before may still be read where the next one's peaks go
  Item it, ahead = fetch(0);
  for (int n = 0; n < left; ++n) {
    it = ahead;
    if (n + 1 < left) {
      advance();
      ahead = fetch((n + 1) & 1);
      copy_wait<1>();
    } else {
      copy_wait<0>();
    }
    if (it.page < 0 || it.page >= p.num_pages) {
      if (threadIdx.x == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
      continue;
    }
    const int row0 = it.row0, lo = it.lo, hi = it.hi, g0 = it.g0, live = min(HC, Hkv - g0);  // (may be none)
    const bool is_k = !it.which, rotate = is_k && p.cos;
    const int old_rows = lo - row0;
    // the rows' values, kept between the peaks and the rounding
    float va[R][HC][8], vb[R][HC][8], peak[HC];
    uint32_t skipped = 0;  // AX: rows of this unit whose turn is not in the tables
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int position = row0 + slot + i * slots;
      bool on = position >= lo && position < hi;
      TurnRows turn_rows;
      if constexpr (AX) {
        if (on && !turn_rows.load(p, it.token0 + position)) {
          on = false;
          skipped |= 1u << i;
          if (c == 0 && p.err_flag) atomicOr(p.err_flag, kErrPosition);
        }
      }
#pragma unroll
      for (int k = 0; k < HC; ++k) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        const bool in = on && k < live;
        Storage<T>::unpack(in ? *place(n & 1, i, k, 0) : none, va[i][k]);
        Storage<T>::unpack(in ? *place(n & 1, i, k, 1) : none, vb[i][k]);
      }
      if (on && rotate) rotate_rows<AX, HC>(p, position, turn_rows, c, va[i], vb[i]);
    }
    auto find_peaks = [&](auto finite) {
#pragma unroll
      for (int k = 0; k < HC; ++k) {
        peak[k] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i)
          peak[k] = decltype(finite)::value ? finite_peak(finite_peak(peak[k], va[i][k]), vb[i][k])
                                            : peak_of(peak_of(peak[k], va[i][k]), vb[i][k]);
      }
      // (non-negative floats order as their bits do)
#pragma unroll
      for (int k = 0; k < HC; ++k) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(peak[k]));
        if (lane == 0) sh_peak[turn][k][warp] = m;
      }
      __syncthreads();
      bool infinity = false;
#pragma unroll
      for (int k = 0; k < HC; ++k) {
        const uint32_t v = sh_peak[turn][k][lane % kWarps];
        infinity |= __any_sync(0xffffffffu, v == 0x7f800000u);  // in any team
        const int w = lane % kWarps - warp0;
        peak[k] = __uint_as_float(__reduce_max_sync(0xffffffffu, w >= 0 && w < team_warps ? v : 0u));
      }
      return infinity;
    };
    const int64_t block = (int64_t)it.page * Hkv + g0;
    float* scale_at = (is_k ? p.k_scale : p.v_scale) + block;
    uint8_t* rows = (is_k ? p.k_pages : p.v_pages) + block * page_bytes;
    float old_scale[HC];
#pragma unroll
    for (int k = 0; k < HC; ++k) old_scale[k] = old_rows > 0 && k < live ? scale_at[k] : 0.f;
    const bool infinities = find_peaks(std::false_type());
    if (infinities) {
      __syncthreads();
      find_peaks(std::true_type());
    }
    float scale[HC];
    bool careful = infinities;
#pragma unroll
    for (int k = 0; k < HC; ++k) {
      scale[k] = fmaxf(scale_of(peak[k]), old_scale[k]);
      careful |= !power_of_two(scale[k]);
      if (old_rows > 0 && k < live && scale[k] != old_scale[k])
        rescale_rows(rows + k * page_bytes, old_rows * p.head_dim, old_scale[k] / scale[k],
                     threadIdx.x % team, team);
    }
    auto round_rows = [&](auto some) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int position = row0 + slot + i * slots;
        if (position < lo || position >= hi || (AX && (skipped >> i & 1))) continue;
#pragma unroll
        for (int k = 0; k < HC; ++k) {
          if (k >= live) break;
          uint2* out = reinterpret_cast<uint2*>(rows + k * page_bytes + (position - row0) * p.head_dim) + c;
          out[0] = quantise8<decltype(some)::value>(va[i][k], scale[k]);
          out[half] = quantise8<decltype(some)::value>(vb[i][k], scale[k]);
        }
      }
    };
    if (careful) {
      round_rows(std::true_type());
    } else {
      round_rows(std::false_type());
    }
    if (slot == 0 && c == 0) {
#pragma unroll
      for (int k = 0; k < HC; ++k)
        if (k < live) scale_at[k] = scale[k];
    }
    turn ^= 1;
  }
}

template <typename T, int R, bool AX>
cudaError_t launch_prompt_q8(cudaLaunchConfig_t cfg, const AppendPagedParams& p, int page_ctas, int chunks,
                             int stride) {
  auto* fn = append_prompt_q8_kernel<T, R, AX>;
  cfg.dynamicSmemBytes = prompt_smem(R);
  static std::atomic<bool> ready[64];  // per device: the shared-memory opt-in is applied
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!ready[device].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, prompt_smem(R));
    if (e != cudaSuccess) return e;
    ready[device].store(true, std::memory_order_release);
  }
  return cudaLaunchKernelEx(&cfg, fn, p, page_ctas, chunks, stride);
}

// Units for each token. A unit that takes more heads looks its place and table
// row up for more bytes, but leaves fewer threads to wait for memory: as many
// heads as keep about one wave of CTAs (two of 256 threads an SM), at most
// kTurns * kAtOnce. Measured for 48 heads of 128, us with one head a unit / this
// rule / the most heads a unit: 32 tokens 2.5 / 2.5 / 8.2, 512 6.6 / 3.6 / 8.5, 1024
// 13.7 / 6.0 / 10.8, 2048 25.5 / 10.4 / 12.0, 4096 49.5 / 17.5 / 17.5.
constexpr int kTurns = 4, kThreadsPerSm = 384;
int units_per_token(int64_t tokens, int heads, int half, int sms) {
  const int64_t fit = tokens * heads * half / ((int64_t)sms * kThreadsPerSm);
  const int each = (int)std::min<int64_t>(std::max<int64_t>(fit, 1), kTurns * kAtOnce);
  return (heads + each - 1) / each;
}

}  // namespace

namespace {

template <typename T, bool AX>
cudaError_t launch_append_as(const AppendPagedParams& p, int sms, cudaStream_t stream) {
  const int half = p.head_dim / 16, units = kThreads / half, query_heads = p.q ? p.n_head : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto grid = [&](int64_t ctas) {
    cfg.gridDim = dim3((unsigned)ctas);
    return ctas <= INT32_MAX;
  };
  auto ctas_of = [&](int64_t n) { return (n + units - 1) / units; };
  if (!p.k_scale) {
    const int heads = 2 * p.n_kv_head + query_heads, stride = units_per_token(p.tokens, heads, half, sms);
    if (!grid(ctas_of((int64_t)p.tokens * stride))) return cudaErrorInvalidConfiguration;
    return cudaLaunchKernelEx(&cfg, append_paged_kernel<T, AX>, p, stride);
  }
  const int stride = query_heads ? units_per_token(p.tokens, query_heads, half, sms) : 1;
  const int64_t query_ctas = query_heads ? ctas_of((int64_t)p.tokens * stride) : 0;
  if (!p.start) {
    const int64_t rows = ctas_of((int64_t)p.B * 2 * p.n_kv_head);
    if (!grid(rows + query_ctas)) return cudaErrorInvalidConfiguration;
    return cudaLaunchKernelEx(&cfg, append_token_q8_kernel<T, AX>, p, (int)rows, stride);
  }
  // n rows touch at most (n - 2) / page + 2 pages
  const int64_t tasks = std::min<int64_t>((int64_t)p.tokens / p.page_rows + 2 * (int64_t)p.B, p.tokens);
  const int R = std::max(1, p.page_rows / units);
  const int chunk_heads = units / (p.page_rows / R) * prompt_heads(R);
  const int chunks = (p.n_kv_head + chunk_heads - 1) / chunk_heads;
  const int64_t page_ctas = std::min(tasks * 2 * chunks, (int64_t)sms * prompt_ctas(R));
  if (!grid(page_ctas + query_ctas)) return cudaErrorInvalidConfiguration;
  auto launch = [&](auto rows) {
    constexpr int kR = decltype(rows)::value;
    return launch_prompt_q8<T, kR, AX>(cfg, p, (int)page_ctas, chunks, stride);
  };
  switch (R) {
    case 1: return launch(std::integral_constant<int, 1>());
    case 2: return launch(std::integral_constant<int, 2>());
    case 4: return launch(std::integral_constant<int, 4>());
    default: return launch(std::integral_constant<int, 8>());
  }
}

}  // namespace

cudaError_t launch_append_paged(const AppendPagedParams& p, int dtype, int sms, cudaStream_t stream) {
  if (p.turn)
    return dtype == DA_F16 ? launch_append_as<__half, true>(p, sms, stream)
                           : launch_append_as<__nv_bfloat16, true>(p, sms, stream);
  return dtype == DA_F16 ? launch_append_as<__half, false>(p, sms, stream)
                         : launch_append_as<__nv_bfloat16, false>(p, sms, stream);
}

}  // namespace da
