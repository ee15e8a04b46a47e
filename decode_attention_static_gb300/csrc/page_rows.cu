// Rows and pages that move inside the pools: copies of pages (forks), and rows
// of accepted tokens moved together.
//
// Both only move bytes. A page of one KV head is contiguous, so that a copy is
// one run for each (entry, layer, K or V, head). Compaction works in place: a
// thread owns one 16-byte column of a sequence's rows (of one layer, K or V and
// head) and moves it row by row in rising order, reading a batch of rows before
// it writes them; since a row never moves up, what is written has been read,
// and no thread waits for another.
//
// Measured on one GB300, device time inside a graph: copies of 64 part-filled
// pages of 12 layers (96 beams, 8 heads of 128, pages of 64), with the resize and the
// fork before them, 37 us, of which the bytes need 29.6; the accepted rows of 8 sequences in one
// layer 3.4 us (launch and three dependent loads), of 64 sequences in 36 layers of
// 8 bits 50 us (66 with nothing in L2), of which 7.7 would move the 6410 blocks whose
// scale grows: a thread rounds its column of a block's other rows one after the other, each load
// behind the store before it. Where no scale grows 19.4 us, floor 5.8: rows of 128 bytes, each
// by itself in 2.4 GB.
#include <stdint.h>

#include "common.cuh"
#include "page_params.h"

namespace da {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const MoveParams p) {
  pdl_wait();
  pdl_trigger();
  // blockIdx.x: (entry, layer, K or V, head), heads fastest
  uint32_t at = blockIdx.x;
  const int g = at % p.n_kv_head;
  at /= p.n_kv_head;
  const bool is_v = at & 1;
  at /= 2;
  const int layer = at % p.layers, i = at / p.layers;
  const int src = p.copies[i], dst = p.copies[p.n + i], rows = p.copies[2 * (int64_t)p.n + i];
  if (src < 0 || dst < 0) return;
  if (src >= p.num_pages || dst >= p.num_pages || rows < 0 || rows > p.page_rows) {
    if (threadIdx.x == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
    return;
  }
  if (src == dst) return;
  const int64_t from = ((int64_t)layer * p.num_pages + src) * p.n_kv_head + g;
  const int64_t to = ((int64_t)layer * p.num_pages + dst) * p.n_kv_head + g;
  uint4* const pool = reinterpret_cast<uint4*>(is_v ? p.v : p.k);
  const int64_t page_vecs = (int64_t)p.page_rows * p.row_vecs;
  const uint4* const x = pool + from * page_vecs;
  uint4* const y = pool + to * page_vecs;
  const int vecs = rows * p.row_vecs;
  for (int v0 = threadIdx.x; v0 < vecs; v0 += 4 * kThreads) {
    uint4 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v0 + k * kThreads < vecs) r[k] = ld_global_nc_v4(x + v0 + k * kThreads);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v0 + k * kThreads < vecs) y[v0 + k * kThreads] = r[k];
  }
  if (p.k_scale && threadIdx.x == 0) {
    float* const scale = is_v ? p.v_scale : p.k_scale;
    scale[to] = scale[from];
  }
}

__device__ __forceinline__ uint32_t scaled4(uint32_t v, float ratio) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(v & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(v >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  uint16_t x, y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(x) : "f"(a.y * ratio), "f"(a.x * ratio));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b.y * ratio), "f"(b.x * ratio));
  return (uint32_t)x | ((uint32_t)y << 16);
}

// 16 codes of scale `from` as codes of scale `to` >= from.
__device__ __forceinline__ uint4 rescaled(const uint4& v, float from, float to) {
  if (from == to) return v;
  const float ratio = from / to;
  return make_uint4(scaled4(v.x, ratio), scaled4(v.y, ratio), scaled4(v.z, ratio), scaled4(v.w, ratio));
}

// Column c of (sequence b, layer, K or V, head g), as numbered by thread.
template <bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? 4 : 3) compact_kernel(const MoveParams p) {
  constexpr int kBatch = EIGHT ? 4 : 8;  // rows on their way at once
  pdl_wait();
  pdl_trigger();
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / p.row_vecs;
  const int c = threadIdx.x % p.row_vecs;  // (row_vecs divides the block)
  int64_t at = unit;
  const int g = (int)(at % p.n_kv_head);
  at /= p.n_kv_head;
  const bool is_v = at & 1;
  at /= 2;
  const int layer = (int)(at % p.layers);
  const int64_t b = at / p.layers;
  if (b >= p.B) return;
  const bool reports = c == 0 && g == 0 && !is_v && layer == 0;
  const int s0 = p.start[b], s1 = p.start[b + 1], first = p.pos[b];
  int errors = 0;
  if (s0 < 0 || s1 < s0 || s1 > p.kept) {
    if (reports && p.err_flag) atomicOr(p.err_flag, kErrTokens);
    return;
  }
  const int n = s1 - s0, limit = p.max_pages << p.page_shift;
  const int32_t* const keep = p.keep + s0;
  const int32_t* const table = p.table + b * p.max_pages;
  uint4* const pool = reinterpret_cast<uint4*>(is_v ? p.v : p.k);
  const int64_t page_vecs = (int64_t)p.page_rows * p.row_vecs;
  // a page's first vector of this column, or null outside the pool
  auto block = [&](int id) { return ((int64_t)layer * p.num_pages + id) * p.n_kv_head + g; };
  auto inside = [&](int id) { return id >= 0 && id < p.num_pages; };
  int last = first - 1;  // keep[i] has to be above it, and at least first + i
  auto valid = [&](int i, int row) { return first >= 0 && row > last && row >= first + (int64_t)i && row < limit; };
  if constexpr (!EIGHT) {
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      const int m = min(kBatch, n - i0);
      uint4 x[kBatch];
      uint4* to[kBatch];
      bool ok = true;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        to[k] = nullptr;
        if (k >= m || !ok) continue;
        const int row = keep[i0 + k], target = first + i0 + k;
        ok = valid(i0 + k, row);
        if (!ok) continue;
        last = row;
        if (row == target) continue;
        const int a = table[row >> p.page_shift], d = table[target >> p.page_shift];
        if (!inside(a) || !inside(d)) {
          errors |= kErrPage;
          continue;
        }
        x[k] = pool[block(a) * page_vecs + (row & (p.page_rows - 1)) * p.row_vecs + c];
        to[k] = pool + block(d) * page_vecs + (target & (p.page_rows - 1)) * p.row_vecs + c;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (to[k]) *to[k] = x[k];
      if (!ok) {
        errors |= kErrPosition;
        break;
      }
    }
  } else {
    float* const scales = is_v ? p.v_scale : p.k_scale;
    // the lanes of a unit share its page scales: they are read by all before one writes them
    const uint32_t team = (p.row_vecs == 32 ? 0xffffffffu : (1u << p.row_vecs) - 1) << (threadIdx.x % 32 / p.row_vecs * p.row_vecs);
    bool ok = true;
    int pages[kBatch];
    for (int i0 = 0; i0 < n && ok;) {
      // rows of one target page
      const int target0 = first + i0;
      if (target0 < 0 || target0 >= limit) {
        ok = false;
        break;
      }
      const int page_end = ((target0 >> p.page_shift) + 1) << p.page_shift;
      const int i1 = min(n, page_end - first);
      const int d = table[target0 >> p.page_shift];
      const bool d_ok = inside(d);
      const float own = d_ok ? scales[block(d)] : 0.f;
      float scale = own;
      // Rows of the first kBatch on their way at once: their numbers, pages, scales, then the rows themselves; of further
      // ones in the page only the scales at first.
      int end = i0;  // rows [i0, end) are valid
      int src[kBatch];
      float from[kBatch];
      for (int j0 = i0; j0 < i1 && end == j0; j0 += kBatch) {
        int row[kBatch], a[kBatch];
        float s[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) row[k] = j0 + k < i1 ? keep[j0 + k] : -1;
        int good = 0;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          if (good == k && j0 + k < i1 && valid(j0 + k, row[k])) {
            last = row[k];
            ++good;
          }
        }
        end = j0 + good;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) a[k] = k < good ? table[row[k] >> p.page_shift] : -1;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const bool in = k < good && inside(a[k]);
          if (k < good && !in) errors |= kErrPage;
          s[k] = in ? scales[block(a[k])] : 0.f;
          scale = fmaxf(scale, s[k]);
          if (j0 == i0) {
            // (a row that stays, or cannot be had, is one of the page's other rows)
            const int target = first + j0 + k;
            const bool moves = in && row[k] != target;
            src[k] = moves ? row[k] : target;
            from[k] = moves ? s[k] : own;
            a[k] = moves ? a[k] : d;
            row[k] = k < good ? a[k] : -1;
          }
        }
        if (j0 == i0) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) pages[k] = row[k];
        }
      }
      __syncwarp(team);
      if (d_ok && end > i0) {
        uint4* const out = pool + block(d) * page_vecs + c;
        for (int j0 = i0; j0 < end; j0 += kBatch) {
          if (j0 > i0) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int row = j0 + k < end ? keep[j0 + k] : -1, target = first + j0 + k;
              const int a = row >= 0 ? table[row >> p.page_shift] : -1;
              const bool moves = inside(a) && row != target;
              src[k] = moves ? row : target;
              pages[k] = row < 0 ? -1 : moves ? a : d;
              from[k] = moves ? (a == d ? own : scales[block(a)]) : own;
            }
          }
          uint4 x[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (pages[k] >= 0 && (pages[k] != d || src[k] != first + j0 + k || scale != own))
              x[k] = pool[block(pages[k]) * page_vecs + (int64_t)(src[k] & (p.page_rows - 1)) * p.row_vecs + c];
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (pages[k] >= 0 && (pages[k] != d || src[k] != first + j0 + k || scale != own))
              out[(int64_t)((first + j0 + k) & (p.page_rows - 1)) * p.row_vecs] = rescaled(x[k], from[k], scale);
          }
        }
        if (scale != own) {
          // the page's other rows
          const int lo = target0 & (p.page_rows - 1), hi = lo + (end - i0);
#pragma unroll 4
          for (int r = 0; r < p.page_rows; ++r)
            if (r < lo || r >= hi) out[(int64_t)r * p.row_vecs] = rescaled(out[(int64_t)r * p.row_vecs], own, scale);
        }
      } else if (end > i0) {
        errors |= kErrPage;
      }
      __syncwarp(team);
      if (d_ok && end > i0 && scale != own && c == 0) scales[block(d)] = scale;
      __syncwarp(team);
      ok = end == i1;
      i0 = i1;
    }
    if (!ok) errors |= kErrPosition;
  }
  if (reports && errors && p.err_flag) atomicOr(p.err_flag, errors);
}

cudaLaunchConfig_t config(int64_t blocks, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_copy_pages(const MoveParams& p, cudaStream_t stream) {
  const int64_t blocks = (int64_t)p.n * p.layers * 2 * p.n_kv_head;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(blocks, stream, &attr);
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, p);
}

cudaError_t launch_compact(const MoveParams& p, cudaStream_t stream) {
  const int64_t threads = (int64_t)p.B * p.layers * 2 * p.n_kv_head * p.row_vecs;
  const int64_t blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(blocks, stream, &attr);
  return p.k_scale ? cudaLaunchKernelEx(&cfg, compact_kernel<true>, p)
                   : cudaLaunchKernelEx(&cfg, compact_kernel<false>, p);
}

}  // namespace da
