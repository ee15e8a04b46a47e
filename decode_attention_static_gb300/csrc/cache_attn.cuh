// Decode attention over a paged cache (16-bit or e4m3 pages) or a static
// cache, with an optional sliding window and sinks.
//
// For sequence b, KV head g and its G <= 8 query heads, over the visible rows j
//   x_j = scale <q_h, K_j>,  out_h = sum_j 2^(x'_j - m) V_j / sum_j 2^(x'_j - m)
// with x' = x log2(e) and a running reference m, one pass over K and V.
//
// Bound: HBM. A step reads 2 n_visible D elements for each KV head and
// computes 4 G operations on each pair, far below the tensor ridge; what has
// to be kept short is the work per byte on the SM, and the tail.
//
// Work split. The visible rows of a group (b, g) are cut into tiles of 16 rows
// that start at multiples of 16 (so that a tile never crosses a page, of at
// least 16 rows), and the tiles of all groups form one list in (b, g, row)
// order. CTA i of n owns an even share of the list, whatever the lengths, the
// window or the batch are: every CTA computes the list from kv_len itself, so
// the launch does not depend on lengths and ragged batches are balanced to
// one tile. A group that lies in several shares is joined through the
// workspace by the last CTA to arrive.
//
// A warp takes every kWarps-th tile of the share, with a ring of its own that
// asynchronous copies keep filled (page numbers are looked up one tile ahead),
// and no barrier within a group. Per tile:
//   S^T [16 rows x 8 heads] = K q^T        mma m16n8k16, K by ldmatrix
//   p = 2^(x' - m), m raised only when a score passes it by 2^8 (a vote)
//   out^T [D x 8 heads] += V^T P^T         V by ldmatrix.trans, P^T by movmatrix
// The heads are the 8 columns of the instruction, so a group of any size
// costs the same, and scores and weights stay in registers. (One decode tile
// is far too small for tcgen05: its 128-row operand would hold 8 tiles of
// different pages, and its accumulator would have to come back from tensor
// memory for every softmax.) Weights are split in two 16-bit pieces, p = hi +
// lo, each multiplied with V: the sum keeps the 16 (bf16) to 22 (fp16) bits
// that one 16-bit weight would lose, for 8 more products a tile.
#pragma once

#include <atomic>

#include "cache_params.h"
#include "common.cuh"

namespace da {

constexpr int kHeads = 8;        // columns of the matrix instruction
constexpr int kTileRows = 16;
constexpr int kMaxCtas = 512;    // parts of one group, at most
constexpr int kCtasPerSm = 2;
constexpr float kLazy = 8.f;     // m is raised when a score passes it by this (log2)
// fp16 weights are 2^(x' - m + 7): at most 2^15, inside the type's range, and
// 2^-32 of the largest one is still held. bf16 has fp32's range: no lift.
constexpr float kLiftF16 = 7.f;

template <bool E4M3, int D>
struct CacheAttnShape {
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kTileBytes = kTileRows * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K tile, V tile
  static constexpr int kStages = 24576 / kStageBytes < 8 ? 24576 / kStageBytes : 8;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeFloats = kWarps * kHeads * D;
  static constexpr int kMergeBytes = (kMergeFloats > kMaxCtas * kHeads ? kMergeFloats : kMaxCtas * kHeads) * 4;
  static constexpr int kMetaOffset = kRingBytes + kMergeBytes;  // per warp and stage: k scale, v scale, bad page
  static constexpr int kStatOffset = kMetaOffset + kWarps * kStages * 16;
  // (m, l) of each warp, factors, group sums; schedule words
  static constexpr int kStatFloats = 2 * kWarps * kHeads + kWarps * kHeads + 2 * kHeads;
  static constexpr int kWordsOffset = kStatOffset + kStatFloats * 4;
  static constexpr int kSmemBytes = kWordsOffset + (2 * kWarps + 8) * 8;
  static_assert(kStages >= 3, "a ring of at least three stages");
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

// Byte offset of 16-byte chunk c of row r in a tile: chunks are permuted
// within 128-byte lines so that ldmatrix and the copies hit every bank once.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t chunk_offset(int r, int c) {
  if constexpr (ROW_BYTES == 64) {
    return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r >> 1) & 7)) << 4);
  } else {
    return r * ROW_BYTES + ((c ^ (r & 7)) << 4);
  }
}

// Column of element d of head h in the merge buffer: heads are rotated
// against each other so that a warp's stores hit every bank once.
template <int D>
__device__ __forceinline__ int merge_column(int h, int d) {
  return (d + 8 * (h >> 1)) & (D - 1);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// (nothing is read, and zeros are written, when bytes is 0)
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Two e4m3 values (the low or the high half of v) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_low(uint32_t v) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(v));
  return h;
}
__device__ __forceinline__ uint32_t e4m3_high(uint32_t v) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(v));
  return h;
}

// a and b rounded to 16 bits, packed; *rest their remainders, packed.
template <bool BF16>
__device__ __forceinline__ uint32_t split_pair(float a, float b, uint32_t* rest) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(a - f.x, b - f.y);
    *rest = *reinterpret_cast<const uint32_t*>(&r);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(a - f.x, b - f.y);
    *rest = *reinterpret_cast<const uint32_t*>(&r);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Tiles of one sequence: visible rows [0, s0) and [w0, len). Tile i < sink_tiles
// is rows [16 i, 16 i + 16); the others start at row 16 first_tile.
struct SequenceTiles {
  int len, w0, s0, sink_tiles, first_tile, tiles;
};

// -1: the length is out of range.
__device__ __forceinline__ int tiles_of(const CacheAttnParams& p, int len, SequenceTiles* s) {
  if (len < 0 || len > p.max_len) {
    s->tiles = 0;
    return -1;
  }
  s->len = len;
  s->w0 = (p.window > 0 && len > p.window) ? len - p.window : 0;
  s->s0 = min(p.sinks, s->w0);
  s->first_tile = s->w0 / kTileRows;
  // a sink tile that the window reaches into belongs to the window's tiles
  s->sink_tiles = min((s->s0 + kTileRows - 1) / kTileRows, s->first_tile);
  s->tiles = len == 0 ? 0 : s->sink_tiles + (len + kTileRows - 1) / kTileRows - s->first_tile;
  return s->tiles;
}

__device__ __forceinline__ int tile_row(const SequenceTiles& s, int i) {
  return (i < s.sink_tiles ? i : i - s.sink_tiles + s.first_tile) * kTileRows;
}

// Bit r: row row0 + r is visible.
__device__ __forceinline__ uint32_t tile_mask(const SequenceTiles& s, int row0) {
  const int end = min(s.len - row0, kTileRows);                       // >= 1
  uint32_t mask = 0xffffu >> (kTileRows - end);
  if (row0 < s.w0) {
    const int gap_lo = max(s.s0 - row0, 0), gap_hi = min(s.w0 - row0, kTileRows);
    if (gap_hi > gap_lo) mask &= ~((0xffffu >> (kTileRows - (gap_hi - gap_lo))) << gap_lo);
  }
  return mask;
}

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(CacheAttnShape<E4M3, D>::kThreads, kCtasPerSm)
    cache_attn_kernel(const CacheAttnParams p) {
  using Sh = CacheAttnShape<E4M3, D>;
  constexpr bool kBf16 = !E4M3 && Storage<T>::kBf16;  // type of the matrix operands
  constexpr float kLift = kBf16 ? 0.f : kLiftF16;
  constexpr int kW = Sh::kWarps, kS = Sh::kStages, kSteps = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + Sh::kRingBytes);
  float* sm_m = reinterpret_cast<float*>(smem + Sh::kStatOffset);  // [kW][8]
  float* sm_l = sm_m + kW * kHeads;
  float* sm_f = sm_l + kW * kHeads;   // factor of each warp's state
  float* sm_gm = sm_f + kW * kHeads;  // group's m and l
  float* sm_gl = sm_gm + kHeads;
  int64_t* words = reinterpret_cast<int64_t*>(smem + Sh::kWordsOffset);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gr = lane >> 2, tq = lane & 3;

  pdl_wait();

  // --- the list of tiles, and this CTA's share [lo, hi) of it
  int64_t total = 0;
  for (int base = 0; base < p.B; base += Sh::kThreads) {
    const int b = base + tid;
    SequenceTiles s;
    int n = 0;
    if (b < p.B) {
      n = tiles_of(p, p.kv_len[b], &s);
      if (n <= 0 && b % gridDim.x == blockIdx.x) {
        // no visible row: zeros; no valid length: NaN
        const uint32_t fill = n < 0 ? (uint32_t)Storage<T>::kNaN * 0x10001u : 0u;
        if (n < 0 && p.err_flag) atomicOr(p.err_flag, kErrKvLen);
        uint4* out = reinterpret_cast<uint4*>(p.out) + (int64_t)b * p.n_head * (D / 8);
        for (int i = 0; i < p.n_head * (D / 8); ++i) out[i] = make_uint4(fill, fill, fill, fill);
      }
      n = max(n, 0);
    }
    int64_t sum = n;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) words[warp] = sum;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) total += words[w];
    __syncthreads();
  }
  total *= p.n_kv_head;
  // at least one tile for every warp
  const int64_t ctas = min((int64_t)gridDim.x, (total + kW - 1) / kW);
  if ((int64_t)blockIdx.x >= ctas) return;
  const int64_t lo = blockIdx.x * total / ctas, hi = (blockIdx.x + 1) * total / ctas;
  {
    int64_t before = 0;
    for (int base = 0; base < p.B; base += Sh::kThreads) {
      const int b = base + tid;
      SequenceTiles s;
      const int64_t n = b < p.B ? (int64_t)max(tiles_of(p, p.kv_len[b], &s), 0) * p.n_kv_head : 0;
      int64_t sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) words[warp] = sum;
      __syncthreads();
      int64_t mine = before + sum - n;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        if (w < warp) mine += words[w];
        before += words[w];
      }
      if (n > 0 && mine <= lo && lo < mine + n) {
        words[kW] = b;
        words[kW + 1] = mine;
      }
      __syncthreads();
      if (before > lo) break;
    }
  }
  int b = (int)words[kW];
  SequenceTiles seq;
  tiles_of(p, p.kv_len[b], &seq);
  int g, first_in_group;  // group of list position `lo`, and its place there
  {
    const int64_t in = lo - words[kW + 1];
    g = (int)(in / seq.tiles);
    first_in_group = (int)(in - (int64_t)g * seq.tiles);
  }

  // --- this warp's loads
  const uint32_t ring = smem_addr(smem) + warp * kS * Sh::kStageBytes;
  const uint32_t meta = smem_addr(smem + Sh::kMetaOffset) + warp * kS * 16;
  constexpr int kChunks = Sh::kRowBytes / 16, kCopies = kTileRows * kChunks / 32;
  // the tile to load next, its page number on the way
  SequenceTiles lseq = seq;
  int lb = b, lg = g, li = first_in_group, lrow = 0, lpage = 0;
  int64_t lat = lo;  // list position of (lb, lg, li)
  auto look_up = [&](int step) {  // moves on by `step` tiles
    lat += step;
    if (lat >= hi) return;
    li += step;
    while (li >= lseq.tiles) {
      li -= lseq.tiles;
      if (++lg == p.n_kv_head) {
        lg = 0;
        do ++lb;
        while (tiles_of(p, p.kv_len[lb], &lseq) <= 0);
      }
    }
    lrow = tile_row(lseq, li);
    lpage = p.table ? p.table[(int64_t)lb * p.max_pages + (lrow >> p.page_shift)] : lb;
  };
  auto issue = [&](int stage, int row0, int page, uint32_t mask, int head) {
    const bool bad = page < 0 || page >= p.num_pages;
    if (bad) {
      page = 0;
      mask = 0;
    }
    const int64_t block = (int64_t)page * p.n_kv_head + head;
    const int64_t at = (block * p.page_rows + (row0 & (p.table ? p.page_rows - 1 : -1))) * Sh::kRowBytes;
    const uint8_t* ksrc = p.k + at;
    const uint8_t* vsrc = p.v + at;
    const uint32_t dst = ring + stage * Sh::kStageBytes;
    if (mask == 0xffffu) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int x = lane + 32 * j;
        const uint32_t d = dst + chunk_offset<Sh::kRowBytes>(x / kChunks, x % kChunks);
        copy16(d, ksrc + x * 16);
        copy16(d + Sh::kTileBytes, vsrc + x * 16);
      }
    } else {
      for (int j = 0; j < kCopies; ++j) {
        const int x = lane + 32 * j, r = x / kChunks;
        const bool on = (mask >> r) & 1;
        const uint32_t d = dst + chunk_offset<Sh::kRowBytes>(r, x % kChunks);
        copy16_or_zero(d, on ? ksrc + x * 16 : p.k, on ? 16 : 0);
        copy16_or_zero(d + Sh::kTileBytes, on ? vsrc + x * 16 : p.v, on ? 16 : 0);
      }
    }
    if constexpr (E4M3) {
      if (lane < 2) copy4(meta + stage * 16 + lane * 4, (lane ? p.v_scale : p.k_scale) + block);
    }
    if (lane == 2) asm volatile("st.shared.u32 [%0], %1;" ::"r"(meta + stage * 16 + 8), "r"((uint32_t)bad) : "memory");
    if (bad && lane == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
  };
  int put = 0;  // stage that the next load goes to
  {
    // the first kS - 1 tiles: their page numbers are looked up together
    int rows[kS - 1], pages[kS - 1], heads[kS - 1];
    uint32_t masks[kS - 1];
#pragma unroll
    for (int j = 0; j < kS - 1; ++j) {
      look_up(j ? kW : warp);
      rows[j] = lrow;
      pages[j] = lpage;
      heads[j] = lg;
      masks[j] = lat < hi ? tile_mask(lseq, lrow) : 0;
    }
#pragma unroll
    for (int j = 0; j < kS - 1; ++j) {
      if (masks[j]) issue(j, rows[j], pages[j], masks[j], heads[j]);
      copy_commit();
    }
    put = kS - 1;
    look_up(kW);
  }

  // --- group by group
  int64_t at = lo;  // list position of the next tile to compute
  int get = 0;      // stage of this warp's next tile
  int tile = first_in_group;
  int turn = warp;  // tiles until this warp's next one
  while (at < hi) {
    const int here = (int)min((int64_t)(seq.tiles - tile), hi - at);  // tiles of the group in this share
    // q as the right operand: columns are heads
    uint32_t qb[kSteps][2];
    float scale0 = p.qscale, scale1 = p.qscale;
    {
      const bool on = gr < p.group;
      const uint8_t* qh = p.q + ((int64_t)b * p.n_head + (int64_t)g * p.group + (on ? gr : 0)) * D * 2;
      if constexpr (!E4M3) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          qb[k][0] = on ? *reinterpret_cast<const uint32_t*>(qh + (16 * k + 2 * tq) * 2) : 0u;
          qb[k][1] = on ? *reinterpret_cast<const uint32_t*>(qh + (16 * k + 2 * tq + 8) * 2) : 0u;
        }
      } else {
        // K is read as fp16, 4 consecutive elements a lane; q has to be fp16
        // too. bf16 values are brought into its range by a power of two for
        // each head: elements below 2^-14 of the head's largest lose bits
        // that are below 2^-25 of it.
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint2 v = on ? *reinterpret_cast<const uint2*>(qh + (16 * k + 4 * tq) * 2) : make_uint2(0u, 0u);
          qb[k][0] = v.x;
          qb[k][1] = v.y;
        }
        if constexpr (Storage<T>::kBf16) {
          float peak = 0.f;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              peak = fmaxf(peak, fabsf(__uint_as_float(qb[k][i] << 16)));
              peak = fmaxf(peak, fabsf(__uint_as_float(qb[k][i] & 0xffff0000u)));
            }
          }
          peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
          peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
          int e = (int)(__float_as_uint(peak) >> 23) - 127;
          e = peak == 0.f ? 0 : max(-126, min(e, 126));
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
          const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const __half2 h = __floats2half2_rn(__uint_as_float(qb[k][i] << 16) * down,
                                                  __uint_as_float(qb[k][i] & 0xffff0000u) * down);
              qb[k][i] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          scale0 *= __shfl_sync(0xffffffffu, up, 8 * tq);
          scale1 *= __shfl_sync(0xffffffffu, up, 8 * tq + 4);
        }
      }
    }
    float o[kSteps][4], m0 = -INFINITY, m1 = -INFINITY, lift0 = kLift, lift1 = kLift, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;

    for (; turn < here; turn += kW) {
      const int row0 = tile_row(seq, tile + turn);
      const uint32_t mask = tile_mask(seq, row0);
      copy_wait<kS - 2>();
      __syncwarp();
      // refill the stage that the tile before this one has left
      if (lat < hi) {
        issue(put, lrow, lpage, tile_mask(lseq, lrow), lg);
        look_up(kW);
      }
      copy_commit();
      put = put + 1 == kS ? 0 : put + 1;
      const uint32_t stage = ring + get * Sh::kStageBytes;
      float ks = 1.f, vs = 1.f;
      uint32_t bad;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(bad) : "r"(meta + get * 16 + 8));
      if constexpr (E4M3) asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(meta + get * 16));
      get = get + 1 == kS ? 0 : get + 1;

      // scores: rows gr and gr + 8, heads 2 tq and 2 tq + 1
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
      const int mr = (lane & 7) + ((lane >> 3) & 1) * 8;
      if constexpr (!E4M3) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          ldmatrix_x4(stage + chunk_offset<Sh::kRowBytes>(mr, 2 * k + (lane >> 4)), a);
          mma_16x8x16<kBf16>(k & 1 ? s2 : s, a[0], a[1], a[2], a[3], qb[k][0], qb[k][1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t a[4];
          ldmatrix_x4(stage + chunk_offset<Sh::kRowBytes>(mr, k + (lane >> 4)), a);
          mma_16x8x16<false>(s, e4m3_low(a[0]), e4m3_low(a[1]), e4m3_high(a[0]), e4m3_high(a[1]), qb[k][0], qb[k][1]);
          mma_16x8x16<false>(s2, e4m3_low(a[2]), e4m3_low(a[3]), e4m3_high(a[2]), e4m3_high(a[3]), qb[k + 1][0],
                             qb[k + 1][1]);
        }
      }
      const float f0 = E4M3 ? scale0 * ks : scale0, f1 = E4M3 ? scale1 * ks : scale1;
      float x[4] = {(s[0] + s2[0]) * f0, (s[1] + s2[1]) * f1, (s[2] + s2[2]) * f0, (s[3] + s2[3]) * f1};
      if (mask != 0xffffu) {
        if (!((mask >> gr) & 1)) x[0] = x[1] = -INFINITY;
        if (!((mask >> (gr + 8)) & 1)) x[2] = x[3] = -INFINITY;
      }
      float a0 = fmaxf(x[0], x[2]), a1 = fmaxf(x[1], x[3]);
      if (__any_sync(0xffffffffu, a0 > m0 + kLazy || a1 > m1 + kLazy)) {
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
          a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, i));
          a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, i));
        }
        a0 = fmaxf(a0, m0);
        a1 = fmaxf(a1, m1);
        const float c0 = a0 == m0 ? 1.f : fast_exp2(m0 - a0), c1 = a1 == m1 ? 1.f : fast_exp2(m1 - a1);
        m0 = a0;
        m1 = a1;
        lift0 = kLift - (m0 == -INFINITY ? 0.f : m0);
        lift1 = kLift - (m1 == -INFINITY ? 0.f : m1);
        l0 *= c0;
        l1 *= c1;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          o[k][0] *= c0;
          o[k][1] *= c1;
          o[k][2] *= c0;
          o[k][3] *= c1;
        }
      }
      x[0] = fast_exp2(x[0] + lift0);
      x[1] = fast_exp2(x[1] + lift1);
      x[2] = fast_exp2(x[2] + lift0);
      x[3] = fast_exp2(x[3] + lift1);
      l0 += x[0] + x[2];
      l1 += x[1] + x[3];
      if (bad) l0 = l1 = NAN;  // a page outside the pool: these heads become NaN
      uint32_t r0, r1;
      uint32_t h0 = split_pair<kBf16>(x[0], x[1], &r0), h1 = split_pair<kBf16>(x[2], x[3], &r1);
      h0 = transpose8x8(h0);
      h1 = transpose8x8(h1);
      r0 = transpose8x8(r0);
      r1 = transpose8x8(r1);
      const uint32_t vstage = stage + Sh::kTileBytes;
      if constexpr (!E4M3) {
        const int vr = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          ldmatrix_x4_trans(vstage + chunk_offset<Sh::kRowBytes>(vr, 2 * k + ((lane >> 3) & 1)), a);
          mma_16x8x16<kBf16>(o[k], a[0], a[1], a[2], a[3], h0, h1);
          mma_16x8x16<kBf16>(o[k], a[0], a[1], a[2], a[3], r0, r1);
        }
      } else {
        // A transposed 16-bit unit holds two neighbouring elements of a row:
        // bytes are paired along the rows, and a lane's output rows are
        // elements 2 gr and 2 gr + 1. The scale multiplies the tile's sum
        // (and takes the lift out of it: V may be as large as fp32 holds).
        vs *= 1.f / (1 << (int)kLift);
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t a[4];
          ldmatrix_x4_trans(vstage + chunk_offset<Sh::kRowBytes>(mr, k + (lane >> 4)), a);
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = __byte_perm(a[i], 0, 0x3120);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v0 = e4m3_low(a[2 * i]), v1 = e4m3_high(a[2 * i]), v2 = e4m3_low(a[2 * i + 1]),
                           v3 = e4m3_high(a[2 * i + 1]);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_16x8x16<false>(t, v0, v1, v2, v3, h0, h1);
            mma_16x8x16<false>(t, v0, v1, v2, v3, r0, r1);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[k + i][e] = fmaf(vs, t[e], o[k + i][e]);
          }
        }
      }
    }
    turn -= here;

    // --- join the warps' states
    if constexpr (E4M3) {
      l0 *= 1.f / (1 << (int)kLift);
      l1 *= 1.f / (1 << (int)kLift);
    }
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, i);
      l1 += __shfl_xor_sync(0xffffffffu, l1, i);
    }
    if (gr == 0) {
      sm_m[warp * kHeads + 2 * tq] = m0;
      sm_m[warp * kHeads + 2 * tq + 1] = m1;
      sm_l[warp * kHeads + 2 * tq] = l0;
      sm_l[warp * kHeads + 2 * tq + 1] = l1;
    }
    {
      float* acc = merge + (warp * kHeads + 2 * tq) * D;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if constexpr (!E4M3) {
          const int d0 = merge_column<D>(2 * tq, 16 * k + gr), d1 = merge_column<D>(2 * tq, 16 * k + 8 + gr);
          acc[d0] = o[k][0];
          acc[d1] = o[k][2];
          acc[D + d0] = o[k][1];
          acc[D + d1] = o[k][3];
        } else {
          const int d0 = merge_column<D>(2 * tq, 16 * k + 2 * gr);
          *reinterpret_cast<float2*>(acc + d0) = make_float2(o[k][0], o[k][2]);
          *reinterpret_cast<float2*>(acc + D + d0) = make_float2(o[k][1], o[k][3]);
        }
      }
    }
    __syncthreads();
    if (tid < kHeads) {
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) mm = fmaxf(mm, sm_m[w * kHeads + tid]);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float mw = sm_m[w * kHeads + tid], f = mw == mm ? 1.f : fast_exp2(mw - mm);
        sm_f[w * kHeads + tid] = f;
        ll += f * sm_l[w * kHeads + tid];
      }
      sm_gm[tid] = mm;
      sm_gl[tid] = ll;
    }
    __syncthreads();
    const bool whole = here == seq.tiles;
    const int items = p.group * (D / 4);
    // shares that hold the group, this one's partial state and the group's counter
    const int64_t group_start = at - tile;
    int from = 0, parts = 1;
    float* slots = p.partials;
    const int slot_floats = cache_attn_slot_floats(p.group, D);
    if (!whole) {
      from = (int)(((group_start + 1) * ctas - 1) / total);
      parts = (int)(((group_start + seq.tiles) * ctas - 1) / total) - from + 1;
    }
    const bool leads = (int)blockIdx.x == from;
    float* slot = slots + (int64_t)(2 * blockIdx.x + (leads ? 1 : 0)) * slot_floats;
    uint8_t* out = p.out + ((int64_t)b * p.n_head + (int64_t)g * p.group) * D * 2;
    for (int i = tid; i < items; i += Sh::kThreads) {
      const int h = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float f = sm_f[w * kHeads + h];
        const float4 v = *reinterpret_cast<const float4*>(merge + (w * kHeads + h) * D + merge_column<D>(h, d));
        r.x = fmaf(f, v.x, r.x);
        r.y = fmaf(f, v.y, r.y);
        r.z = fmaf(f, v.z, r.z);
        r.w = fmaf(f, v.w, r.w);
      }
      if (whole) {
        const float inv = 1.f / sm_gl[h];
        *reinterpret_cast<uint2*>(out + i * 8) =
            make_uint2((uint32_t)Storage<T>::round(r.x * inv) | ((uint32_t)Storage<T>::round(r.y * inv) << 16),
                       (uint32_t)Storage<T>::round(r.z * inv) | ((uint32_t)Storage<T>::round(r.w * inv) << 16));
      } else {
        __stcg(reinterpret_cast<float4*>(slot + h * D + d), r);
      }
    }
    if (!whole) {
      if (tid < p.group) {
        __stcg(slot + p.group * D + tid, sm_gm[tid]);
        __stcg(slot + p.group * D + p.group + tid, sm_gl[tid]);
      }
      __threadfence();
      __syncthreads();
      unsigned int* arrived = reinterpret_cast<unsigned int*>(&words[kW + 2]);
      if (tid == 0) {
        *arrived = atomicAdd(p.counters + from, 1u);
        __threadfence();
      }
      __syncthreads();
      const unsigned int order = *arrived;
      if (order >= (unsigned int)parts) {
        // the counter was not zero before this call
        if (tid == 0 && p.err_flag) atomicOr(p.err_flag, kErrWorkspace);
        const uint32_t nan2 = (uint32_t)Storage<T>::kNaN * 0x10001u;
        for (int i = tid; i < items; i += Sh::kThreads) *reinterpret_cast<uint2*>(out + i * 8) = make_uint2(nan2, nan2);
      } else if (order == (unsigned int)parts - 1) {
        // the last to arrive: join the partial states
        auto slot_of = [&](int part) {
          return slots + (int64_t)(part ? 2 * (from + part) : 2 * from + 1) * slot_floats;
        };
        float* factor = merge;  // [parts][8]
        for (int h = warp; h < p.group; h += kW) {
          float mm = -INFINITY, ll = 0.f;
          for (int s = lane; s < parts; s += 32) mm = fmaxf(mm, __ldcg(slot_of(s) + p.group * D + h));
#pragma unroll
          for (int i = 16; i; i >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, i));
          for (int s = lane; s < parts; s += 32) {
            const float mw = __ldcg(slot_of(s) + p.group * D + h), f = mw == mm ? 1.f : fast_exp2(mw - mm);
            factor[s * kHeads + h] = f;
            ll += f * __ldcg(slot_of(s) + p.group * D + p.group + h);
          }
#pragma unroll
          for (int i = 16; i; i >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, i);
          if (lane == 0) sm_gl[h] = ll;
        }
        __syncthreads();
        for (int i = tid; i < items; i += Sh::kThreads) {
          const int h = i / (D / 4);
          float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int s = 0; s < parts; ++s) {
            const float f = factor[s * kHeads + h];
            const float4 v = __ldcg(reinterpret_cast<const float4*>(slot_of(s) + i * 4));
            r.x = fmaf(f, v.x, r.x);
            r.y = fmaf(f, v.y, r.y);
            r.z = fmaf(f, v.z, r.z);
            r.w = fmaf(f, v.w, r.w);
          }
          const float inv = 1.f / sm_gl[h];
          *reinterpret_cast<uint2*>(out + i * 8) =
              make_uint2((uint32_t)Storage<T>::round(r.x * inv) | ((uint32_t)Storage<T>::round(r.y * inv) << 16),
                         (uint32_t)Storage<T>::round(r.z * inv) | ((uint32_t)Storage<T>::round(r.w * inv) << 16));
        }
        if (tid == 0) p.counters[from] = 0;  // ready for the next call
      }
    }
    __syncthreads();  // the merge buffer is free

    // --- the next group
    at += here;
    tile = 0;
    if (at < hi && ++g == p.n_kv_head) {
      g = 0;
      do ++b;
      while (tiles_of(p, p.kv_len[b], &seq) <= 0);
    }
  }
  copy_wait<0>();
}

template <typename T, bool E4M3, int D>
cudaError_t launch_cache_attn_t(const CacheAttnParams& p, int sms, cudaStream_t stream) {
  using Sh = CacheAttnShape<E4M3, D>;
  auto* fn = cache_attn_kernel<T, E4M3, D>;
  static std::atomic<bool> ready[64];  // per device: the shared-memory opt-in is applied
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (!ready[device].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
    if (e != cudaSuccess) return e;
    ready[device].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cache_attn_ctas(sms));
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

template <typename T>
cudaError_t launch_cache_attn_type(const CacheAttnParams& p, int head_dim, bool e4m3, int sms, cudaStream_t stream) {
  if (head_dim == 128)
    return e4m3 ? launch_cache_attn_t<T, true, 128>(p, sms, stream) : launch_cache_attn_t<T, false, 128>(p, sms, stream);
  return e4m3 ? launch_cache_attn_t<T, true, 64>(p, sms, stream) : launch_cache_attn_t<T, false, 64>(p, sms, stream);
}

}  // namespace da
