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
// Work split. The visible rows of a group (b, g) are cut into tiles that start
// at multiples of 16 or 32 rows, in pieces of 16 rows that never cross a page
// (of at least 16), and the tiles of all groups form one list in (b, g, row)
// order. CTA i of n owns an even share of the list, whatever the lengths, the
// window or the batch are: every CTA computes the list from kv_len itself, so
// the launch does not depend on lengths and ragged batches are balanced to a
// tile (groups of about one length get the same number of CTAs each instead,
// so that fewer parts are joined). A group that lies in several shares is joined
// through the workspace by the last CTA to arrive; nothing waits for another CTA.
//
// A warp takes every kWarps-th tile of the share, with a ring of its own in
// shared memory that asynchronous copies keep filled (page numbers are looked
// up one tile ahead, over the ends of groups), and no barrier within a group.
// Per tile and piece:
//   S^T [16 rows x 8 heads] = K q^T        mma m16n8k16, K by ldmatrix
//   p = 2^(x' - m), m raised only when a score passes it by some bits (a vote)
//   out^T [D x 8 heads] += V^T P^T         V by ldmatrix.trans, P^T by movmatrix
// The heads are the 8 columns of the instruction, so a group of 1, 2, 4 or 8
// costs the same, and scores and weights stay in registers. (For tcgen05 a
// tile of one query token is too small: its 128-row operand would hold 8
// pieces of different pages, and its accumulator would have to come back from
// tensor memory for every softmax; here the tensor pipe is busy 11 to 25% of
// the time.) Weights are split in 16-bit pieces, each multiplied with V: three
// of bf16, which hold all 24 bits of a float (two hold 16; then 0.21% of the
// bf16 outputs of 8 ragged to 8191 differed from the rounded exact ones, for
// 0.05% with three or in a plain fp32 form), or two of fp16, which hold 22. The
// third costs bf16 caches 0 to 4% (64 ragged to 400 14.4 -> 14.9 us, 8 ragged to
// 8191 29.9 -> 30.2). A tile's product starts from zero and is added to the
// output in fp32: the matrix instruction truncates its sums, and 200 tiles on
// one accumulator drift towards zero (32 ragged to 32768: 0.31% of the outputs
// differed, now 0.02%; 0 to 0.1 us). e4m3 is converted to fp16 (exact) on its way
// from shared memory to the matrix instruction; the scales multiply scores and
// sums.
//
// Measured (graph of calls, data from HBM, of the measured 6782 GB/s copy): 32
// ragged sequences up to 32768 rows, 32 / 8 heads, 2.04 GB in 297 us (101%),
// in 8 bits 1.02 GB in 153 us (98%); 8 ragged up to 8191, 16 / 8 heads, 159 MB
// in 30.2 us (78%); 16 ragged with window 1021 and 16 / 8 heads, 68 MB in 13.0
// us (77%); window 4096 in 8 bits, 16 ragged, 64 / 8 heads, 135 MB in 26.3 us
// (76%); one of 1024 rows, 16 / 16 heads, 7.0 us. Short calls are a chain of
// dependent steps, each about as long as a memory round trip: page numbers (0.6
// us after the wait; lengths, share and L2 prefetch come before it), rows (0.8),
// the tile, the join of the warps (0.7), arrival (1.0) and the join of the parts
// (1.5).
#pragma once

#include <atomic>

#include "cache_params.h"
#include "common.cuh"

namespace da {

constexpr int kHeads = 8;        // columns of the matrix instruction
constexpr int kMaxCtas = 256;    // one for each SM; parts of one group, at most
// The split, in tiles; each was swept on the device (with ragged lengths from an
// eighth of the longest on, as lengths() of perf/operators.py draws them for lens
// = 1; figures of bf16 caches from before their weights' third piece, which added
// 0 to 5% with the rounded sums). A share of kFewestTiles (as
// the only rule for short batches: 4 ragged to 200 rows of 32/8 heads 4.2 us, with 4
// 5.9, with 16 9.0; 1 x 1024 of 16/16 6.7, 7.2, 7.5). The end of a group costs
// kGroupCost, that of one in parts kJoinCost: without the latter 8 ragged to 8191
// take 32.4 us for 29.2. With as many CTAs for every group a share saves kEvenGain,
// and kAloneGain where there is then nothing to join; its tiles take 7/8 of the
// time, as fewer SMs share HBM. 16 x 8192 of 16/8 heads: 81.7 us even, 85.3 not;
// 12 ragged to 2000, e4m3: 13.8 and 15.1; but 5 ragged to 3000: 13.4 and 12.7.
constexpr int kFewestTiles = 8, kGroupCost = 8, kJoinCost = 16, kEvenGain = 12, kAloneGain = 48;
// A group in more than kJoinWide parts (at most 256) is joined in two rounds, of
// kJoinWidth neighbours and of the sums of those.
constexpr int kJoinWide = 64, kJoinWidth = 16;
// With more groups than CTAs, teams of 1, 2 or 4 warps may take whole groups: no
// barrier of the CTA, nothing to join. The cost of either way is counted in tiles
// a warp goes through, a group's end as one and an even share's joins as kTeamGain.
// us in teams / in even shares, 8 KV heads: 256 ragged to 128 rows 19.2 / 42.7, 64 to
// 400 14.4 / 19.9, 24 to 300 8.1 / 10.5, e4m3 64 to 800 20.9 / 24.9. With 3 for 6 the
// last three stay in even shares; with 10, e4m3 40 to 2000 of 64 goes in teams and
// takes 23.0 for 20.8.
constexpr int kTeamGain = 6;
// m is raised when a score passes it by kLazy (log2). bf16 weights have fp32's
// range. fp16 weights are 2^13 2^(x' - m): at most 2^15, inside the type's range,
// and what lies above 2^-38 of the largest one is held, so that the weights of
// 16k rows together lose less than one fp32 rounding of it (with 8 and 2^7, 2^-32,
// at the same time; with 1 and 2^14 8-bit caches take 0.5% longer). They are
// scaled after the exponential: added to x' - m, 13 would round its last bits
// away (twice as many outputs differ from the exact ones; 8-bit caches save 0.3%).
constexpr float kLazyBf16 = 8.f, kLazyF16 = 2.f, kLiftF16 = 8192.f;

template <bool E4M3, int D>
struct CacheAttnShape {
  static constexpr int kWarps = E4M3 && D == 64 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kRows = kRowBytes > 128 ? 16 : 32;  // of a tile, in pieces of 16
  static constexpr int kTileBytes = kRows * kRowBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K tile, V tile
  // Tiles of a warp that take as long as a join: 1 x 300 of 16/8 heads 4.9 us with
  // 2 or 3 (no join), 5.9 with 1; 3 ragged to 1000, 16/4 heads of 64, 5.6 with 3, 6.0
  // with 2; 1 x 700 in e4m3, 32/8 heads, whose tiles take longer, 6.6 with 1, 6.8 with 2.
  static constexpr int kJoinTurns = E4M3 ? 1 : 3;
  static constexpr int kStages = 196608 / (kWarps * kStageBytes);
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeFloats = kWarps * kHeads * D;
  static constexpr int kMergeBytes = kMergeFloats * 4;
  static constexpr int kMetaOffset = kRingBytes + kMergeBytes;
  static constexpr int kMetaBytes = 32;  // of a stage: K and V scale of each piece, bad pages, visible rows
  static constexpr int kStatOffset = kMetaOffset + kWarps * kStages * kMetaBytes;
  // (m, l) of each warp, and of joined parts; schedule words
  static constexpr int kStatFloats = 2 * kWarps * kHeads + 2 * kHeads;
  static constexpr int kWordsOffset = kStatOffset + kStatFloats * 4;
  static constexpr int kSmemBytes = kWordsOffset + (2 * kWarps + 4 + (kWarps + 1) / 2) * 8;
  static_assert(kStages >= 3, "a ring of at least three stages");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
  static_assert(kJoinWide * kHeads * 4 + kThreads * 16 <= kMergeBytes,
                "the join's factors and sums fit the merge buffer");
  static_assert(kMaxCtas <= kJoinWidth * kJoinWidth && kJoinWide <= 64 && 3 * kMaxCtas <= kMaxCounterGroups,
                "two rounds of parts that a warp holds; a counter for each CTA and round");
  static_assert(kHeads * (D / 4) <= kThreads && kHeads <= kWarps,
                "a thread for each output vector, a warp for each head");
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

// a and b as sums of PIECES 16-bit numbers each, packed: each piece is what the
// ones before leave, rounded to nearest. Three bf16 pieces hold all 24 bits of a
// float (8, 8 and 8), two fp16 pieces 22.
template <bool BF16, int PIECES>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&piece)[PIECES]) {
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    float2 f;
    if constexpr (BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      piece[i] = *reinterpret_cast<const uint32_t*>(&h);
      f = __bfloat1622float2(h);
    } else {
      const __half2 h = __floats2half2_rn(a, b);
      piece[i] = *reinterpret_cast<const uint32_t*>(&h);
      f = __half22float2(h);
    }
    a -= f.x;
    b -= f.y;
  }
}

// Tiles of one sequence: visible rows [0, s0) and [w0, len). Tile i < sink_tiles
// starts at row ROWS i; the others follow from row ROWS first_tile on.
struct SequenceTiles {
  int len, w0, s0, sink_tiles, first_tile, tiles;
};

// Number of tiles (0: no visible row), or -1 for a length out of range.
template <int ROWS>
__device__ __forceinline__ int tiles_of(const CacheAttnParams& p, int len, SequenceTiles* s) {
  s->tiles = 0;
  if (len < 0 || len > p.max_len) return -1;
  s->len = len;
  s->w0 = (p.window > 0 && len > p.window) ? len - p.window : 0;
  s->s0 = min(p.sinks, s->w0);
  s->first_tile = s->w0 / ROWS;
  // a sink tile that the window reaches into belongs to the window's tiles
  s->sink_tiles = min((s->s0 + ROWS - 1) / ROWS, s->first_tile);
  if (len > 0) s->tiles = s->sink_tiles + (len + ROWS - 1) / ROWS - s->first_tile;
  return s->tiles;
}

template <int ROWS>
__device__ __forceinline__ int tile_row(const SequenceTiles& s, int i) {
  return (i < s.sink_tiles ? i : i - s.sink_tiles + s.first_tile) * ROWS;
}

// Bit r: row row0 + r is visible (some row of a tile of the list is).
template <int ROWS>
__device__ __forceinline__ uint32_t tile_mask(const SequenceTiles& s, int row0) {
  constexpr uint32_t kFull = 0xffffffffu >> (32 - ROWS);
  const int end = min(s.len - row0, ROWS);
  uint32_t mask = kFull >> (ROWS - end);
  if (row0 < s.w0) {
    const int lo = max(s.s0 - row0, 0), hi = min(s.w0 - row0, ROWS);
    if (hi > lo) mask &= ~((kFull >> (ROWS - (hi - lo))) << lo);
  }
  return mask;
}

// Counts this CTA in and returns how many were before it: its writes ahead of
// the last barrier are visible to whoever counts later, and theirs to it.
__device__ __forceinline__ unsigned int arrive(unsigned int* counter) {
  unsigned int n;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
  return n;
}

// (out of line: a 64-bit division is some hundred instructions)
static __device__ __noinline__ int64_t divide(int64_t a, int64_t b) { return a / b; }

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(CacheAttnShape<E4M3, D>::kThreads, 1) cache_attn_kernel(const CacheAttnParams p) {
  using Sh = CacheAttnShape<E4M3, D>;
  constexpr bool kBf16 = !E4M3 && Storage<T>::kBf16;  // type of the matrix operands
  constexpr float kLift = kBf16 ? 1.f : kLiftF16, kLazy = kBf16 ? kLazyBf16 : kLazyF16;
  constexpr int kPieces = kBf16 ? 3 : 2;  // of a weight
  constexpr int kW = Sh::kWarps, kS = Sh::kStages, kSteps = D / 16, kRows = Sh::kRows, kHalves = kRows / 16;
  constexpr uint32_t kFull = 0xffffffffu >> (32 - kRows);
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + Sh::kRingBytes);
  float* sm_m = reinterpret_cast<float*>(smem + Sh::kStatOffset);  // [kW][8]
  float* sm_l = sm_m + kW * kHeads;
  float* sm_gl = sm_l + kW * kHeads;  // l and m of joined parts
  float* sm_gm = sm_gl + kHeads;
  int64_t* words = reinterpret_cast<int64_t*>(smem + Sh::kWordsOffset);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gr = lane >> 2, tq = lane & 3;

  // --- the list of places, and this CTA's share [lo, hi) of it: the tiles of
  // each group, and some places that stand for its end (groups are then
  // balanced by what they cost, and those places hold cuts that would split a
  // group); or, with groups about equal, as many places for each, so that the
  // cuts fall between them. One pass over the lengths, and, for more sequences
  // than threads, a second one for the sequence that holds `lo`. A batch of at
  // most 32, and of no more groups than CTAs, is seen by each warp alone, without
  // a barrier.
  // Where one pass will do it is made while the kernel before this one still
  // runs: the lengths of then say which rows to bring into L2 (a hint; page
  // numbers are checked), and if they are still those after the wait, the share
  // stands.
  struct Found {
    int64_t start;  // first place of the sequence
    int b, len;
  };
  Found* found = reinterpret_cast<Found*>(words + kW);
  constexpr int kCount = 44;  // tiles and non-empty sequences are summed in one word: tiles + sequences * 2^44
  static_assert(kMaxBatch < 1 << (63 - kCount) && (int64_t)kMaxBatch << 27 <= 1ll << kCount,
                "a batch of sequences of fewer than 2^31 rows, in tiles of 16, fits the word");
  constexpr int kChunks = Sh::kRowBytes / 16, kLanes = 32 / kHalves, kCopies = 16 * kChunks / kLanes;
  const int half = kHalves == 2 ? lane >> 4 : 0, sub = lane % kLanes;
  const bool alone = p.B <= 32 && p.B * p.n_kv_head <= gridDim.x;  // (teams have to agree on the split)
  const int column = alone ? lane : tid, columns = alone ? 32 : Sh::kThreads;
  int64_t before = 0, mine = 0, own = 0;  // before this pass, before this thread's sequence, and its own
  int len = 0, most = 0;                  // most tiles of a sequence
  int* tops = reinterpret_cast<int*>(words + kW + 4);  // [kW]
  auto pass = [&](int base) {
    const int b = base + column;
    int n = 0;
    if (b < p.B) {
      SequenceTiles s;
      len = __ldcg(p.kv_len + b);  // (L2: read before the wait, it may be read again)
      n = max(tiles_of<kRows>(p, len, &s), 0);
    }
    own = n ? n + (1ll << kCount) : 0;
    const int top = __reduce_max_sync(0xffffffffu, n);
    int64_t sum = own;
#pragma unroll 1
    for (int o = 1; o < (alone ? p.B : 32); o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    mine = before + sum - own;
    if (alone) {
      before = __shfl_sync(0xffffffffu, sum, p.B - 1);
      most = top;
      return;
    }
    if (base) __syncthreads();  // the words of the pass before have been read
    if (lane == 31) {
      words[warp] = sum;
      tops[warp] = top;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) mine += words[w];
      before += words[w];
      most = max(most, tops[w]);
    }
  };
  // Sequences without a visible row get zeros, those without a valid length NaN.
  auto fill_idle = [&](int base) {
    const int b = base + column;
    const bool bad = len < 0 || len > p.max_len;
    unsigned todo = __ballot_sync(0xffffffffu, b < p.B && (bad || len == 0) && b % gridDim.x == blockIdx.x);
    if (alone && warp) todo = 0;
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t row = __shfl_sync(0xffffffffu, b, src);
      const uint32_t fill = __shfl_sync(0xffffffffu, bad ? (uint32_t)Storage<T>::kNaN * 0x10001u : 0u, src);
      if (fill && lane == 0 && p.err_flag) atomicOr(p.err_flag, kErrKvLen);
      uint4* out = reinterpret_cast<uint4*>(p.out) + row * p.n_head * (D / 8);
#pragma unroll 1
      for (int i = lane; i < p.n_head * (D / 8); i += 32) out[i] = make_uint4(fill, fill, fill, fill);
    }
  };
  int64_t ctas = 0, total = 0, lo = 0, hi = 0;
  int end_cost = 0, even = 0;  // places behind a group's tiles; with even groups, places of every group
  bool small = true;
  auto places = [&](int64_t word) {
    const int64_t n = word >> kCount;
    return (even ? n * even : (word & ((1ll << kCount) - 1)) + n * end_cost) * p.n_kv_head;
  };
  auto behind = [&](const SequenceTiles& s) { return even ? even - s.tiles : end_cost; };
  // first place of share i, and the share that holds place x (in 32 bits where
  // they suffice: a 64-bit division is some hundred instructions)
  auto share_start = [&](int64_t i) {
    return small ? (int64_t)((uint32_t)i * (uint32_t)total / (uint32_t)ctas) : divide(i * total, ctas);
  };
  auto share_of = [&](int64_t x) {
    return (int)(small ? ((uint32_t)(x + 1) * (uint32_t)ctas - 1) / (uint32_t)total
                       : divide((x + 1) * ctas - 1, total));
  };
  SequenceTiles seq;  // the sequence that holds `lo`
  int b = 0, g = 0, tile = 0;  // group of list position `lo`, and its place there
  bool strided = false;  // groups are taken whole, by teams of warps
  int team = kW;         // warps that share a group,
  int lead = warp;       // and those of them before this one
  int hop = 1;           // groups from one of a team to its next one
  const bool one_pass = p.B <= Sh::kThreads;
  bool waited = !one_pass;
  // From (b, g) on to the first group with rows, in steps of the list (strided:
  // of the teams); false when there is none. (After the wait only.)
  auto settle = [&](int& b, int& g, SequenceTiles& s) {
#pragma unroll 1
    while (b < p.B && tiles_of<kRows>(p, p.kv_len[b], &s) <= 0) {
      if (strided) g += hop;
      b += strided ? g / p.n_kv_head : 1;
      g = strided ? g % p.n_kv_head : 0;
    }
    return b < p.B;
  };
  if (waited) {
    pdl_wait();
    pdl_trigger();  // the next grid can take the SMs as they fall free; it waits for this one's memory
  }
  for (;;) {
    before = lo = 0;
    most = 0;
    strided = false;
    team = kW;
    lead = warp;
    hop = 1;
    for (int base = 0; base < p.B; base += columns) {
      pass(base);
      if (!one_pass) fill_idle(base);
    }
    const int64_t tiles = (before & ((1ll << kCount) - 1)) * p.n_kv_head, groups = (before >> kCount) * p.n_kv_head;
    even = 0;
    if (groups > gridDim.x) {
      // whole groups, by teams of 1, 2 or 4 warps, where the longest way through
      // them is no longer than an even share with its ends and joins (in floats:
      // an estimate, and a 64-bit division is some hundred instructions)
      const float each = 1.f / (float)(gridDim.x * kW);
      float least = (float)tiles * each + (float)groups * each * kW + kTeamGain;
#pragma unroll
      for (int t = 1; t <= 4; t *= 2) {
        const float cost = ceilf(((float)groups - 0.5f) * each * t) * (float)((uint32_t)(most + t - 1) / t + 1);
        if (cost <= least) {
          least = cost;
          strided = true;
          team = t;
          lead = warp % t;
          hop = kW / t * gridDim.x;
          g = warp / t * gridDim.x + blockIdx.x;
        }
      }
      if (strided) {
        ctas = gridDim.x;
        b = g / p.n_kv_head;
        g -= b * p.n_kv_head;
        tiles_of<kRows>(p, b < p.B ? __ldcg(p.kv_len + b) : 0, &seq);  // (for the prefetch; settled after the wait)
        tile = 0;
        hi = INT32_MAX;
        end_cost = 0;
      }
    }
    // as many CTAs as find kFewestTiles
    if (!strided) {
      ctas = min((int64_t)gridDim.x, (tiles + kFewestTiles - 1) / kFewestTiles);
      end_cost = kGroupCost;
      if (groups <= gridDim.x && groups > 0) {
        // As many CTAs for every group: one where a warp then has at most
        // kJoinTurns tiles more than with all CTAs, or else as few as leave it no
        // more tiles. Taken where the largest part then takes no
        // longer than an even share of all tiles with the ends of groups in it.
        const uint32_t n = (uint32_t)ctas, fit = gridDim.x / (uint32_t)groups;
        const uint32_t turns = ((uint32_t)most + kW * fit - 1) / (kW * fit);
        const uint32_t each = (uint32_t)most <= kW * (turns + Sh::kJoinTurns)
                                  ? 1 : ((uint32_t)most + kW * turns - 1) / (kW * turns);
        const int64_t part = ((uint32_t)most + each - 1) / each;
        if (part * n * 7 <= (tiles + n * (each == 1 ? kAloneGain : kEvenGain)) * 8) {
          ctas = each * groups;
          even = (int)(part * each);
        } else if (groups <= n) {
          end_cost = tiles >= ctas * kJoinCost * 8 ? kJoinCost : (int)((uint32_t)tiles / n / 8);
        }
      }
    }
    if (!strided && (int64_t)blockIdx.x < ctas) {
      total = places(before);
      small = total * ctas < (1ll << 32);
      lo = share_start(blockIdx.x);
      hi = share_start(blockIdx.x + 1);
      Found first;
      auto holds = [&]() {
        const int64_t at = places(mine);
        return at <= lo && lo < at + places(own);
      };
      if (alone) {
        const int src = __ffs(__ballot_sync(0xffffffffu, holds())) - 1;
        first = {__shfl_sync(0xffffffffu, places(mine), src), src, __shfl_sync(0xffffffffu, len, src)};
      } else {
        if (one_pass) {
          if (holds()) *found = {places(mine), tid, len};
        } else {
          before = 0;
          for (int base = 0; places(before) <= lo; base += Sh::kThreads) {
            __syncthreads();
            pass(base);
            if (holds()) *found = {places(mine), base + tid, len};
          }
        }
        __syncthreads();
        first = *found;
      }
      b = first.b;
      tiles_of<kRows>(p, first.len, &seq);
      const int64_t in = lo - first.start;
      const int size = seq.tiles + behind(seq);
      g = small ? (int)((uint32_t)in / (uint32_t)size) : (int)divide(in, size);
      tile = (int)(in - (int64_t)g * size);
    }
    if (waited) break;
    if ((int64_t)blockIdx.x < ctas) {
#pragma unroll 1
      for (int i = tile + lead, j = 0; j < kS - 1 && i < seq.tiles && i - tile < hi - lo; i += team, ++j) {
        const int row = tile_row<kRows>(seq, i) + 16 * half;
        if (row + 16 > seq.len) break;
        const int page = p.table ? __ldcg(p.table + (int64_t)b * p.max_pages + (row >> p.page_shift)) : b;
        if (page < 0 || page >= p.num_pages || sub > 1) continue;
        const int64_t from =
            ((int64_t)page * p.n_kv_head + g) * p.page_rows + (row & (p.table ? p.page_rows - 1 : -1));
        prefetch_l2((sub ? p.v : p.k) + from * Sh::kRowBytes, 16 * Sh::kRowBytes);
      }
    }
    pdl_wait();
    pdl_trigger();
    waited = true;
    const bool same = column >= p.B || __ldcg(p.kv_len + column) == len;
    if (alone ? __all_sync(0xffffffffu, same) : __syncthreads_and(same)) break;
  }
  if (one_pass) fill_idle(0);
  if ((int64_t)blockIdx.x >= ctas) return;
  // A team goes where its first warp goes: its barriers count its warps, and a
  // length that changes under the call (an error of the caller's) must not part
  // them. (b, g and the length in one word; all ones, which no group is, at the
  // end.)
  static_assert(kMaxBatch <= 0xffff, "b < B and g < n_kv_head are below 0xffff");
  uint64_t* next = reinterpret_cast<uint64_t*>(words + kW + 4 + (kW + 1) / 2) + (warp - lead);
  auto team_sync = [&]() {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (warp - lead) / 2), "r"(team * 32) : "memory");
  };
  auto send = [&](bool any) {
    if (lane == 0) *next = any ? (uint64_t)b << 48 | (uint64_t)g << 32 | (uint32_t)seq.len : ~0ull;
  };
  auto receive = [&]() {  // (after a barrier of the team)
    const uint64_t word = *next;
    b = (int)(word >> 48);
    g = (int)(word >> 32) & 0xffff;
    tiles_of<kRows>(p, (int)(uint32_t)word, &seq);
    return word != ~0ull;
  };
  if (strided) {
    bool any = lead == 0 && settle(b, g, seq);
    if (team > 1) {
      if (lead == 0) send(any);
      team_sync();
      any = receive();
    }
    if (!any) return;
  }
  const int step = team;             // tiles between this warp's
  const int share = (int)(hi - lo);  // (below 2^31: checked on the host)
  int at = 0;                        // place in the share of the next tile to compute
  // the next group of this CTA (strided, of this team); false when
  // the share ends before it
  auto next_group = [&](int place, int& b, int& g, SequenceTiles& s) {
    if (place >= share) return false;
    g += hop;
    if (g < p.n_kv_head) return true;
    b += strided ? g / p.n_kv_head : 1;
    g = strided ? g % p.n_kv_head : 0;
    return settle(b, g, s);
  };
  if (tile >= seq.tiles) {
    // the share begins in the places of a group's end
    at += seq.tiles + behind(seq) - tile;
    tile = 0;
    if (!next_group(at, b, g, seq)) return;
  }

  // --- this warp's loads. A tile is kHalves pieces of 16 rows, each inside one
  // page; with two, either half of the warp looks up and copies its own.
  const uint32_t ring = smem_addr(smem) + warp * kS * Sh::kStageBytes;
  const uint32_t meta = smem_addr(smem + Sh::kMetaOffset) + warp * kS * Sh::kMetaBytes;
  // a group's q, on its way to L1 when the first of its tiles is looked up
  auto prefetch_q = [&](int b, int g) {
    const int bytes = p.group * D * 2;
    if (lane * 128 < bytes)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + ((int64_t)b * p.n_head + g * p.group) * D * 2 + lane * 128));
  };
  SequenceTiles lseq = seq;  // the tile to load next, its page number on the way
  int lb = b, lg = g, li = tile, lrow = 0, lpage = 0;
  uint32_t lmask = 0;  // 0: no tile is left
  int lat = at;
  bool more = true;
  auto look_up = [&](int step) {  // moves on by `step` tiles
    lat += step;
    li += step;
    lmask = 0;
    while (more && li >= lseq.tiles) {
      li -= lseq.tiles;
      lat += behind(lseq);
      more = next_group(lat - li, lb, lg, lseq);
      if (more) prefetch_q(lb, lg);
    }
    more = more && lat < share;
    if (!more) return;
    const int row0 = tile_row<kRows>(lseq, li);
    lmask = tile_mask<kRows>(lseq, row0);
    lrow = row0 + 16 * half;
    if (p.table) {
      // (a piece with no visible row may lie past the table)
      lpage = (kHalves == 1 || ((lmask >> (16 * half)) & 0xffffu))
                  ? p.table[(int64_t)lb * p.max_pages + (lrow >> p.page_shift)] : 0;
    } else {
      lpage = lb;
    }
  };
  auto issue = [&](int stage, int row, int page, uint32_t mask, int head) {
    const bool bad = page < 0 || page >= p.num_pages;
    if (bad) page = 0;
    const int64_t block = (int64_t)page * p.n_kv_head + head;
    const int64_t at = (block * p.page_rows + (row & (p.table ? p.page_rows - 1 : -1))) * Sh::kRowBytes + sub * 16;
    const uint8_t* ksrc = p.k + at;
    const uint8_t* vsrc = p.v + at;
    const uint32_t dst = ring + stage * Sh::kStageBytes + half * 16 * Sh::kRowBytes;
    const uint32_t rows = bad ? 0u : (mask >> (16 * half)) & 0xffffu;
    if (__all_sync(0xffffffffu, rows == 0xffffu)) {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int x = sub + kLanes * j;
        const uint32_t d = dst + chunk_offset<Sh::kRowBytes>(x / kChunks, x % kChunks);
        copy16(d, ksrc + kLanes * j * 16);
        copy16(d + Sh::kTileBytes, vsrc + kLanes * j * 16);
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < kCopies; ++j) {
        const int x = sub + kLanes * j, r = x / kChunks;
        const bool on = (rows >> r) & 1;
        const uint32_t d = dst + chunk_offset<Sh::kRowBytes>(r, x % kChunks);
        copy16_or_zero(d, on ? ksrc + kLanes * j * 16 : p.k, on ? 16 : 0);
        copy16_or_zero(d + Sh::kTileBytes, on ? vsrc + kLanes * j * 16 : p.v, on ? 16 : 0);
      }
    }
    const uint32_t m = meta + stage * Sh::kMetaBytes;
    if constexpr (E4M3) {
      // (the scales of a piece without rows are zeros)
      if (sub < 2) copy4_or_zero(m + half * 8 + sub * 4, (sub ? p.v_scale : p.k_scale) + block, rows ? 4 : 0);
    }
    if (sub == 2) asm volatile("st.shared.u32 [%0], %1;" ::"r"(m + 16 + half * 4), "r"((uint32_t)bad) : "memory");
    if (lane == 3) asm volatile("st.shared.u32 [%0], %1;" ::"r"(m + 24), "r"(mask) : "memory");
    if (bad && sub == 0 && p.err_flag) atomicOr(p.err_flag, kErrPage);
  };
  int put = 0;  // stage that the next load goes to
  auto load_next = [&]() {
    if (lmask) {
      issue(put, lrow, lpage, lmask, lg);
      look_up(step);
    }
    copy_commit();
    put = put + 1 == kS ? 0 : put + 1;
  };
  look_up(lead);
#pragma unroll 1
  for (int j = 0; j < kS - 1; ++j) load_next();

  // --- group by group
  int get = 0;      // stage of this warp's next tile
  int turn = lead;  // tiles until this warp's next one
  for (;;) {
    const int here = min(seq.tiles - tile, share - at);  // tiles of the group in this share
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
    float o[kSteps][4], m0 = -INFINITY, m1 = -INFINITY, base0 = 0.f, base1 = 0.f, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;

    for (; turn < here; turn += step) {
      copy_wait<kS - 2>();
      __syncwarp();
      // refill the stage that the tile before this one has left
      load_next();
      const uint32_t stage = ring + get * Sh::kStageBytes, m = meta + get * Sh::kMetaBytes;
      get = get + 1 == kS ? 0 : get + 1;
      uint32_t bad[2], mask;
      float scales[4];  // K and V of either piece
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(bad[0]), "=r"(bad[1]) : "r"(m + 16));
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(m + 24));
      if constexpr (E4M3)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(scales[0]), "=f"(scales[1]), "=f"(scales[2]), "=f"(scales[3])
                     : "r"(m));

      // scores: rows gr and gr + 8 of each piece, heads 2 tq and 2 tq + 1
      float x[kHalves][4];
      const int mr = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int i = 0; i < kHalves; ++i) {
        const uint32_t kst = stage + i * 16 * Sh::kRowBytes;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        if constexpr (!E4M3) {
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            uint32_t a[4];
            ldmatrix_x4(kst + chunk_offset<Sh::kRowBytes>(mr, 2 * k + (lane >> 4)), a);
            mma_16x8x16<kBf16>(k & 1 ? s2 : s, a[0], a[1], a[2], a[3], qb[k][0], qb[k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            uint32_t a[4];
            ldmatrix_x4(kst + chunk_offset<Sh::kRowBytes>(mr, k + (lane >> 4)), a);
            mma_16x8x16<false>(s, e4m3_low(a[0]), e4m3_low(a[1]), e4m3_high(a[0]), e4m3_high(a[1]), qb[k][0],
                               qb[k][1]);
            mma_16x8x16<false>(s2, e4m3_low(a[2]), e4m3_low(a[3]), e4m3_high(a[2]), e4m3_high(a[3]), qb[k + 1][0],
                               qb[k + 1][1]);
          }
        }
        const float f0 = E4M3 ? scale0 * scales[2 * i] : scale0, f1 = E4M3 ? scale1 * scales[2 * i] : scale1;
        x[i][0] = (s[0] + s2[0]) * f0;
        x[i][1] = (s[1] + s2[1]) * f1;
        x[i][2] = (s[2] + s2[2]) * f0;
        x[i][3] = (s[3] + s2[3]) * f1;
      }
      if (mask != kFull) {
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          if (!((mask >> (16 * i + gr)) & 1)) x[i][0] = x[i][1] = -INFINITY;
          if (!((mask >> (16 * i + gr + 8)) & 1)) x[i][2] = x[i][3] = -INFINITY;
        }
      }
      float a0 = fmaxf(x[0][0], x[0][2]), a1 = fmaxf(x[0][1], x[0][3]);
      if constexpr (kHalves == 2) {
        a0 = fmaxf(a0, fmaxf(x[1][0], x[1][2]));
        a1 = fmaxf(a1, fmaxf(x[1][1], x[1][3]));
      }
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
        base0 = m0 == -INFINITY ? 0.f : m0;
        base1 = m1 == -INFINITY ? 0.f : m1;
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
      uint32_t pw[kHalves][2][kPieces];  // weights as the right operand, in pieces
#pragma unroll
      for (int i = 0; i < kHalves; ++i) {
        x[i][0] = fast_exp2(x[i][0] - base0) * kLift;
        x[i][1] = fast_exp2(x[i][1] - base1) * kLift;
        x[i][2] = fast_exp2(x[i][2] - base0) * kLift;
        x[i][3] = fast_exp2(x[i][3] - base1) * kLift;
        l0 += x[i][0] + x[i][2];
        l1 += x[i][1] + x[i][3];
        if (bad[i]) l0 = l1 = NAN;  // a page outside the pool: these heads become NaN
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          split_pair<kBf16>(x[i][2 * e], x[i][2 * e + 1], pw[i][e]);
#pragma unroll
          for (int n = 0; n < kPieces; ++n) pw[i][e][n] = transpose8x8(pw[i][e][n]);
        }
      }
      const uint32_t vst = stage + Sh::kTileBytes;
      if constexpr (!E4M3) {
        const int vr = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kHalves; ++i) {
            uint32_t a[4];
            ldmatrix_x4_trans(vst + i * 16 * Sh::kRowBytes + chunk_offset<Sh::kRowBytes>(vr, 2 * k + ((lane >> 3) & 1)),
                              a);
#pragma unroll
            for (int n = 0; n < kPieces; ++n)
              mma_16x8x16<kBf16>(t, a[0], a[1], a[2], a[3], pw[i][0][n], pw[i][1][n]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] += t[e];
        }
      } else {
        // A transposed 16-bit unit holds two neighbouring elements of a row:
        // bytes are paired along the rows, and a lane's output rows are
        // elements 2 gr and 2 gr + 1. The scale multiplies the sum of the
        // pieces that share it (and takes the lift out of it: V may be as large
        // as fp32 holds).
        const float vs0 = scales[1] * (1.f / kLift), vs1 = scales[3] * (1.f / kLift);
        const bool apart = vs0 != vs1;
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          float t[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[4];
            ldmatrix_x4_trans(vst + i * 16 * Sh::kRowBytes + chunk_offset<Sh::kRowBytes>(mr, k + (lane >> 4)), a);
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = __byte_perm(a[e], 0, 0x3120);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t v0 = e4m3_low(a[2 * n]), v1 = e4m3_high(a[2 * n]), v2 = e4m3_low(a[2 * n + 1]),
                             v3 = e4m3_high(a[2 * n + 1]);
#pragma unroll
              for (int w = 0; w < kPieces; ++w)
                mma_16x8x16<false>(t[n], v0, v1, v2, v3, pw[i][0][w], pw[i][1][w]);
            }
            if (i == 1 || apart) {
              const float vs = i ? vs1 : vs0;
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  o[k + n][e] = fmaf(vs, t[n][e], o[k + n][e]);
                  if (i == 0) t[n][e] = 0.f;
                }
            }
          }
        }
      }
    }
    turn -= here;

    // --- join the warps' states
    if constexpr (E4M3) {
      l0 *= 1.f / kLift;
      l1 *= 1.f / kLift;
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
    uint8_t* out = p.out + ((int64_t)b * p.n_head + (int64_t)g * p.group) * D * 2;
    auto store = [&](int i, const float4& r, float l) {
      const float inv = 1.f / l;
      *reinterpret_cast<uint2*>(out + i * 8) =
          make_uint2((uint32_t)Storage<T>::round(r.x * inv) | ((uint32_t)Storage<T>::round(r.y * inv) << 16),
                     (uint32_t)Storage<T>::round(r.z * inv) | ((uint32_t)Storage<T>::round(r.w * inv) << 16));
    };
    auto add = [](float4& r, float f, const float4& v) {
      r.x = fmaf(f, v.x, r.x);
      r.y = fmaf(f, v.y, r.y);
      r.z = fmaf(f, v.z, r.z);
      r.w = fmaf(f, v.w, r.w);
    };
    const int items = p.group * (D / 4);  // outputs in vectors of 4
    if (team == 1) {
      // the group is this warp's alone
      __syncwarp();
      for (int i = lane; i < items; i += 32) {
        const int h = i / (D / 4), d = (i % (D / 4)) * 4;
        store(i, *reinterpret_cast<const float4*>(merge + (warp * kHeads + h) * D + merge_column<D>(h, d)),
              sm_l[warp * kHeads + h]);
      }
      __syncwarp();  // the merge buffer is free
    } else if (strided) {
      team_sync();
      const int w0 = warp - lead;
      for (int i = lead * 32 + lane; i < items; i += team * 32) {
        const int h = i / (D / 4), d = (i % (D / 4)) * 4;
        float mm = -INFINITY, ll = 0.f;
#pragma unroll 2
        for (int w = w0; w < w0 + team; ++w) mm = fmaxf(mm, sm_m[w * kHeads + h]);
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int w = w0; w < w0 + team; ++w) {
          const float m = sm_m[w * kHeads + h], f = m == mm ? 1.f : fast_exp2(m - mm);
          ll = fmaf(f, sm_l[w * kHeads + h], ll);
          add(r, f, *reinterpret_cast<const float4*>(merge + (w * kHeads + h) * D + merge_column<D>(h, d)));
        }
        store(i, r, ll);
      }
    } else {
      __syncthreads();
      const bool whole = here == seq.tiles;
      // shares that hold the group, and this one's partial state
      const int64_t group_start = lo + at - tile;
      const int slot_floats = cache_attn_slot_floats(p.group, D);
      int from = 0, parts = 1;
      if (!whole) {
        from = share_of(group_start);
        parts = share_of(group_start + seq.tiles - 1) - from + 1;
      }
      // (a CTA has at most two groups that others share: the one it begins in
      // the middle of, slot 0, and the one it leaves in the middle of, slot 1)
      auto slot_of = [&](int part) {
        return p.partials + (int64_t)(part ? 2 * (from + part) : 2 * from + 1) * slot_floats;
      };
      float* slot = slot_of((int)blockIdx.x - from);
      if (tid < items) {
        const int h = tid / (D / 4), d = (tid % (D / 4)) * 4;
        float mw[kW], mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          mw[w] = sm_m[w * kHeads + h];
          mm = fmaxf(mm, mw[w]);
        }
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          const float f = mw[w] == mm ? 1.f : fast_exp2(mw[w] - mm);
          ll = fmaf(f, sm_l[w * kHeads + h], ll);
          add(r, f, *reinterpret_cast<const float4*>(merge + (w * kHeads + h) * D + merge_column<D>(h, d)));
        }
        if (whole) {
          store(tid, r, ll);
        } else {
          __stcg(reinterpret_cast<float4*>(slot) + tid, r);
          if (d == 0) {
            __stcg(slot + p.group * D + h, mm);
            __stcg(slot + p.group * D + p.group + h, ll);
          }
        }
      }
      if (!whole) {
        // Join the parts: the last CTA to arrive at a counter joins the parts that
        // are counted there. Many parts are joined in two rounds, neighbours
        // first, into the slot of the first of them.
        const int part = (int)blockIdx.x - from;
        const bool wide = parts > kJoinWide;
        int width = wide ? kJoinWidth : parts;                   // parts counted together,
        int head = wide ? part / kJoinWidth * kJoinWidth : 0;    // the first of them,
        int step = 1;                                            // and their distance
        unsigned int* arrived = reinterpret_cast<unsigned int*>(&words[kW + 2]);
        for (;;) {
          const bool last_round = width == parts || step > 1;
          const int count = min((parts - head + step - 1) / step, width);
          // the last round's counter is that of the group's first share; a share
          // leads the first round of at most one group as its part 0 and of one
          // as a later part
          unsigned int* counter = p.counters + (last_round ? from : (head ? 2 : 1) * kMaxCtas + from + head);
          __syncthreads();
          if (tid == 0) {
            *arrived = arrive(counter);
          }
          __syncthreads();
          const unsigned int order = *arrived;
          if (order >= (unsigned int)count) {
            // the counter was not zero before this call
            if (tid == 0 && p.err_flag) atomicOr(p.err_flag, kErrWorkspace);
            const uint32_t nan2 = (uint32_t)Storage<T>::kNaN * 0x10001u;
            if (tid < items) *reinterpret_cast<uint2*>(out + tid * 8) = make_uint2(nan2, nan2);
            break;
          }
          if (order != (unsigned int)count - 1) break;
          // the threads share the vectors, and with fewer vectors than threads also
          // the parts; a thread's first ten are on their way while the warps
          // find the parts' factors
          float* factor = merge;                        // [count][8]
          float4* sums = reinterpret_cast<float4*>(merge + kJoinWide * kHeads);  // [kThreads]
          const int crews = Sh::kThreads / items, crew = tid / items, i = tid - crew * items, h = i / (D / 4);
          float4 v[10], r = make_float4(0.f, 0.f, 0.f, 0.f);
          auto fetch = [&](int s0) {
#pragma unroll
            for (int j = 0; j < 10; ++j)
              if (s0 + j * crews < count)
                v[j] = __ldcg(reinterpret_cast<const float4*>(slot_of(head + (s0 + j * crews) * step)) + i);
          };
          fetch(crew);
          if (warp < p.group) {
            // lane s has parts s and s + 32
            float m_s[2] = {-INFINITY, -INFINITY}, l_s[2] = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int s = lane + 32 * k;
              const float* at_s = slot_of(head + s * step) + p.group * D + warp;
              if (s < count) {
                m_s[k] = __ldcg(at_s);
                l_s[k] = __ldcg(at_s + p.group);
              }
            }
            float mm = fmaxf(m_s[0], m_s[1]), ll = 0.f;
#pragma unroll
            for (int k = 16; k; k >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, k));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int s = lane + 32 * k;
              if (s < count) {
                const float f = m_s[k] == mm ? 1.f : fast_exp2(m_s[k] - mm);
                factor[s * kHeads + warp] = f;
                ll += f * l_s[k];
              }
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, k);
            if (lane == 0) {
              sm_gl[warp] = ll;
              sm_gm[warp] = mm;
            }
          }
          __syncthreads();
          for (int s0 = crew; s0 < count;) {
#pragma unroll
            for (int j = 0; j < 10; ++j)
              if (s0 + j * crews < count) add(r, factor[(s0 + j * crews) * kHeads + h], v[j]);
            s0 += 10 * crews;
            if (s0 < count) fetch(s0);
          }
          if (crews > 1) {
            sums[tid] = r;
            __syncthreads();
            if (crew == 0)
              for (int c = 1; c < crews; ++c) add(r, 1.f, sums[c * items + i]);
          }
          if (tid == 0) *counter = 0;  // ready for the next call
          if (last_round) {
            if (crew == 0) store(i, r, sm_gl[h]);
            break;
          }
          float* joined = slot_of(head);
          if (crew == 0) {
            __stcg(reinterpret_cast<float4*>(joined) + i, r);
            if (i % (D / 4) == 0) {
              __stcg(joined + p.group * D + h, sm_gm[h]);
              __stcg(joined + p.group * D + p.group + h, sm_gl[h]);
            }
          }
          width = (parts + kJoinWidth - 1) / kJoinWidth;
          head = 0;
          step = kJoinWidth;
        }
      }
      __syncthreads();  // the merge buffer is free
    }

    // --- the next group
    at += here + behind(seq);
    tile = 0;
    bool any = true;
    if (lead == 0 || !strided) any = next_group(at, b, g, seq);
    if (__builtin_expect(strided && team > 1, 0)) {
      if (lead == 0) send(any);
      team_sync();  // and the team's part of the merge buffer is free
      any = receive();
    }
    if (!any) break;
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
    return e4m3 ? launch_cache_attn_t<T, true, 128>(p, sms, stream)
                : launch_cache_attn_t<T, false, 128>(p, sms, stream);
  return e4m3 ? launch_cache_attn_t<T, true, 64>(p, sms, stream) : launch_cache_attn_t<T, false, 64>(p, sms, stream);
}

}  // namespace da
