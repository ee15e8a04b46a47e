// Attention of several new tokens of each sequence over a paged cache: one pass
// over K and V on the fifth-generation tensor cores.
//
// The query rows that share a KV head (its G heads for each token) are the rows of
// the products: 128 to a tile, row = token * G + head. A unit is (sequence, KV
// head, 256 query rows) over all tiles of 128 cache rows; the launch's CTAs (one
// an SM) take equal runs of the tiles of all units, whatever the lengths. A unit
// that several CTAs take is joined from their partial states by the last of them
// to arrive, with the help of those that are still there (a row for each warp).
//
//   warps 0-7   two groups of 128 threads, a query row each: softmax with a
//               running maximum, weights to tensor memory, output
//   warp 8      page numbers and copies of K and V tiles into a ring
//   warp 9      the products: S = Q K^T (both in shared memory), O += P V (P in
//               tensor memory, V in shared memory as it lies, read transposed)
//   warps 12-15 8-bit pages: e4m3 to fp16 (exact), raw ring to operand ring
//
// Units of more than 128 rows ("two") give each group its own query tile and every
// K and V tile is used twice; smaller ones share the query tile, the groups take
// the cache tiles in turn, each with its own state, and join them at the end. So
// one group's exponentials run under the other's products.
//
// Mathematics, for a query row: w_j = 2^(s_j - m), s_j = log2(e) scale <q, K_j> for
// the rows j it sees; out = sum w_j V_j / sum w_j; the reference m is the maximum of
// the first tile in which the row sees something (so the weight of a row's only key, or of
// a sink, is 1, which no rounding changes) and is raised by a whole number when a score
// passes it by 7, so that what was summed before is rescaled exactly. Scores, sums and outputs are held in fp32, weights are rounded
// to the products' type (bf16 in two pieces, 16 bits, where one query tile leaves
// time for it; fp16, with 8-bit pages, lifted by 2^8 against its smallest numbers).
// With 8 bits a score is multiplied by K's scale, log2 |V's scale| is added to the
// weight's exponent (with a reference of its own: m; ml is that of the sum l).
//
// What bounds it (one GB300, device time inside a graph, from HBM): few query rows
// on long prefixes the bytes (32 sequences ragged up to 32768, chains of 5, 32/8
// heads: 418 us, 98% of the copy rate); many the chain of a group, products ->
// softmax -> products, with the other group's in between: 3000 cycles for a tile of
// 128 rows and 256 query rows (2048 of them the products'; 16 ragged up to 8191,
// trees of 64, 32/8 heads: 85 us), 3800 with 8 bits (32 ragged up to 16384, trees of
// 32, 64/8 heads: 343 us). Before the first tile there are 10 000 cycles (lengths,
// share, page numbers, query and first K rows), behind the last one 10 000 to 25 000
// (partial states, arrival, join): all of a small call (1 x 1024, a tree of 8, 16/16
// heads: 14.7 us).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "common.cuh"
#include "tree_params.h"

namespace da {

constexpr int kTreeTile = 128;             // cache rows of a tile, query rows of a tile
constexpr int kTreeUnitRows = 256;         // query rows of a unit
constexpr unsigned long long kTreeHelpNs = 20000;  // how long a CTA waits for a unit's other parts, to help with their join
constexpr int kTreeMinTiles = 2;            // a part of a unit has at least as many tiles
constexpr int kTreeJoinTiles = 8;           // what the ends of a share inside units cost, in tiles (at most the warps)
constexpr int kTreeUnitTiles = 6;           // ... what beginning and ending a unit takes
constexpr int kTreeAloneRows = 32;          // a unit of few rows is joined by the last CTA alone (1 x 1024: 16.5 -> 15.3 us)
constexpr float kTreeLazy = 7.f;            // a running maximum is raised when a score passes it by 2^7
constexpr float kTreeLift = 8.f;            // fp16 weights are held 2^8 times as large: a row's largest lies in (2^7, 2^15]

// A partial state: O, then (m, m of l, l) [256] float4. O is [256][D] for 16-bit pages; for 8 bits it lies as it does in
// shared memory on its way, [D / 32][256][32] with the 16-byte chunks of a row exchanged by the row's lowest bits.
__host__ __device__ constexpr int tree_slot_floats(int D) { return kTreeUnitRows * D + kTreeUnitRows * 4; }
template <int D, bool EIGHT>
__device__ __forceinline__ int tree_slot_at(int row, int column) {
  if constexpr (EIGHT) return (column / 32 * kTreeUnitRows + row) * 32 + (((column / 4 % 8) ^ (row & 7)) << 2);
  return row * D + column;
}
// Where the CTAs of one unit meet, by the CTA that begins it: a counter of arrivals in the workspace's first 4 KiB, where
// every attention operator has counters that are zero between calls, and these words behind it, whose values between
// calls do not matter (partial states of another operator may lie there). The last to arrive zeroes the counter and
// the ticket and then raises the generation.
struct alignas(8) TreeMeet {
  unsigned generation, ticket;
};
// A unit that this CTA has a part of.
struct TreePending {
  int c0, parts;           // its first CTA, and how many take part (0: the counter was not zero before the call)
  unsigned generation;     // of its meeting place before this CTA arrived
  int last;                // this CTA arrived last
  int rows, token0, g;
};

struct alignas(64) TreeLaunch {
  TensorMap k_map, v_map;  // 16-bit pages as rows of D elements; boxes of a page's rows (at most 128) by 64
  TreeParams p;
};

// The parts of a workspace.
struct TreeSpace {
  unsigned* arrived;
  TreeMeet* meets;
  float* partials;
};

cudaError_t launch_tree_f16(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, const TreeSpace& space,
                            cudaStream_t stream);
cudaError_t launch_tree_bf16(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, const TreeSpace& space,
                             cudaStream_t stream);

template <int D, bool EIGHT>
struct TreeShape {
  static constexpr int kBlocks = D / 64;                   // 64-column blocks of an operand tile
  static constexpr int kBlockBytes = kTreeTile * 128;
  static constexpr int kTileBytes = kBlocks * kBlockBytes; // 16-bit operand tile
  static constexpr int kRawBytes = kTreeTile * D;          // e4m3 tile
  static constexpr int kSlots = EIGHT ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  static constexpr int kRaw = EIGHT ? (D == 128 ? 4 : 6) : 0;
  // whole warpgroups (setmaxnreg); registers of a thread: at launch, of the softmax groups, of the others
  static constexpr int kThreads = EIGHT ? 512 : 384;
  // (8 bits with 184 and 72: 347 us where these take 340, 32 sequences ragged up to 16384)
  static constexpr int kRegsSoftmax = EIGHT ? 192 : 224, kRegsOther = EIGHT ? 64 : 56;
  static constexpr int kConverters = kThreads - 384;  // threads
  static constexpr int kQ = 0, kRing = 2 * kTileBytes, kRawRing = kRing + kSlots * kTileBytes;
  static constexpr int kControl = kRawRing + kRaw * kRawBytes;
  // At the end of a segment the query tiles are free: weighted outputs [2][128][32] for the exchange, and behind
  // them (or behind the control area) the states.
  static constexpr int kExchange = kQ, kExchangeBytes = 2 * kTreeTile * 32 * 4;
  static constexpr int kStateBytes = 2 * kTreeTile * 16 + kTreeUnitRows * 4;
  static constexpr int kStates = D == 128 ? kQ + kExchangeBytes : kControl + 2048;
  static constexpr int kSmem = 1024 + kControl + 2048 + (D == 128 ? 0 : kStateBytes);
  // bf16 weights of units with one query tile are held in two pieces (16 bits): the products have time for it, and
  // the columns behind the weights are free where they lie over the scores. With two query tiles the second piece
  // would cost 16 ragged up to 8191 and trees of 64 86 -> 101 us (relative error 0.0023 -> 0.0017, that of rounding the
  // output to bf16), with 8 bits 32 ragged up to 16384 342 -> 419 us; fp16 weights of one query tile 34.6 -> 36.0 us (4 x 8192,
  // 5 drafts), 39.6 -> 42.2 (32 drafts; 0.00024 -> 0.00021). A sum of the weights as they are held instead of before their
  // rounding: 86 -> 94 us.
  static constexpr bool kTwoPieces = D == 128 && !EIGHT;
  // tensor memory columns: scores of the groups, outputs, weights (in place of the scores where D is 128, whose two
  // products have one shape and therefore run in order)
  static constexpr int kS = 0, kO = 256, kP = D == 128 ? 0 : 384;
  static constexpr int kPStride = D == 128 ? 128 : 64;
};

struct TreeControl {
  uint64_t full[8], empty[8], raw_full[8], raw_empty[8];
  uint64_t s_full[2], p_full[2], q_full, o_final, o_free, drain;
  uint32_t tmem;
  int abort;
  int start[8];           // of this CTA's tiles: sequence, its first token, tokens, rows; KV head, unit, tile; tiles
  int piece, pieces;      // ... as a part of its unit; or where its first unit begins in the list, and its last tile + 1
  int unit_at, end_tile;
  int counts[32];
  TreePending pending[2];
  int pendings, ready, ticket;
  int16_t exponent[kTreeTile];  // 8 bits: of a query row's largest element
  alignas(16) float2 scales[8][8];  // 8 bits: of a warp's column groups: factor of a score, log2 of V's scale
  int sums[32];
  // of segment s, in entry s % 8: drafted rows whose V is not finite, and whether a page lies outside the pool
  uint32_t bad[8][8];
  int bad_page[8];
};
static_assert(sizeof(TreeControl) <= 2048 && offsetof(TreeControl, scales) % 16 == 0, "control area");
static_assert(128 * (2 * 224 + 56) <= 384 * 168 && 128 * (2 * 192 + 2 * 64) <= 512 * 128, "registers of the launch");

// Tokens and rows of a sequence; kt tiles for each of mps units a KV head.
struct TreeSeq {
  int first, n, rows, kt, mps;
  int state;  // 1 valid, 0 nothing to write, -1 NaN rows
};

__device__ __forceinline__ TreeSeq tree_sequence(const TreeParams& p, int b, int* errors) {
  TreeSeq s = {b, 1, 0, 0, 0, 0};
  if (p.start) {
    s.first = p.start[b];
    const int e = p.start[b + 1];
    if (s.first < 0 || e < s.first || e > p.tokens) {
      *errors |= kErrTokens;
      return s;
    }
    s.n = e - s.first;
  }
  if (s.n == 0) return s;
  s.state = -1;
  if (s.n > kTreeMaxTokens || (p.mask && s.n > 64 * p.mask_words)) {
    *errors |= kErrTokens;
    return s;
  }
  s.rows = p.kv_len[b];
  if (s.rows < s.n || s.rows > p.max_pages << p.page_shift) {
    *errors |= kErrKvLen;
    return s;
  }
  s.state = 1;
  s.kt = (s.rows + kTreeTile - 1) / kTreeTile;
  s.mps = (s.n * p.group + kTreeUnitRows - 1) / kTreeUnitRows;
  return s;
}

// Tiles [t0, t1) of one unit.
struct TreeSegment {
  int b, g, t0, t1, kt;
  int rows;        // rows of the sequence
  int base;        // first drafted row
  int count;       // query rows of the unit
  int token0;      // its first packed token
  int local0;      // ... as a token of its sequence
};

// A CTA's run of tiles, segment by segment (every role walks it by itself).
struct TreeCursor {
  int b, g, mp, tile, left;
  TreeSeq s;

  __device__ __forceinline__ void begin(const TreeParams& p, const int (&start)[8], int tiles) {
    left = tiles;
    if (tiles == 0) return;
    b = start[0];
    s.first = start[1];
    s.n = start[2];
    s.rows = start[3];
    s.kt = (s.rows + kTreeTile - 1) / kTreeTile;
    s.mps = (s.n * p.group + kTreeUnitRows - 1) / kTreeUnitRows;
    g = start[4];
    mp = start[5];
    tile = start[6];
  }
  __device__ __forceinline__ bool next(const TreeParams& p, TreeSegment* out) {
    if (left == 0) return false;
    if (tile == s.kt) {
      tile = 0;
      if (++mp == s.mps) {
        mp = 0;
        if (++g == p.n_kv_head) {
          g = 0;
          int none = 0;
          do {
            if (++b >= p.B) return false;
            s = tree_sequence(p, b, &none);
          } while (s.kt == 0);
        }
      }
    }
    out->b = b;
    out->g = g;
    out->t0 = tile;
    out->t1 = min(s.kt, tile + left);
    out->kt = s.kt;
    out->rows = s.rows;
    out->base = s.rows - s.n;
    out->count = min(kTreeUnitRows, s.n * p.group - mp * kTreeUnitRows);
    out->local0 = mp * (kTreeUnitRows / p.group);
    out->token0 = s.first + out->local0;
    left -= out->t1 - tile;
    tile = out->t1;
    return true;
  }
};

// A wait that ends with the CTA's other roles: false when one of them gave up.
__device__ __forceinline__ bool tree_wait(TreeControl* c, const TreeParams& p, uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int*>(&c->abort)) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      atomicOr(&c->abort, 1);
      if (p.err_flag) atomicOr(p.err_flag, kErrTimeout);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ void tensor_load_2d(uint32_t smem_dst, const TensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// From shared memory to `to`, and this thread's waits: until what it copies has been read, until it is written.
__device__ __forceinline__ void bulk_store(float* to, const void* from, int bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_addr(from)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 (or 16) columns of this warp's lanes; the caller waits with tmem_wait_load.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (tensor memory) = A B^T (+ D), A in shared or in tensor memory. The whole warp comes here, converged and with
// the same operands, and one elected lane issues: so the operands stay in uniform registers. What it costs to issue a
// product is what the kernel would wait for (64 cycles would do for one of 128 x 128 x 16; under a branch for one lane
// it cost 125, with a predicate made of the lane's number as much, whatever the product's size), so one vote serves
// several products.
// Four products along the contracted axis: of a 64-column block of both operands ...
__device__ __forceinline__ void tree_mma_ss4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc, add, one;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 acc, %4, 0;\n\tsetp.eq.b32 add, 0, 0;\n\t"
      "elect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, acc;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, add;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, add;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, add;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// ... of 64 rows of the second one and 32 columns of tensor memory.
__device__ __forceinline__ void tree_mma_ts4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc, add, one;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\tsetp.ne.b32 acc, %4, 0;\n\tsetp.eq.b32 add, 0, 0;\n\t"
      "elect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, acc;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, add;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, add;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, add;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tree_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc, one;\n\tsetp.ne.b32 acc, %4, 0;\n\telect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, acc;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tree_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
      "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
// M = 128; B transposed (its rows are the contracted ones) where `transpose`.
__host__ __device__ constexpr uint32_t tree_idesc(bool bf16, int n, bool transpose) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((transpose ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// An operand whose rows are the contracted ones, in the 128-byte swizzle: 64-column blocks `block` bytes apart,
// groups of eight rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc_rows(uint32_t addr, int block) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(block >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t sw128_desc_at(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// Byte of 16-byte chunk c of row r in a swizzled operand tile.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 3) * (kTreeTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Whether a packed pair of 16-bit values holds one that is not finite, by element.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_pair_mask(uint32_t v) {
  constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t keep = 0xffffffffu;
  if ((v & kExp) == kExp) keep &= 0xffff0000u;
  if ((v >> 16 & kExp) == kExp) keep &= 0x0000ffffu;
  return keep;
}

// Bits [at, at + 32) of a token's mask over the new rows (at may be negative).
__device__ __forceinline__ uint32_t draft_bits(const TreeParams& p, int token, int local, int n, int at) {
  if (at >= n || at <= -32) return 0;
  uint32_t v;
  if (p.mask) {
    const uint64_t* words = p.mask + (int64_t)token * p.mask_words;
    if (at < 0) {
      v = (uint32_t)(__ldg(words) << -at);
    } else {
      const int w = at >> 6, shift = at & 63;
      uint64_t x = __ldg(words + w) >> shift;
      if (shift > 32 && w + 1 < p.mask_words) x |= __ldg(words + w + 1) << (64 - shift);
      v = (uint32_t)x;
    }
  } else {
    const int ones = local + 1 - at;  // columns up to the token's own
    v = ones <= 0 ? 0u : ones >= 32 ? 0xffffffffu : (1u << ones) - 1;
    if (at < 0) v &= 0xffffffffu << -at;
  }
  const int most = n - at;
  return most >= 32 ? v : v & ((1u << most) - 1);
}

// Which of the rows [j, j + 32) a token sees.
__device__ __forceinline__ uint32_t seen_bits(const TreeParams& p, const TreeSegment& s, int token, int local, int j) {
  const int before = s.base - j;
  const uint32_t prefix = before <= 0 ? 0u : before >= 32 ? 0xffffffffu : (1u << before) - 1;
  return prefix | draft_bits(p, token, local, s.rows - s.base, -before);
}

template <int REGS>
__device__ __forceinline__ void raise_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void lower_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// A row's softmax state: m for the output and the weights, ml for l (they differ with scales of V).
struct TreeState {
  float m, ml, l;
};

// Tensor-memory column of the weights of cache row k of a tile (two to a column). In two pieces they lie by halves of
// the tile, first pieces, then second ones: the half of the scores that is still to be read is not written over.
template <int PIECES>
__device__ __forceinline__ int weight_column(int k) {
  return PIECES == 2 ? k / 64 * 64 + k % 64 / 2 : k / 2;
}

// COLS columns of scores, from column `col` on, to weights in tensor memory, their sum to the state. The weights are
// taken against a running maximum: that of the row's first columns, and where a score passes it by 2^7 it is raised by a
// whole number, and the output, the sum and earlier weights of the tile are rescaled (by powers of two: exact). a: factor
// of a score (positive); seen: bits of the columns, looked at where `masked`. 8 bits: scales holds the factor that K's scale is and log2 |V's scale|
// of each 16 rows (-inf where it is zero: such rows count for l alone, and raise no reference but its own), sign (in lanes 0 to
// 7) the sign of V's scale or zero; PLAIN: all of K's are positive, and so are V's
// (a branch for every 16 columns took 4000 cycles an item). Straight code for the columns held in registers: as a loop
// over 32 at a time, 128 took 4000 cycles instead of 1700.
template <bool BF16, int D, bool EIGHT, int COLS, int PIECES, bool PLAIN>
__device__ __forceinline__ void softmax_columns(TreeState& st, uint32_t s_at, uint32_t p_at, uint32_t o_at, int col,
                                                bool first, float a, bool masked, const uint32_t (&seen)[4],
                                                const float2* scales, float sign) {
  constexpr float kLift = BF16 ? 0.f : kTreeLift;
  // (8 bits have fewer registers: 128 columns by halves)
  constexpr int kHold = EIGHT && COLS == 128 ? 64 : COLS;
  // (a NaN of no other origin where factors may be zero or negative)
  constexpr uint32_t kHidden = EIGHT && !PLAIN ? 0x7fdeadedu : 0xff800000u;
  constexpr int kGroups = EIGHT ? kHold / 16 : 1, kPart = kHold / kGroups;
#pragma unroll 1
  for (int from = 0; from < COLS; from += kHold) {
    uint32_t r[kHold];
#pragma unroll
    for (int k = 0; k < kHold / 32; ++k) tmem_load32(s_at + col + from + 32 * k, r + 32 * k);
    float ak[kGroups], vk[kGroups];
    if constexpr (EIGHT) {
#pragma unroll
      for (int g = 0; g < kGroups; g += 2) {
        const float4 x = *reinterpret_cast<const float4*>(scales + (col + from) / 16 + g);
        ak[g] = PLAIN ? fmaxf(a * x.x, 1.2e-38f) : a * x.x;  // (never zero, which would make hidden scores NaN)
        vk[g] = x.y;
        ak[g + 1] = PLAIN ? fmaxf(a * x.z, 1.2e-38f) : a * x.z;
        vk[g + 1] = x.w;
      }
    } else {
      ak[0] = a;
      vk[0] = 0.f;
    }
    tmem_wait_load();
    if (masked) {
#pragma unroll
      for (int k = 0; k < kHold / 32; ++k) {
        const uint32_t bits = kHold < COLS && from > 0 ? seen[2 + k] : seen[k];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(bits >> i & 1)) r[32 * k + i] = kHidden;
      }
    }
    float m_tile = -INFINITY, ml_tile = -INFINITY;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kPart; i += 2)
        top[i / 2 % 4] = fmaxf(fmaxf(__uint_as_float(r[kPart * g + i]), __uint_as_float(r[kPart * g + i + 1])), top[i / 2 % 4]);
      top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (EIGHT && !PLAIN && ak[g] < 0.f) {
        top[0] = INFINITY;
#pragma unroll
        for (int i = 0; i < kPart; ++i) top[0] = fminf(top[0], __uint_as_float(r[kPart * g + i]));
      }
      // (nothing seen: no product with a factor that may be zero)
      if (!EIGHT || PLAIN) {
        top[0] *= ak[g];
      } else {
        top[0] = fabsf(top[0]) < INFINITY ? top[0] * ak[g] : top[0] == INFINITY && ak[g] > 0.f ? INFINITY : -INFINITY;
      }
      ml_tile = fmaxf(ml_tile, top[0]);
      m_tile = fmaxf(m_tile, EIGHT ? top[0] + vk[g] : top[0]);
    }
    const bool up = m_tile > st.m + kTreeLazy || (st.m == -INFINITY && m_tile > -INFINITY);
    const bool up_l = EIGHT && (ml_tile > st.ml + kTreeLazy || (st.ml == -INFINITY && ml_tile > -INFINITY));
    if (__any_sync(0xffffffffu, up || up_l)) {
      // (what was summed before counts for nothing, 2^-256, where the maximum rises by more: taken anew, as a sum with a
      // reference so far away would be rounded to a step of many powers of two)
      const bool none = st.m == -INFINITY || m_tile - st.m > 256.f;
      const float step = up && !none ? ceilf(m_tile - st.m) : 0.f;
      const float factor = up && none ? 0.f : fast_exp2(-step);
      st.m = up && none ? m_tile : st.m + step;
      if constexpr (EIGHT) {
        if (up_l) {
          const float ml_new = ceilf(ml_tile);
          st.l *= st.ml == -INFINITY ? 0.f : fast_exp2(st.ml - ml_new);
          st.ml = ml_new;
        }
      } else {
        st.l *= factor;
        st.ml = st.m;
      }
      if (kHold < COLS && from > 0) {
        tmem_wait_store();
        // the weights of the first half, two fp16 numbers to a column
#pragma unroll 1
        for (int k = 0; k < from / 2; k += 16) {
          uint32_t w[16];
          tmem_load16(p_at + k, w);
          tmem_wait_load();
          const __half2 f = __float2half2_rn(factor);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&w[i]), f);
            w[i] = *reinterpret_cast<const uint32_t*>(&x);
          }
          tmem_store16(p_at + k, w);
        }
      }
      if (!first) {
#pragma unroll 1
        for (int k = 0; k < D; k += 16) {
          uint32_t o[16];
          tmem_load16(o_at + k, o);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
          tmem_store16(o_at + k, o);
        }
      }
    }
    const float ref = st.m == -INFINITY ? 0.f : st.m - kLift, lref = st.ml == -INFINITY ? 0.f : st.ml;
    if constexpr (EIGHT && !PLAIN) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        if (vk[g] == -INFINITY) vk[g] = ref - lref;  // (no scale: weights of l as they are)
    }
    float total = 0.f;
#pragma unroll
    for (int h = 0; h < kHold; h += 32) {
      uint32_t hi[16], lo[16];
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const int at = h + i, g = EIGHT ? at / 16 : 0;
        float2 y = __ffma2_rn(make_float2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])),
                              make_float2(ak[g], ak[g]), make_float2(vk[g] - ref, vk[g] - ref));
        if (EIGHT && !PLAIN && masked) {
          if (r[at] == kHidden) y.x = -INFINITY;
          if (r[at + 1] == kHidden) y.y = -INFINITY;
        }
        y.x = fast_exp2(y.x);
        y.y = fast_exp2(y.y);
        sum[i / 16] = __fadd2_rn(sum[i / 16], y);
        const uint32_t v = pack2<BF16>(y.x, y.y);
        hi[i / 2] = v;
        if constexpr (PIECES == 2)
          lo[i / 2] = pack2<true>(y.x - __uint_as_float(v << 16), y.y - __uint_as_float(v & 0xffff0000u));
      }
      if constexpr (EIGHT) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // l counts the weights without the scale of V
          total += (sum[g].x + sum[g].y) * fast_exp2(fminf(ref - lref - vk[h / 16 + g], 126.f));
          if constexpr (!PLAIN) {
            const float sg = __shfl_sync(0xffffffffu, sign, (col + from + h) / 16 + g);
            if (sg != 1.f) {
#pragma unroll
              for (int i = 8 * g; i < 8 * g + 8; ++i) hi[i] = sg == 0.f ? 0u : hi[i] ^ 0x80008000u;
            }
          }
        }
      } else {
        total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // (over scores that are in registers, or were used)
      tmem_store16(p_at + weight_column<PIECES>(col + from + h), hi);
      if constexpr (PIECES == 2) tmem_store16(p_at + weight_column<PIECES>(col + from + h) + 32, lo);
    }
    st.l += total;
  }
  if constexpr (COLS < 128) {
    // the other columns of this row belong to its copies
    uint32_t none[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) none[i] = 0;
#pragma unroll
    for (int k = 0; k < 128; k += 32) {
      if (k >= col && k < col + COLS) continue;
      tmem_store16(p_at + weight_column<PIECES>(k), none);
      if constexpr (PIECES == 2) tmem_store16(p_at + weight_column<PIECES>(k) + 32, none);
    }
  }
  tmem_wait_store();
}

__device__ __forceinline__ unsigned arrive_acq_rel(unsigned* at) {
  unsigned before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(at) : "memory");
  return before;
}
__device__ __forceinline__ void store_release(unsigned* at, unsigned v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(at), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned load_acquire(const unsigned* at) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}

// Rows [r0, r1) of a unit from its parts, by the 256 softmax threads: the parts' weights of each row into shared memory
// (a thread for each row), then four columns a thread over the parts. The first CTA's part is its second state, the
// others' their first. No parts: NaN.
template <typename T, int D, bool EIGHT>
__device__ __forceinline__ void tree_join_rows(const TreeParams& p, const float* partials, const TreePending& x, int r0,
                                               int r1, float* weights) {
  const int rows = r1 - r0, parts = x.parts;
  auto slot = [&](int i) { return partials + ((int64_t)(x.c0 + i) * 2 + (i == 0 ? 1 : 0)) * tree_slot_floats(D); };
  for (int r = threadIdx.x; r < rows; r += 256) {
    auto state = [&](int i) { return __ldcg(reinterpret_cast<const float4*>(slot(i) + kTreeUnitRows * D) + r0 + r); };
    float m = -INFINITY, ml = -INFINITY, l = parts > 0 ? 0.f : NAN;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float4 s = state(i);
      m = fmaxf(m, s.x);
      ml = fmaxf(ml, s.y);
    }
    const float m0 = m == -INFINITY ? 0.f : m, ml0 = ml == -INFINITY ? 0.f : ml;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
      const float4 s = state(i);
      weights[i * rows + r] = fast_exp2(s.x - m0);
      l += s.z * fast_exp2(s.y - ml0);
    }
    // (no reference: nothing but rows whose V has a scale of zero)
    weights[parts * rows + r] = l == 0.f ? 0.f : (m == -INFINITY ? 0.f : fast_exp2(m0 - ml0)) / l;
  }
  named_barrier_sync<1, 256>();
  // four rows of a thread at once, so that as many loads of each part are on their way
  constexpr int kStep = 256 / (D / 4), kRows = 4;
  const int shift = __ffs(p.group) - 1, col = threadIdx.x % (D / 4);
#pragma unroll 1
  for (int first = threadIdx.x / (D / 4); first < rows; first += kRows * kStep) {
    float4 acc[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll(EIGHT ? 4 : 2)
    for (int i = 0; i < parts; ++i) {
      const float* const from = slot(i);
      float4 o[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        o[k] = __ldcg(reinterpret_cast<const float4*>(from + tree_slot_at<D, EIGHT>(r0 + min(first + k * kStep, rows - 1), 4 * col)));
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const float w = weights[i * rows + min(first + k * kStep, rows - 1)];
        acc[k].x = fmaf(o[k].x, w, acc[k].x);
        acc[k].y = fmaf(o[k].y, w, acc[k].y);
        acc[k].z = fmaf(o[k].z, w, acc[k].z);
        acc[k].w = fmaf(o[k].w, w, acc[k].w);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = first + k * kStep, row = r0 + r;
      if (r >= rows) break;
      const float inv = weights[parts * rows + r];
      const int64_t at = ((int64_t)(x.token0 + (row >> shift)) * p.n_head + x.g * p.group + (row & (p.group - 1))) * D;
      *reinterpret_cast<uint2*>(p.out + (at + 4 * col) * 2) =
          make_uint2(pack2<Storage<T>::kBf16>(acc[k].x * inv, acc[k].y * inv),
                     pack2<Storage<T>::kBf16>(acc[k].z * inv, acc[k].w * inv));
    }
  }
}

template <typename T, int D, bool EIGHT>
__global__ void __launch_bounds__(TreeShape<D, EIGHT>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeLaunch launch, unsigned* arrived, TreeMeet* meets, float* partials) {
  using Shape = TreeShape<D, EIGHT>;
  using S = Storage<T>;
  constexpr bool kBf16 = S::kBf16 && !EIGHT;  // type of the products
  constexpr int kThreads = Shape::kThreads, kWarps = kThreads / 32;
  const TreeParams& p = launch.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  TreeControl* const c = reinterpret_cast<TreeControl*>(smem + Shape::kControl);
  const uint32_t ring = smem_addr(smem + Shape::kRing), raw_ring = smem_addr(smem + Shape::kRawRing);
  const uint32_t q_tiles = smem_addr(smem + Shape::kQ);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&c->full[i], EIGHT ? Shape::kConverters : 1);
      mbar_init(&c->empty[i], 1);
      mbar_init(&c->raw_full[i], 1);
      mbar_init(&c->raw_empty[i], max(Shape::kConverters, 1));
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_full[i], 128);
    }
    mbar_init(&c->q_full, 256);
    mbar_init(&c->o_final, 2);
    mbar_init(&c->o_free, 256);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    for (int i = 0; i < 8; ++i) {
      c->bad_page[i] = 0;
      for (int w = 0; w < 8; ++w) c->bad[i][w] = 0;
    }
    fence_mbar_init();
    fence_proxy_async_shared();
  }
  if (warp == 9) {
    tmem_alloc(&c->tmem, 512);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  pdl_wait();
  pdl_trigger();

  // This CTA's share of all tiles, and where it begins: a part of one unit, or an even share of the list of all units.
  // Every unit is cut into parts of its own, a CTA each, where there are not more of them than CTAs and the largest is
  // longer than an even share by less than kTreeJoinTiles tiles: even shares end and begin inside units, which costs a
  // CTA partial states and joins. In the list a unit counts for its tiles and kTreeUnitTiles more, which is what
  // beginning and ending one takes; a share that would begin within those begins with the unit.
  int errors = 0, total = 0, part_tiles = 0, ctas = 0;  // total: of the list, with what units count for
  {
    auto units_of = [&](int b, int* kt) {
      *kt = 1;
      if (b >= p.B) return 0;
      const TreeSeq s = tree_sequence(p, b, &errors);
      if (s.kt) *kt = s.kt;
      return s.kt ? p.n_kv_head * s.mps : 0;
    };
    // (up to 32 sequences every warp looks at them by itself, without barriers)
    const bool small = p.B <= 32;
    int my_kt, kt;
    const int my_units = units_of(small ? lane : threadIdx.x, &my_kt);
    int tiles = my_units * my_kt, units = my_units;
    for (int b = threadIdx.x + kThreads; b < p.B; b += kThreads) {
      const int n = units_of(b, &kt);
      tiles += n * kt;
      units += n;
    }
    // the sequences' units and tiles, as far as one pass goes, for the search of the parts' size
    int2* const table = reinterpret_cast<int2*>(smem + Shape::kQ);
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    units = __reduce_add_sync(0xffffffffu, units);
    if (!small) {
      table[threadIdx.x] = make_int2(my_units, my_kt);
      if (lane == 0) {
        c->sums[warp] = tiles;
        c->counts[warp] = units;
      }
      __syncthreads();
      tiles = __reduce_add_sync(0xffffffffu, lane < kWarps ? c->sums[lane] : 0);
      units = __reduce_add_sync(0xffffffffu, lane < kWarps ? c->counts[lane] : 0);
    }
    const int grid = gridDim.x, share = max((tiles + grid - 1) / grid, kTreeMinTiles);
    total = tiles + kTreeUnitTiles * units;
    ctas = min(grid, total);
    if (small && units <= grid) {
      for (int size = share; size < share + kTreeJoinTiles && part_tiles == 0; ++size) {
        if (__reduce_add_sync(0xffffffffu, my_units * ((my_kt + size - 1) / size)) <= grid) part_tiles = size;
      }
    } else if (units <= grid && p.B <= kThreads) {  // (the same in every thread)
      // one candidate for each warp: share, share + 1, ...
      int parts = 0;
      for (int i = lane; i < p.B; i += 32) parts += table[i].x * ((table[i].y + share + warp - 1) / (share + warp));
      parts = __reduce_add_sync(0xffffffffu, parts);
      __syncthreads();
      if (lane == 0) c->counts[warp] = parts;
      __syncthreads();
      const uint32_t fits = __ballot_sync(0xffffffffu, lane < kTreeJoinTiles && c->counts[lane] <= grid);
      if (fits) part_tiles = share + __ffs(fits) - 1;
    }
    // the part's number; or where the share begins in the list, and the next one
    int want = blockIdx.x, next = 0;
    if (part_tiles == 0) {
      const bool on = (int)blockIdx.x < ctas;
      want = on ? (int)((int64_t)total * blockIdx.x / ctas) : total;
      next = on ? (int)((int64_t)total * (blockIdx.x + 1) / ctas) : total;
    }
    if (threadIdx.x == 0) {
      c->start[7] = 0;
      c->end_tile = tiles;
    }
    __syncwarp();
    int before = 0, units_before = 0;
    for (int base = 0; base < p.B && before <= max(want, next); base += kThreads) {
      int n = my_units;
      kt = my_kt;
      if (base > 0) n = units_of(base + threadIdx.x, &kt);
      // what a unit counts for, and all of the sequence
      const int each = part_tiles > 0 ? (kt + part_tiles - 1) / part_tiles : kt + kTreeUnitTiles, v = n * each;
      int scan = v, scan_units = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o), up_units = __shfl_up_sync(0xffffffffu, scan_units, o);
        if (lane >= o) {
          scan += up;
          scan_units += up_units;
        }
      }
      int w = 0, wu = 0;
      if (!small) {
        __syncthreads();
        if (lane == 31) {
          c->sums[warp] = scan;
          c->counts[warp] = scan_units;
        }
        __syncthreads();
        w = lane < kWarps ? c->sums[lane] : 0;
        wu = lane < kWarps ? c->counts[lane] : 0;
      }
      const int at = before + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + scan - v;
      const int first_unit = units_before + __reduce_add_sync(0xffffffffu, lane < warp ? wu : 0) + scan_units - n;
      // (tiles before the sequence's, in the list)
      const int tiles_at = at - kTreeUnitTiles * first_unit;
      const bool writes = !small || warp == 0;
      if (writes && want >= at && want < at + v) {
        int none = 0;
        const TreeSeq x = tree_sequence(p, base + threadIdx.x, &none);
        const int off = want - at, unit = off / each, piece = off - unit * each, head = unit / x.mps;
        c->start[0] = base + threadIdx.x;
        c->start[1] = x.first;
        c->start[2] = x.n;
        c->start[3] = x.rows;
        c->start[4] = head;
        c->start[5] = unit - head * x.mps;
        if (part_tiles > 0) {
          const int share_tiles = x.kt / each, more = x.kt - share_tiles * each;
          c->start[6] = piece * share_tiles + min(piece, more);
          c->start[7] = share_tiles + (piece < more ? 1 : 0);
          c->piece = piece;
          c->pieces = each;
        } else {
          const int tile = max(0, piece - kTreeUnitTiles);
          c->start[6] = tile;
          c->start[7] = -(tiles_at + unit * x.kt + tile) - 1;  // (the number of tiles once the end is known)
          c->unit_at = at + unit * each;
        }
      }
      if (writes && part_tiles == 0 && next >= at && next < at + v) {
        const int off = next - at, unit = off / each;
        c->end_tile = tiles_at + unit * kt + max(0, off - unit * each - kTreeUnitTiles);
      }
      before += __reduce_add_sync(0xffffffffu, w);
      units_before += __reduce_add_sync(0xffffffffu, wu);
    }
    __syncthreads();
  }
  const int my_tiles = c->start[7] >= 0 ? c->start[7] : c->end_tile + c->start[7] + 1;
  if (blockIdx.x == 0 && errors && p.err_flag) atomicOr(p.err_flag, errors);
  TreeCursor cursor;
  cursor.begin(p, c->start, my_tiles);
  TreeSegment seg;

  if (warp == 8) {
    // ---------------- producer ----------------
    lower_registers<Shape::kRegsOther>();
    const int step = min(p.page_rows, kTreeTile);  // rows of a page in a tile
    uint8_t* const pools[2] = {const_cast<uint8_t*>(p.k), const_cast<uint8_t*>(p.v)};
    constexpr int kStages = EIGHT ? Shape::kRaw : Shape::kSlots;
    uint64_t* const full = EIGHT ? c->raw_full : c->full;
    uint64_t* const empty = EIGHT ? c->raw_empty : c->empty;
    int stage = 0, round = 0, issued = 0;
    bool ok = true;
    for (int s = 0; ok && cursor.next(p, &seg); ++s) {
      const int32_t* const table = p.table + (int64_t)seg.b * p.max_pages;
      for (int t = seg.t0; ok && t < seg.t1; ++t) {
        const int j0 = t * kTreeTile, pages = (min(kTreeTile, seg.rows - j0) + step - 1) / step;
        int id = lane < pages ? table[(j0 + lane * step) >> p.page_shift] : 0;
        const bool fine = id >= 0 && id < p.num_pages;
        const uint32_t on = __ballot_sync(0xffffffffu, lane < pages && fine);
        if (__popc(on) != pages && lane == 0) {
          c->bad_page[s & 7] = 1;
          if (p.err_flag) atomicOr(p.err_flag, kErrPage);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (round > 0) ok = __all_sync(0xffffffffu, tree_wait(c, p, &empty[stage], (round - 1) & 1));
          if (!ok) break;
          const int row_bytes = EIGHT ? D : 2 * D;
          const bool skipped = issued == p.skip_slot && blockIdx.x == 0;  // (failure test: a copy that never comes)
          if (lane == 0 && !skipped) mbar_arrive_expect_tx(&full[stage], __popc(on) * step * row_bytes);
          __syncwarp();
          if constexpr (EIGHT) {
            if (lane < pages && fine && !skipped) {
              const int64_t row = ((int64_t)id * p.n_kv_head + seg.g) * p.page_rows + ((j0 + lane * step) & (p.page_rows - 1));
              bulk_load_plain(smem + Shape::kRawRing + stage * Shape::kRawBytes + lane * step * D, pools[kv] + row * D,
                              step * D, &full[stage]);
            }
          } else {
            const int page = lane / Shape::kBlocks, block = lane % Shape::kBlocks;
            const int at = __shfl_sync(0xffffffffu, id, page);
            if (page < pages && (on >> page & 1) && !skipped) {
              const int row = (at * p.n_kv_head + seg.g) * p.page_rows + ((j0 + page * step) & (p.page_rows - 1));
              tensor_load_2d(ring + stage * Shape::kTileBytes + block * Shape::kBlockBytes + page * step * 128,
                             kv ? &launch.v_map : &launch.k_map, block * 64, row, &full[stage]);
            }
          }
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            ++round;
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // copies in flight land before the CTA leaves (bounded)
      for (int u = max(0, issued - kStages); u < issued; ++u) mbar_wait(&full[u % kStages], (u / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------- products ----------------
    lower_registers<Shape::kRegsOther>();
    constexpr uint32_t kScores = tree_idesc(kBf16, kTreeTile, false), kOut = tree_idesc(kBf16, D, true);
    const uint32_t tm = uniform(tmem), q0 = uniform(q_tiles), ring0 = uniform(ring), bars = uniform(smem_addr(c));
    auto bar = [&](uint64_t* b) { return bars + (uint32_t)(reinterpret_cast<uint8_t*>(b) - reinterpret_cast<uint8_t*>(c)); };
    int tau = 0, phase_p[2] = {0, 0};
    bool ok = true;
    for (int s = 0; ok && cursor.next(p, &seg); ++s) {
      const bool two = uniform(seg.count) > kTreeTile;
      const int tiles = uniform(seg.t1 - seg.t0), items = two ? 2 * tiles : tiles;
      const int last_steps = (uniform(min(kTreeTile, seg.rows - (seg.t1 - 1) * kTreeTile)) + 15) / 16;
      const bool pieces = kBf16 && Shape::kTwoPieces && !two;
      ok = __all_sync(0xffffffffu, tree_wait(c, p, &c->q_full, s & 1));
      for (int u = 0; ok && u <= items; ++u) {
        if (u < items) {
          const int use = 2 * (tau + (two ? u >> 1 : u)), slot = use % Shape::kSlots;
          if (!two || !(u & 1)) ok = __all_sync(0xffffffffu, tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = sw128_desc_at(q0 + (two ? (u & 1) * Shape::kTileBytes : 0));
          const uint64_t b = sw128_desc_at(ring0 + slot * Shape::kTileBytes);
          const uint32_t to = tm + Shape::kS + (u & 1) * 128;
#pragma unroll
          for (int k = 0; k < Shape::kBlocks; ++k) {
            const uint64_t off = (uint64_t)(k * Shape::kBlockBytes >> 4);
            tree_mma_ss4(to, a + off, b + off, kScores, k > 0);
          }
          tree_commit(bar(&c->s_full[u & 1]));
          if (!two || (u & 1)) tree_commit(bar(&c->empty[slot]));
        }
        if (u > 0) {
          const int v = u - 1, grp = v & 1, t = two ? v >> 1 : v;
          const int use = 2 * (tau + t) + 1, slot = use % Shape::kSlots;
          if (v == 0 && s > 0) ok = tree_wait(c, p, &c->o_free, (s - 1) & 1);
          if (ok) ok = tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1);
          if (ok) ok = tree_wait(c, p, &c->p_full[grp], phase_p[grp] & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++phase_p[grp];
          tc_fence_after();
          const int steps = t == tiles - 1 ? last_steps : kTreeTile / 16;
          const uint64_t b = sw128_desc_rows(ring0 + slot * Shape::kTileBytes, Shape::kBlockBytes);
          const uint32_t weights = tm + Shape::kP + grp * Shape::kPStride, to = tm + Shape::kO + grp * D;
          if (steps == kTreeTile / 16) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t rows = b + (uint64_t)((k * 64 * 128) >> 4);
              const uint32_t at = weights + (pieces ? weight_column<2>(64 * k) : weight_column<1>(64 * k));
              tree_mma_ts4(to, at, rows, kOut, k > 0 || v >= 2);
              if (pieces) tree_mma_ts4(to, at + 32, rows, kOut, true);
            }
          } else {
#pragma unroll 1
            for (int k = 0; k < steps; ++k) {
              const uint64_t rows = b + (uint64_t)((k * 2048) >> 4);
              const uint32_t at = weights + (pieces ? weight_column<2>(16 * k) : weight_column<1>(16 * k));
              tree_mma_ts(to, at, rows, kOut, k > 0 || v >= 2);
              if (pieces) tree_mma_ts(to, at + 32, rows, kOut, true);
            }
          }
          if (!two || (v & 1)) tree_commit(bar(&c->empty[slot]));
        }
      }
      if (!ok) break;
      tree_commit(bar(&c->o_final));
      if (lane == 0) mbar_arrive(&c->o_final);
      __syncwarp();
      tau += tiles;
    }
    if (!ok) {
      // products in flight end before the memory is freed (bounded)
      tree_commit(bar(&c->drain));
      mbar_wait(&c->drain, 0);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- e4m3 to fp16 (and two warps that complete a group) ----------------
    lower_registers<Shape::kRegsOther>();
    if (warp < 12) {
      // sequences that are refused: NaN rows
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        int none = 0;
        const TreeSeq x = tree_sequence(p, b, &none);
        if (x.state >= 0) continue;
        const uint32_t n = (uint32_t)S::kNaN * 0x10001u;
        uint4* const out = reinterpret_cast<uint4*>(p.out + (int64_t)x.first * p.n_head * D * 2);
        for (int64_t i = threadIdx.x - 320; i < (int64_t)x.n * p.n_head * (D / 8); i += 64) out[i] = make_uint4(n, n, n, n);
      }
    }
    if constexpr (EIGHT) if (warp >= 12) {
      const int th = threadIdx.x - 384;
      constexpr int kChunks = D / 16;                                       // 16-byte chunks of a raw row
      constexpr int kEach = kTreeTile * kChunks / Shape::kConverters;       // ... of a thread
      int use = 0;
      bool ok = true;
      for (int s = 0; ok && cursor.next(p, &seg); ++s) {
        for (int t = seg.t0; ok && t < seg.t1; ++t) {
          const int j0 = t * kTreeTile, valid = min(kTreeTile, seg.rows - j0);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++use) {
            const int raw = use % Shape::kRaw, slot = use % Shape::kSlots, round = use / Shape::kSlots;
            ok = tree_wait(c, p, &c->raw_full[raw], (use / Shape::kRaw) & 1);
            if (ok && round > 0) ok = tree_wait(c, p, &c->empty[slot], (round - 1) & 1);
            if (!ok) break;
            const uint8_t* const from = smem + Shape::kRawRing + raw * Shape::kRawBytes;
            uint8_t* const to = smem + Shape::kRing + slot * Shape::kTileBytes;
            auto store = [&](const uint32_t (&h)[8], int idx) {
              const int r = idx / kChunks, ch = idx % kChunks;
              *reinterpret_cast<uint4*>(to + chunk_at<D>(r, 2 * ch)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(to + chunk_at<D>(r, 2 * ch + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
            };
            auto convert = [&](const uint4& x, int idx) {
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              uint32_t h[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * k]) : "h"((uint16_t)(w[k] & 0xffffu)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * k + 1]) : "h"((uint16_t)(w[k] >> 16)));
              }
              store(h, idx);
            };
            if (kv == 0 || j0 + kTreeTile <= seg.base) {
#pragma unroll
              for (int i = 0; i < kEach; ++i)
                convert(ld_shared_v4(from + (th + i * Shape::kConverters) * 16), th + i * Shape::kConverters);
            } else {
#pragma unroll 1
              for (int i = 0; i < kEach; ++i) {
                const int idx = th + i * Shape::kConverters, r = idx / kChunks;
                uint4 x = ld_shared_v4(from + idx * 16);
                if (r >= valid) {
                  x = make_uint4(0u, 0u, 0u, 0u);
                } else if (j0 + r >= seg.base) {
                  // drafted rows: NaN reaches only those who see it (added at the end)
                  bool nan = false;
                  auto clean = [&](uint32_t& w) {
                    const uint32_t m = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    nan |= m != 0;
                    w &= ~m;
                  };
                  clean(x.x);
                  clean(x.y);
                  clean(x.z);
                  clean(x.w);
                  const int d = j0 + r - seg.base;
                  if (nan) atomicOr(&c->bad[s & 7][d >> 5], 1u << (d & 31));
                }
                convert(x, idx);
              }
            }
            fence_proxy_async_shared();
            mbar_arrive(&c->full[slot]);
            mbar_arrive(&c->raw_empty[raw]);
          }
        }
      }
    }
  } else {
    // ---------------- softmax and output ----------------
    raise_registers<Shape::kRegsSoftmax>();
    const int grp = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + Shape::kS + grp * 128, p_at = tmem + lanes + Shape::kP + grp * Shape::kPStride;
    const uint32_t o_at = tmem + lanes + Shape::kO + grp * D;
    const bool negate = p.qscale < 0.f, flat = p.qscale == 0.f;
    const int gshift = __ffs(p.group) - 1;
    int phase_s = 0, tau = 0;
    bool dead = false;
    int unit_at = c->unit_at;  // where the unit at hand begins in the list
    if (threadIdx.x == 0) c->pendings = 0;
    for (int s = 0; cursor.next(p, &seg); ++s) {
      const bool two = seg.count > kTreeTile;
      const int tiles = seg.t1 - seg.t0, items = two ? 2 * tiles : tiles;
      // A unit of few rows has them several times in its tile: each copy takes its part of a cache tile's columns, so
      // that all warps work on the exponentials.
      const int copies = seg.count <= 32 ? 4 : seg.count <= 64 ? 2 : 1;
      const int own = kTreeTile / copies;                  // rows of a copy, and columns it takes
      const int urow = two ? grp * kTreeTile + row : row & (own - 1);
      const int col = two ? 0 : row / own * own;
      const bool live = urow < seg.count;
      const bool busy = urow - lane < seg.count;           // any row of the warp
      const int token = seg.token0 + (urow >> gshift), local = seg.local0 + (urow >> gshift);
      float a = flat ? 1.f : fabsf(p.qscale);  // of a score (flat: the query is zero)
      int e_row = 14;
      // The query tile: a warp brings its 32 rows, D / 8 lanes to a row.
      if (busy) {
        constexpr int kRowLanes = D / 8, kStep = 32 / kRowLanes;  // lanes of a row, rows at once
        uint8_t* const to = smem + Shape::kQ + (two ? grp * Shape::kTileBytes : 0);
        const int ch = lane % kRowLanes, sub = lane / kRowLanes;
        auto source = [&](int i, bool* there) {
          const int r = urow - lane + i * kStep + sub;
          *there = r < seg.count && !flat;
          return p.q + (((int64_t)(seg.token0 + (r >> gshift)) * p.n_head + seg.g * p.group + (r & (p.group - 1))) * D + ch * 8) * 2;
        };
        auto target = [&](int i) { return to + chunk_at<D>((warp % 4) * 32 + i * kStep + sub, ch); };
        if (two || grp == 0) {
#pragma unroll 4
          for (int i = 0; i < kRowLanes; ++i) {
            bool there;
            const uint8_t* const from = source(i, &there);
            copy16_or_zero(smem_addr(target(i)), there ? from : p.q, there ? 16 : 0);
          }
          copy_commit();
          copy_wait<0>();
          if (EIGHT && S::kBf16) {
            // To fp16 with the row's largest element in [2^14, 2^15): the eight bits of an element of 2^-17 and more
            // are exact (2^-31 of 2^14), smaller ones err by 2^-25 (2^-39 of it). A thread its own row.
            __syncwarp();
            uint32_t top = 0;
            auto at = [&](int i) { return reinterpret_cast<uint4*>(to + chunk_at<D>(row, i)); };
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 x = *at(i);
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                           __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
            }
            top = max(top & 0xffffu, top >> 16);
            if (top != 0 && (int)(top >> 7) != 255) e_row = (int)(top >> 7) - 127;  // exponent of the largest one
            const float up = __uint_as_float((uint32_t)(min(14 - e_row, 100) + 127) << 23);
            const float more = __uint_as_float((uint32_t)(max(14 - e_row, 100) - 100 + 127) << 23);
            auto half2 = [&](uint32_t w) {
              return pack2<false>(__uint_as_float(w << 16) * up * more, __uint_as_float(w & 0xffff0000u) * up * more);
            };
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 x = *at(i);
              *at(i) = make_uint4(half2(x.x), half2(x.y), half2(x.z), half2(x.w));
            }
            if (!two) c->exponent[row] = (int16_t)e_row;
            __syncwarp();
          }
          if (negate) {
            for (int i = 0; i < kRowLanes; ++i) {
              uint4* const at = reinterpret_cast<uint4*>(target(i));
              *at = make_uint4(at->x ^ 0x80008000u, at->y ^ 0x80008000u, at->z ^ 0x80008000u, at->w ^ 0x80008000u);
            }
          }
        }
      }
      if (EIGHT && S::kBf16 && !two) {
        named_barrier_sync<1, 256>();  // the groups share the query tile
        e_row = c->exponent[row];
      }
      if constexpr (EIGHT && S::kBf16)
        a = a / __uint_as_float((uint32_t)(min(14 - e_row, 100) + 127) << 23) /
            __uint_as_float((uint32_t)(max(14 - e_row, 100) - 100 + 127) << 23);
      fence_proxy_async_shared();
      mbar_arrive(&c->q_full);

      // Scales of 16 rows, in lanes 0 to 7, are on their way an item ahead, their pages' numbers two.
      const int32_t* const table = p.table + (int64_t)seg.b * p.max_pages;
      auto page_of = [&](int u) {
        const int j = (seg.t0 + (two ? u >> 1 : u)) * kTreeTile + lane * 16;
        return u < items && lane < 8 && j < seg.rows ? table[j >> p.page_shift] : -1;
      };
      int id_next = -1;
      float k_next = 0.f, v_next = 0.f;
      auto scales_of = [&](int id) {
        const bool fine = id >= 0 && id < p.num_pages;
        const int64_t at = (int64_t)id * p.n_kv_head + seg.g;
        k_next = fine ? p.k_scale[at] : 0.f;
        v_next = fine ? p.v_scale[at] : 1.f;
        if (!fine) k_next = 1.f;  // (columns that nobody sees)
      };
      if constexpr (EIGHT) {
        scales_of(page_of(grp));
        id_next = page_of(grp + 2);
      }
      const bool whole = seg.t0 == 0 && seg.t1 == seg.kt;
      TreePending part;
      if (threadIdx.x == 0 && !whole) {
        // where the CTAs of the unit meet
        // (the last CTA whose share begins at or before a place in the list)
        auto owner = [&](int64_t place) { return (int)(((place + 1) * ctas + total - 1) / total) - 1; };
        if (part_tiles > 0) {
          part.c0 = blockIdx.x - c->piece;
          part.parts = c->pieces;
        } else {
          part.c0 = seg.t0 == 0 ? (int)blockIdx.x : owner((int64_t)unit_at + kTreeUnitTiles);
          part.parts = owner((int64_t)unit_at + kTreeUnitTiles + seg.kt - 1) - part.c0 + 1;
        }
        part.rows = seg.count;
        part.token0 = seg.token0;
        part.g = seg.g;
        part.generation = *reinterpret_cast<volatile unsigned*>(&meets[part.c0].generation);
      }
      TreeState st = {-INFINITY, -INFINITY, 0.f};
      for (int u = grp; u < items; u += 2) {
        const int t = seg.t0 + (two ? u >> 1 : u), j0 = t * kTreeTile;
        const bool masked = j0 + kTreeTile > seg.base;
        float sign = 1.f;
        bool plain = true;
        if constexpr (EIGHT) {
          sign = v_next == 0.f ? 0.f : v_next < 0.f ? -1.f : 1.f;
          plain = __all_sync(0xffffffffu, lane >= 8 || (k_next > 0.f && sign == 1.f));
          __syncwarp();
          if (lane < 8) c->scales[warp][lane] = make_float2(k_next, log2f(fabsf(v_next)));
          __syncwarp();
          scales_of(id_next);
          id_next = page_of(u + 4);
        }
        uint32_t seen[4] = {0u, 0u, 0u, 0u};
        if (masked && live) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (32 * k < own) seen[k] = seen_bits(p, seg, token, local, j0 + col + 32 * k);
        }
        if constexpr (!EIGHT) {
          // V rows behind the last one become zero, elements of drafted rows that are not finite too: they are added at
          // the end for those who see them. (Before the wait for the scores, which are being made meanwhile.)
          if (masked && !dead && (!two || grp == 0)) {
            const int use = 2 * (tau + t - seg.t0) + 1, slot = use % Shape::kSlots, j = j0 + row;
            const int valid = min(kTreeTile, seg.rows - j0);
            if (row < (valid + 15) / 16 * 16 && j >= seg.base) {
              if (!tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1)) dead = true;
              uint8_t* const v = smem + Shape::kRing + slot * Shape::kTileBytes;
              auto at = [&](int i) { return reinterpret_cast<uint4*>(v + chunk_at<D>(row, i)); };
              if (row >= valid) {
                for (int i = 0; i < D / 8; ++i) *at(i) = make_uint4(0u, 0u, 0u, 0u);
              } else {
                // (an exponent of ones, and one more, carries into the sign's place)
                constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u, kOne = kBf16 ? 0x00800080u : 0x04000400u;
                uint32_t bad = 0;
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                  const uint4 x = *at(i);
                  bad |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
                }
                if (bad & 0x80008000u) {
                  for (int i = 0; i < D / 8; ++i) {
                    const uint4 x = *at(i);
                    *at(i) = make_uint4(x.x & finite_pair_mask<kBf16>(x.x), x.y & finite_pair_mask<kBf16>(x.y),
                                        x.z & finite_pair_mask<kBf16>(x.z), x.w & finite_pair_mask<kBf16>(x.w));
                  }
                  const int d = j - seg.base;
                  atomicOr(&c->bad[s & 7][d >> 5], 1u << (d & 31));
                }
              }
              fence_proxy_async_shared();
            }
            dead = __any_sync(0xffffffffu, dead);
          }
        }
        if (!dead) dead = !__all_sync(0xffffffffu, tree_wait(c, p, &c->s_full[grp], phase_s & 1));
        ++phase_s;
        if (dead) continue;
        tc_fence_after();
        if (busy) {
          auto columns = [&](auto cols, auto pieces) {
            constexpr int kCols = decltype(cols)::value, kPieces = decltype(pieces)::value;
            const float2* const scales = c->scales[warp];
            if (!EIGHT || plain) {
              softmax_columns<kBf16, D, EIGHT, kCols, kPieces, true>(st, s_at, p_at, o_at, col, u < 2, a, masked, seen, scales, sign);
            } else {
              softmax_columns<kBf16, D, EIGHT, kCols, kPieces, !EIGHT>(st, s_at, p_at, o_at, col, u < 2, a, masked, seen, scales, sign);
            }
          };
          using std::integral_constant;
          constexpr integral_constant<int, kBf16 && Shape::kTwoPieces ? 2 : 1> kPieces;
          if (two) {
            columns(integral_constant<int, 128>(), integral_constant<int, 1>());
          } else if (copies == 1) {
            columns(integral_constant<int, 128>(), kPieces);
          } else if (copies == 2) {
            columns(integral_constant<int, 64>(), kPieces);
          } else {
            columns(integral_constant<int, 32>(), kPieces);
          }
        }
        tc_fence_before();
        mbar_arrive(&c->p_full[grp]);
      }

      // ---- the segment's output ----
      if constexpr (EIGHT) st.m -= kTreeLift;  // (of which l knows nothing)
      if (!dead) dead = !__all_sync(0xffffffffu, tree_wait(c, p, &c->o_final, s & 1));
      tc_fence_after();
      const bool nan = dead || c->bad_page[s & 7] != 0;
      float* const slot = partials + ((int64_t)blockIdx.x * 2 + (seg.t0 == 0 ? 1 : 0)) * tree_slot_floats(D);
      // Values of drafted V rows that are not finite, for a row that sees them: columns [at, at + 32) of o.
      auto add_bad = [&](uint32_t (&o)[32], int at) {
        for (int k = 0; k < 8; ++k) {
          uint32_t left = c->bad[s & 7][k];
          if (left) left &= draft_bits(p, token, local, seg.rows - seg.base, 32 * k);
          for (; left; left &= left - 1) {
            const int j = seg.base + 32 * k + __ffs(left) - 1;
            if (j < seg.t0 * kTreeTile || j >= seg.t1 * kTreeTile) continue;
            const int id = table[j >> p.page_shift];
            if (id < 0 || id >= p.num_pages) continue;
            const int64_t from = (((int64_t)id * p.n_kv_head + seg.g) * p.page_rows + (j & (p.page_rows - 1))) * D + at;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float x;
              if constexpr (EIGHT) {
                x = (p.v[from + i] & 0x7f) == 0x7f ? NAN : 0.f;
              } else {
                x = (float)reinterpret_cast<const T*>(p.v)[from + i];
              }
              if (!(fabsf(x) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
            }
          }
        }
      };
      bool any_bad = false;
#pragma unroll
      for (int k = 0; k < 8; ++k) any_bad |= c->bad[s & 7][k] != 0;
      // The state of the row: this thread's own (two), or that of both groups and of the copies.
      float4* const states = reinterpret_cast<float4*>(smem + Shape::kStates);
      float* const inverse = reinterpret_cast<float*>(states + 2 * kTreeTile);
      float m = st.m, ml = st.ml, l = st.l, w0 = 1.f, w1 = 0.f;
      if (!two) {
        const int groups = tiles > 1 ? 2 : 1;
        states[grp * kTreeTile + row] = make_float4(st.m, st.ml, st.l, 0.f);
        named_barrier_sync<1, 256>();
        m = ml = -INFINITY;
        l = 0.f;
        for (int i = urow; i < groups * kTreeTile; i += own) {
          m = fmaxf(m, states[i].x);
          ml = fmaxf(ml, states[i].y);
        }
        const float m0 = m == -INFINITY ? 0.f : m, ml0 = ml == -INFINITY ? 0.f : ml;
        for (int i = urow; i < groups * kTreeTile; i += own) l += states[i].z * fast_exp2(states[i].y - ml0);
        w0 = fast_exp2(states[row].x - m0);
        w1 = groups > 1 ? fast_exp2(states[kTreeTile + row].x - m0) : 0.f;
      }
      const float inv = nan ? NAN : l == 0.f ? 0.f : (EIGHT ? fast_exp2(m - ml) : 1.f) / l;
      const bool first_copy = two || row < own;
      if (two || (grp == 0 && first_copy)) {
        inverse[urow] = inv;
        if (live && !whole) reinterpret_cast<float4*>(slot + kTreeUnitRows * D)[urow] = make_float4(m, ml, nan ? NAN : l, 0.f);
      }
      named_barrier_sync<1, 256>();
      // 32 columns at a time through shared memory, so that rows are written in whole lines: of its own group's output
      // (two), or of both groups' for half of the columns; copies are summed on the way out.
      uint8_t* const exchange = smem + Shape::kExchange + (grp * kTreeTile) * 128;  // rows of this group
      const int c0 = two ? 0 : grp * (D / 2), c1 = two ? D : c0 + D / 2;
      const uint32_t o0 = two ? o_at : tmem + lanes + Shape::kO;
      // 8 bits: a warp's own rows of a partial state leave by a bulk copy. (256 rows of 128 by the threads' stores, and
      // the wait for them at the arrival, took 15 000 cycles; what an SM can write takes 5 900. With copies, and four
      // parts of a join on their way: 98 -> 94 us, 4 x 16384 of 64/8 heads, 32 drafts. 16-bit pages gained 1 us of 47
      // where rows are many and lost 0.4 to 2 us where they are few.)
      const bool copied = EIGHT && !whole && (two || copies == 1);
#pragma unroll 1
      for (int at = c0; at < c1; at += 32) {
        if (copied && lane == 0) bulk_wait_read();
        if (busy) {
          uint32_t o[32], o1[32];
          __syncwarp();
          if (!dead) {
            tmem_load32(o0 + at, o);
            if (!two && tiles > 1) tmem_load32(o0 + D + at, o1);
            tmem_wait_load();
          }
          if (!two) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * w0);
            if (tiles > 1) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), w1, __uint_as_float(o[i])));
            }
          }
          if (any_bad && live && first_copy) add_bad(o, at);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(exchange + row * 128 + ((i ^ (row & 7)) << 4)) =
                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if (copied) {
          const int first = (two ? grp * kTreeTile : 0) + row - lane;
          if (first < seg.count) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) bulk_store(slot + tree_slot_at<D, EIGHT>(first, at), exchange + (row - lane) * 128, 32 * 128);
          }
          continue;
        }
        if (two || copies == 1) __syncwarp(); else if (grp == 0) named_barrier_sync<3, 128>(); else named_barrier_sync<4, 128>();
        // (a warp's own rows, or the group's first copy)
        const bool alone = two || copies == 1;
        const int th = alone ? lane : (int)threadIdx.x % 128, ch = th % 8, step = alone ? 4 : 16;
        const int r0 = (alone ? row - lane : 0) + th / 8, rows = alone ? 32 : own;
        auto emit = [&](int r, float4 sum) {
          const int ur = (two ? grp * kTreeTile : 0) + r;
          if (ur >= seg.count) return;
          if (whole) {
            const float f = inverse[ur];
            const int64_t to = ((int64_t)(seg.token0 + (ur >> gshift)) * p.n_head + seg.g * p.group + (ur & (p.group - 1))) * D;
            *reinterpret_cast<uint2*>(p.out + (to + at + 4 * ch) * 2) =
                make_uint2(pack2<S::kBf16>(sum.x * f, sum.y * f), pack2<S::kBf16>(sum.z * f, sum.w * f));
          } else {
            *reinterpret_cast<float4*>(slot + tree_slot_at<D, EIGHT>(ur, at + 4 * ch)) = sum;
          }
        };
        auto place = [&](int r) { return *reinterpret_cast<const float4*>(exchange + r * 128 + ((ch ^ (r & 7)) << 4)); };
        if (alone) {
          float4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = place(r0 + 4 * i);
#pragma unroll
          for (int i = 0; i < 8; ++i) emit(r0 + 4 * i, x[i]);
        } else {
          for (int r = r0; r < rows; r += step) {
            float4 sum = place(r);
            for (int k = r + own; k < kTreeTile; k += own) {
              const float4 x = place(k);
              sum.x += x.x;
              sum.y += x.y;
              sum.z += x.z;
              sum.w += x.w;
            }
            emit(r, sum);
          }
        }
        if (two || copies == 1) __syncwarp(); else if (grp == 0) named_barrier_sync<3, 128>(); else named_barrier_sync<4, 128>();
      }
      if (copied && lane == 0) bulk_wait();
      tc_fence_before();
      named_barrier_sync<2, 256>();  // the states, and the notes on the segment's rows, have been read
      if (threadIdx.x < 8) c->bad[s & 7][threadIdx.x] = 0;
      if (threadIdx.x == 0) c->bad_page[s & 7] = 0;
      mbar_arrive(&c->o_free);
      if (!whole && threadIdx.x == 0) {
        // this CTA's part of the unit is written: arrive where its CTAs meet
        TreeMeet* const meet = meets + part.c0;
        const unsigned before = arrive_acq_rel(arrived + part.c0);
        part.last = before + 1 == (unsigned)part.parts;
        if (part.last) {
          arrived[part.c0] = 0;
          meet->ticket = 0;
          store_release(&meet->generation, part.generation + 1);
        } else if (before >= (unsigned)part.parts) {
          // nobody can tell when the unit's parts are written: its rows become NaN (the counter stays as it is, so that
          // every later call on it says so too)
          if (p.err_flag) atomicOr(p.err_flag, kErrWorkspace);
          part.parts = 0;
          part.last = 1;
        }
        c->pending[c->pendings++] = part;
      }
      if (seg.t1 == seg.kt) unit_at += seg.kt + kTreeUnitTiles;
      tau += tiles;
    }
    named_barrier_sync<2, 256>();
    const int pendings = c->pendings;
    for (int i = 0; i < pendings; ++i) {
      const TreePending x = c->pending[i];
      TreeMeet* const meet = meets + x.c0;
      const bool alone = x.rows <= kTreeAloneRows || x.parts == 0;  // few rows: the last to arrive joins them, nobody waits
      named_barrier_sync<1, 256>();
      if (threadIdx.x == 0) {
        // The last to arrive joins the unit. The others wait for it a while, to help: it does without them, so that no
        // CTA depends on another one being there.
        bool ready = x.last;
        const unsigned long long t0 = global_ns();
        while (!alone && !ready && global_ns() - t0 < kTreeHelpNs) ready = load_acquire(&meet->generation) != x.generation;
        c->ready = ready;
      }
      named_barrier_sync<1, 256>();
      if (!c->ready) continue;
      if (alone) {
        tree_join_rows<T, D, EIGHT>(p, partials, x, 0, x.rows, reinterpret_cast<float*>(smem + Shape::kExchange));
        continue;
      }
      const int share = max(16, ((x.rows + x.parts - 1) / x.parts + 7) & ~7), shares = (x.rows + share - 1) / share;
      for (;;) {
        if (threadIdx.x == 0) c->ticket = (int)atomicAdd(&meet->ticket, 1u);
        named_barrier_sync<1, 256>();
        const int ticket = c->ticket;
        named_barrier_sync<1, 256>();
        if (ticket >= shares) break;
        // (weights: at most max(16 parts, rows + 8 parts) + rows floats)
        tree_join_rows<T, D, EIGHT>(p, partials, x, ticket * share, min(x.rows, (ticket + 1) * share),
                             reinterpret_cast<float*>(smem + Shape::kExchange));
      }
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

}  // namespace da
