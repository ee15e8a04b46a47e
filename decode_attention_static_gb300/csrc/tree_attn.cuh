// Attention of several new tokens of each sequence over a paged cache: one pass
// over K and V on the fifth-generation tensor cores.
//
// The query rows that share a KV head (its G heads for each token) are the rows of
// the products: 128 to a tile, row = token * G + head. A unit is (sequence, KV
// head, 256 query rows) over all tiles of 128 cache rows; the launch's CTAs (one
// an SM) take equal runs of the tiles of all units, whatever the lengths, and a
// unit that several CTAs take is joined from their partial states by a second
// small kernel (tree_attn.cu).
//
//   warps 0-7   two groups of 128 threads, a query row each: softmax with a
//               running maximum, weights to tensor memory, output
//   warp 8      page numbers and copies of K and V tiles into a ring
//   warp 9      the products: S = Q K^T (both in shared memory), O += P V (P in
//               tensor memory, V in shared memory as it lies, read transposed)
//   warps 10-13 8-bit pages: e4m3 to fp16 (exact), raw ring to operand ring
//
// Units of more than 128 rows ("two") give each group its own query tile and every
// K and V tile is used twice; smaller ones share the query tile, the groups take
// the cache tiles in turn, each with its own state, and join them at the end. So
// one group's exponentials run under the other's products.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "tree_params.h"

namespace da {

constexpr int kTreeTile = 128;             // cache rows of a tile, query rows of a tile
constexpr int kTreeUnitRows = 256;         // query rows of a unit
constexpr float kTreeLazy = 8.f;           // a running maximum is raised when a score passes it by 2^8

// A partial state: O [2][D / 4][128] float4, then (m, m of l, l) [256] float4.
__host__ __device__ constexpr int tree_slot_floats(int D) { return kTreeUnitRows * D + kTreeUnitRows * 4; }
// What the merge needs of a unit that several CTAs take, by the CTA that begins it.
struct TreeJoin {
  int token0;   // first packed token of the unit
  int rows;     // query rows (0: nothing to join)
  int g;        // KV head
  int last;     // the last CTA of the unit
};

struct alignas(64) TreeLaunch {
  TensorMap k_map, v_map;  // 16-bit pages as rows of D elements; boxes of a page's rows (at most 128) by 64
  TreeParams p;
};

cudaError_t launch_tree_f16(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, TreeJoin* joins, float* partials,
                            cudaStream_t stream);
cudaError_t launch_tree_bf16(const TreeLaunch& l, int head_dim, bool e4m3, int ctas, TreeJoin* joins, float* partials,
                             cudaStream_t stream);

template <int D, bool EIGHT>
struct TreeShape {
  static constexpr int kBlocks = D / 64;                   // 64-column blocks of an operand tile
  static constexpr int kBlockBytes = kTreeTile * 128;
  static constexpr int kTileBytes = kBlocks * kBlockBytes; // 16-bit operand tile
  static constexpr int kRawBytes = kTreeTile * D;          // e4m3 tile
  static constexpr int kSlots = EIGHT ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  static constexpr int kRaw = EIGHT ? (D == 128 ? 4 : 6) : 0;
  static constexpr int kThreads = EIGHT ? 448 : 320;
  static constexpr int kQ = 0, kRing = 2 * kTileBytes, kRawRing = kRing + kSlots * kTileBytes;
  static constexpr int kControl = kRawRing + kRaw * kRawBytes;
  static constexpr int kSmem = 1024 + kControl + 2048;
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
  int start_b, start_off;
  int sums[16];
  // of segment s, in entry s % 8: drafted rows whose V is not finite, and whether a page lies outside the pool
  uint32_t bad[8][8];
  int bad_page[8];
};
static_assert(sizeof(TreeControl) <= 2048, "control area");

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

  __device__ __forceinline__ void begin(const TreeParams& p, int b0, int off, int tiles) {
    left = tiles;
    if (tiles == 0) return;
    int none = 0;
    b = b0;
    s = tree_sequence(p, b, &none);
    const int unit = off / s.kt;
    tile = off - unit * s.kt;
    g = unit / s.mps;
    mp = unit - g * s.mps;
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
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (tensor memory) = A (tensor memory) B (+ D), issued by one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred acc;\n\tsetp.ne.b32 acc, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, acc;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
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

// A row's softmax state: m for the output and the weights, ml for l (they differ with scales of V).
struct TreeState {
  float m, ml, l;
};

template <typename T, int D, bool EIGHT>
__global__ void __launch_bounds__(TreeShape<D, EIGHT>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeLaunch launch, TreeJoin* joins, float* partials) {
  using Shape = TreeShape<D, EIGHT>;
  using S = Storage<T>;
  constexpr bool kBf16 = S::kBf16 && !EIGHT;  // type of the products
  // fp16 weights are held 2^7 times as large: the largest one of a row lies in [2^7, 2^15]
  constexpr float kLift = kBf16 ? 0.f : 7.f;
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
      mbar_init(&c->full[i], EIGHT ? 128 : 1);
      mbar_init(&c->empty[i], 1);
      mbar_init(&c->raw_full[i], 1);
      mbar_init(&c->raw_empty[i], 128);
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

  // This CTA's share of all tiles, and where it begins.
  int errors = 0, begin = 0, end = 0, total = 0;
  {
    auto tiles_of = [&](int b) {
      if (b >= p.B) return 0;
      const TreeSeq s = tree_sequence(p, b, &errors);
      return p.n_kv_head * s.mps * s.kt;
    };
    const int mine = tiles_of(threadIdx.x);
    int sum = mine;
    for (int b = threadIdx.x + kThreads; b < p.B; b += kThreads) sum += tiles_of(b);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) c->sums[warp] = sum;
    __syncthreads();
    total = __reduce_add_sync(0xffffffffu, lane < kWarps ? c->sums[lane] : 0);
    const int ctas = min((int)gridDim.x, total);
    if ((int)blockIdx.x < ctas) {
      begin = (int)((int64_t)total * blockIdx.x / ctas);
      end = (int)((int64_t)total * (blockIdx.x + 1) / ctas);
    }
    int before = 0;
    for (int base = 0; base < p.B && before <= begin && end > 0; base += kThreads) {
      const int v = base == 0 ? mine : tiles_of(base + threadIdx.x);
      int scan = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
      }
      __syncthreads();
      if (lane == 31) c->sums[warp] = scan;
      __syncthreads();
      const int w = lane < kWarps ? c->sums[lane] : 0;
      const int at = before + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + scan - v;
      if (begin >= at && begin < at + v) {
        c->start_b = base + threadIdx.x;
        c->start_off = begin - at;
      }
      before += __reduce_add_sync(0xffffffffu, w);
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && errors && p.err_flag) atomicOr(p.err_flag, errors);
  TreeCursor cursor;
  cursor.begin(p, c->start_b, c->start_off, end - begin);
  TreeSegment seg;

  if (warp == 8) {
    // ---------------- producer ----------------
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
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(on) * step * row_bytes);
          __syncwarp();
          if constexpr (EIGHT) {
            if (lane < pages && fine) {
              const int64_t row = ((int64_t)id * p.n_kv_head + seg.g) * p.page_rows + ((j0 + lane * step) & (p.page_rows - 1));
              bulk_load_plain(smem + Shape::kRawRing + stage * Shape::kRawBytes + lane * step * D, pools[kv] + row * D,
                              step * D, &full[stage]);
            }
          } else {
            const int page = lane / Shape::kBlocks, block = lane % Shape::kBlocks;
            const int at = __shfl_sync(0xffffffffu, id, page);
            if (page < pages && (on >> page & 1)) {
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
    if (lane == 0) {
      constexpr uint32_t kScores = tree_idesc(kBf16, kTreeTile, false), kOut = tree_idesc(kBf16, D, true);
      int tau = 0, phase_p[2] = {0, 0};
      bool ok = true;
      for (int s = 0; ok && cursor.next(p, &seg); ++s) {
        const bool two = seg.count > kTreeTile;
        const int tiles = seg.t1 - seg.t0, items = two ? 2 * tiles : tiles;
        ok = tree_wait(c, p, &c->q_full, s & 1);
        for (int u = 0; ok && u <= items; ++u) {
          if (u < items) {
            const int use = 2 * (tau + (two ? u >> 1 : u)), slot = use % Shape::kSlots;
            if (!two || !(u & 1)) ok = tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t a = sw128_desc_at(q_tiles + (two ? (u & 1) * Shape::kTileBytes : 0));
            const uint64_t b = sw128_desc_at(ring + slot * Shape::kTileBytes);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint64_t off = (uint64_t)(((k / 4) * Shape::kBlockBytes + (k % 4) * 32) >> 4);
              mma_f16_ss(tmem + Shape::kS + (u & 1) * 128, a + off, b + off, kScores, k > 0);
            }
            mma_commit(&c->s_full[u & 1]);
            if (!two || (u & 1)) mma_commit(&c->empty[slot]);
          }
          if (u > 0) {
            const int v = u - 1, grp = v & 1, t = two ? v >> 1 : v;
            const int use = 2 * (tau + t) + 1, slot = use % Shape::kSlots;
            if (v == 0 && s > 0) ok = tree_wait(c, p, &c->o_free, (s - 1) & 1);
            if (ok) ok = tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1);
            if (ok) ok = tree_wait(c, p, &c->p_full[grp], phase_p[grp] & 1);
            if (!ok) break;
            ++phase_p[grp];
            tc_fence_after();
            const int steps = (min(kTreeTile, seg.rows - (seg.t0 + t) * kTreeTile) + 15) / 16;
            const uint64_t b = sw128_desc_rows(ring + slot * Shape::kTileBytes, Shape::kBlockBytes);
            for (int k = 0; k < steps; ++k)
              mma_f16_ts(tmem + Shape::kO + grp * D, tmem + Shape::kP + grp * Shape::kPStride + k * 8,
                         b + (uint64_t)((k * 2048) >> 4), kOut, v >= 2 || k > 0);
            if (!two || (v & 1)) mma_commit(&c->empty[slot]);
          }
        }
        if (!ok) break;
        mma_commit(&c->o_final);
        mbar_arrive(&c->o_final);
        tau += tiles;
      }
      if (!ok) {
        // products in flight end before the memory is freed (bounded)
        mma_commit(&c->drain);
        mbar_wait(&c->drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---------------- e4m3 to fp16 ----------------
    if constexpr (EIGHT) {
      const int th = threadIdx.x - 320;
      constexpr int kChunks = D / 16;  // 16-byte chunks of a raw row, and of a thread
      int use = 0;
      bool ok = true;
      for (int s = 0; ok && cursor.next(p, &seg); ++s) {
        for (int t = seg.t0; ok && t < seg.t1; ++t) {
          const int j0 = t * kTreeTile, valid = min(kTreeTile, seg.rows - j0);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++use) {
            const int raw = use % Shape::kRaw, slot = use % Shape::kSlots, round = use / Shape::kSlots;
            ok = tree_wait(c, p, &c->raw_full[raw], (use / Shape::kRaw) & 1);
            if (ok && round > 0) ok = tree_wait(c, p, &c->empty[slot], (round - 1) & 1);
            if (!ok) break;
            const uint8_t* const from = smem + Shape::kRawRing + raw * Shape::kRawBytes;
            uint8_t* const to = smem + Shape::kRing + slot * Shape::kTileBytes;
            const bool special = kv == 1 && j0 + kTreeTile > seg.base;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
              const int idx = th + i * 128, r = idx / kChunks, ch = idx % kChunks;
              uint4 x = ld_shared_v4(from + idx * 16);
              if (special) {
                uint32_t* const w = &x.x;
                if (r >= valid) {
                  x = make_uint4(0u, 0u, 0u, 0u);
                } else if (j0 + r >= seg.base) {
                  // drafted rows: NaN reaches only those who see it (added at the end)
                  bool nan = false;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t m = __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    nan |= m != 0;
                    w[k] &= ~m;
                  }
                  const int d = j0 + r - seg.base;
                  if (nan) atomicOr(&c->bad[s & 7][d >> 5], 1u << (d & 31));
                }
              }
              uint32_t h[8];
              const uint32_t* const w = &x.x;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * k]) : "h"((uint16_t)(w[k] & 0xffffu)));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[2 * k + 1]) : "h"((uint16_t)(w[k] >> 16)));
              }
              *reinterpret_cast<uint4*>(to + chunk_at<D>(r, 2 * ch)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(to + chunk_at<D>(r, 2 * ch + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
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
    const int grp = warp / 4, row = (warp % 4) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_at = tmem + lanes + Shape::kS + grp * 128, p_at = tmem + lanes + Shape::kP + grp * Shape::kPStride;
    const uint32_t o_at = tmem + lanes + Shape::kO;  // outputs of group 0; of group 1 D columns on
    const float qscale = fabsf(p.qscale);
    const bool negate = p.qscale < 0.f;
    int phase_s = 0, tau = 0;
    bool dead = false;
    for (int s = 0; cursor.next(p, &seg); ++s) {
      const bool two = seg.count > kTreeTile;
      const int tiles = seg.t1 - seg.t0, items = two ? 2 * tiles : tiles;
      const int urow = (two ? grp * kTreeTile : 0) + row;  // row of the unit
      const bool live = urow < seg.count;
      const bool busy = urow - lane < seg.count;           // any row of the warp
      const int token = seg.token0 + urow / p.group, local = seg.local0 + urow / p.group;
      const int head = seg.g * p.group + urow % p.group;
      const int64_t out_row = ((int64_t)token * p.n_head + head) * D;
      float a = qscale;  // of a score
      // the query tile
      if (busy) {
        const uint4* const from = reinterpret_cast<const uint4*>(p.q + out_row * 2);
        uint8_t* const to = smem + Shape::kQ + (two ? grp * Shape::kTileBytes : 0);
        const bool writes = two || grp == 0;
        uint4 x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = live ? ld_global_nc_v4(from + i) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t* const w = &x[0].x;
        if constexpr (EIGHT && S::kBf16) {
          // to fp16 with the row's largest element in [2^14, 2^15): exact above 2^-39 of it
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < D / 2; ++i) top = max(top, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
          int e = (int)(top >> 7) - 127;  // exponent of the largest one
          if (top == 0 || e == 128) e = 14;
          const float up = __uint_as_float((uint32_t)(min(14 - e, 100) + 127) << 23);
          const float more = __uint_as_float((uint32_t)(max(14 - e, 100) - 100 + 127) << 23);
#pragma unroll
          for (int i = 0; i < D / 2; ++i)
            w[i] = pack2<false>(__uint_as_float(w[i] << 16) * up * more, __uint_as_float(w[i] & 0xffff0000u) * up * more);
          a = a / up / more;
        }
        if (negate) {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) w[i] ^= 0x80008000u;
        }
        if (writes) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) *reinterpret_cast<uint4*>(to + chunk_at<D>(row, i)) = x[i];
        }
      }
      fence_proxy_async_shared();
      mbar_arrive(&c->q_full);

      TreeState st = {-INFINITY, -INFINITY, 0.f};
      for (int u = grp; u < items; u += 2) {
        const int t = seg.t0 + (two ? u >> 1 : u), j0 = t * kTreeTile;
        const bool masked = j0 + kTreeTile > seg.base;
        float sk = 0.f, lv = 0.f, sv = 1.f;  // scales of 16 rows, in lanes 0 to 7
        if constexpr (EIGHT) {
          if (lane < 8 && j0 + lane * 16 < seg.rows) {
            const int id = p.table[(int64_t)seg.b * p.max_pages + ((j0 + lane * 16) >> p.page_shift)];
            if (id >= 0 && id < p.num_pages) {
              const int64_t at = (int64_t)id * p.n_kv_head + seg.g;
              sk = p.k_scale[at];
              const float v = p.v_scale[at];
              lv = v == 0.f ? 0.f : log2f(fabsf(v));
              sv = v == 0.f ? 0.f : v < 0.f ? -1.f : 1.f;
            }
          }
        }
        uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (masked) {
#pragma unroll
          for (int k = 0; k < 4; ++k) seen[k] = live ? seen_bits(p, seg, token, local, j0 + 32 * k) : 0u;
        }
        if (!dead) dead = !__all_sync(0xffffffffu, tree_wait(c, p, &c->s_full[grp], phase_s & 1));
        ++phase_s;
        if (dead) continue;
        tc_fence_after();
        if (busy) {
          uint32_t r[EIGHT ? 32 : 128];
          float m_tile = -INFINITY, ml_tile = -INFINITY;
          if constexpr (!EIGHT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_load32(s_at + 32 * k, r + 32 * k);
            tmem_wait_load();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 128; ++i)
                if (!(seen[i / 32] >> (i % 32) & 1)) r[i] = 0xff800000u;
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 128; ++i) top[i % 4] = fmaxf(top[i % 4], __uint_as_float(r[i]));
            const float top1 = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            m_tile = top1 == -INFINITY ? -INFINITY : top1 * a;
            ml_tile = m_tile;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tmem_load32(s_at + 32 * k, r);
              tmem_wait_load();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float ak = a * __shfl_sync(0xffffffffu, sk, 2 * k + h);
                const float vk = __shfl_sync(0xffffffffu, lv, 2 * k + h);
                const uint32_t bits = seen[k] >> (16 * h) & 0xffffu;
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float x = __uint_as_float(r[16 * h + i]) * ak;
                  top = fmaxf(top, !masked || (bits >> i & 1) ? x : -INFINITY);
                }
                ml_tile = fmaxf(ml_tile, top);
                m_tile = fmaxf(m_tile, top + vk);
              }
            }
          }
          // raise the maximum where a score passes it by 2^8 (or is the first one)
          const bool up = m_tile > st.m + kTreeLazy || (st.m == -INFINITY && m_tile > -INFINITY);
          if (__any_sync(0xffffffffu, up)) {
            const float factor = !up ? 1.f : st.m == -INFINITY ? 0.f : fast_exp2(st.m - m_tile);
            if (up) st.m = m_tile;
            if constexpr (!EIGHT) st.l *= factor;
            if (u >= 2) {
              uint32_t o[32];
#pragma unroll
              for (int k = 0; k < D / 32; ++k) {
                tmem_load32(o_at + grp * D + 32 * k, o);
                tmem_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                tmem_store32(o_at + grp * D + 32 * k, o);
              }
            }
          }
          if constexpr (EIGHT) {
            if (ml_tile > st.ml + kTreeLazy || (st.ml == -INFINITY && ml_tile > -INFINITY)) {
              st.l *= st.ml == -INFINITY ? 0.f : fast_exp2(st.ml - ml_tile);
              st.ml = ml_tile;
            }
          } else {
            st.ml = st.m;
          }
          const float ref = st.m == -INFINITY ? 0.f : st.m - kLift;
          if constexpr (!EIGHT) {
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 128; ++i) {
              float x = fmaf(__uint_as_float(r[i]), a, -ref);
              if (masked && !(seen[i / 32] >> (i % 32) & 1)) x = -INFINITY;
              x = fast_exp2(x);
              sum[i % 4] += x;
              r[i] = __float_as_uint(x);
            }
            st.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int i = 0; i < 64; ++i)
              r[i] = pack2<kBf16>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            tmem_store32(p_at, r);
            tmem_store32(p_at + 32, r + 32);
          } else {
            const float lref = st.ml == -INFINITY ? 0.f : st.ml;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tmem_load32(s_at + 32 * k, r);
              tmem_wait_load();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float ak = a * __shfl_sync(0xffffffffu, sk, 2 * k + h);
                const float vk = __shfl_sync(0xffffffffu, lv, 2 * k + h);
                const float sg = __shfl_sync(0xffffffffu, sv, 2 * k + h);
                const uint32_t bits = seen[k] >> (16 * h) & 0xffffu;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float x = fmaf(__uint_as_float(r[16 * h + i]), ak, vk - ref);
                  if (masked && !(bits >> i & 1)) x = -INFINITY;
                  x = fast_exp2(x);
                  sum += x;
                  r[16 * h + i] = __float_as_uint(x);
                }
                // l counts the weights without the scale of V
                if (sum != 0.f) st.l += sum * fast_exp2(ref - lref - vk);
                if (sg != 1.f) {
#pragma unroll
                  for (int i = 0; i < 16; ++i) r[16 * h + i] = __float_as_uint(__uint_as_float(r[16 * h + i]) * sg);
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i)
                r[i] = pack2<false>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
              tmem_store16(p_at + 16 * k, r);
            }
          }
          tmem_wait_store();
        }
        if constexpr (!EIGHT) {
          // V rows behind the last one become zero, elements of drafted rows that are not finite too: they
          // are added at the end for those who see them
          if (masked && (!two || grp == 0)) {
            const int use = 2 * (tau + t - seg.t0) + 1, slot = use % Shape::kSlots, j = j0 + row;
            const int valid = min(kTreeTile, seg.rows - j0);
            if (row < (valid + 15) / 16 * 16 && j >= seg.base) {
              if (!tree_wait(c, p, &c->full[slot], (use / Shape::kSlots) & 1)) dead = true;
              uint8_t* const v = smem + Shape::kRing + slot * Shape::kTileBytes;
              bool bad = false;
#pragma unroll 4
              for (int i = 0; i < D / 8; ++i) {
                uint4* const at = reinterpret_cast<uint4*>(v + chunk_at<D>(row, i));
                if (row >= valid) {
                  *at = make_uint4(0u, 0u, 0u, 0u);
                } else {
                  uint4 x = *at;
                  const uint4 m = make_uint4(finite_pair_mask<kBf16>(x.x), finite_pair_mask<kBf16>(x.y),
                                             finite_pair_mask<kBf16>(x.z), finite_pair_mask<kBf16>(x.w));
                  if ((m.x & m.y & m.z & m.w) != 0xffffffffu) {
                    bad = true;
                    *at = make_uint4(x.x & m.x, x.y & m.y, x.z & m.z, x.w & m.w);
                  }
                }
              }
              const int d = j - seg.base;
              if (bad) atomicOr(&c->bad[s & 7][d >> 5], 1u << (d & 31));
              fence_proxy_async_shared();
            }
            dead = __any_sync(0xffffffffu, dead);
          }
        }
        tc_fence_before();
        mbar_arrive(&c->p_full[grp]);
      }

      // ---- the segment's output ----
      if constexpr (EIGHT) st.m -= kLift;
      if (!dead) dead = !__all_sync(0xffffffffu, tree_wait(c, p, &c->o_final, s & 1));
      tc_fence_after();
      bool nan = dead || c->bad_page[s & 7] != 0;
      const bool whole = seg.t0 == 0 && seg.t1 == seg.kt;
      float w0 = 1.f, w1 = 0.f;
      if (!two) {
        // both groups have states of the same rows: each writes half of the columns
        float4* const states = reinterpret_cast<float4*>(smem + Shape::kQ + Shape::kTileBytes);
        states[grp * kTreeTile + row] = make_float4(st.m, st.ml, st.l, 0.f);
        named_barrier_sync<1, 256>();
        const float4 x = states[row], y = states[kTreeTile + row];
        st.m = fmaxf(x.x, y.x);
        st.ml = fmaxf(x.y, y.y);
        const float m = st.m == -INFINITY ? 0.f : st.m, ml = st.ml == -INFINITY ? 0.f : st.ml;
        w0 = fast_exp2(x.x - m);
        w1 = fast_exp2(y.x - m);
        st.l = x.z * fast_exp2(x.y - ml) + y.z * fast_exp2(y.y - ml);
      }
      const int c0 = two ? 0 : grp * (D / 2), c1 = two ? D : c0 + D / 2;
      if (busy) {
        const bool second = !two && tiles > 1;
        const float inv = st.l == 0.f ? 0.f : (EIGHT ? fast_exp2(st.m - st.ml) : 1.f) / st.l;
        // which drafted rows with values that are not finite this row sees
        uint32_t bad[8], any = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          bad[k] = c->bad[s & 7][k];
          if (bad[k]) bad[k] &= draft_bits(p, token, local, seg.rows - seg.base, 32 * k);
          any |= bad[k];
        }
        float* const slot = partials + ((int64_t)blockIdx.x * 2 + (seg.t0 == 0 ? 1 : 0)) * tree_slot_floats(D);
        float4* const part = reinterpret_cast<float4*>(slot) + (two ? grp : 0) * (D / 4) * kTreeTile + row;
        for (int col = c0; col < c1; col += 32) {
          uint32_t o[32];
          __syncwarp();
          if (!dead) {
            tmem_load32(o_at + (two ? grp * D : 0) + col, o);
            tmem_wait_load();
            if (!two) {
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * w0);
              if (second) {
                uint32_t o1[32];
                tmem_load32(o_at + D + col, o1);
                tmem_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), w1, __uint_as_float(o[i])));
              }
            }
          }
          if (any && live) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              for (uint32_t left = bad[k]; left; left &= left - 1) {
                const int j = seg.base + 32 * k + __ffs(left) - 1;
                if (j < seg.t0 * kTreeTile || j >= seg.t1 * kTreeTile) continue;
                const int id = p.table[(int64_t)seg.b * p.max_pages + (j >> p.page_shift)];
                if (id < 0 || id >= p.num_pages) continue;
                const int64_t at = (((int64_t)id * p.n_kv_head + seg.g) * p.page_rows + (j & (p.page_rows - 1))) * D + col;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  float x;
                  if constexpr (EIGHT) {
                    x = (p.v[at + i] & 0x7f) == 0x7f ? NAN : 0.f;
                  } else {
                    x = (float)reinterpret_cast<const T*>(p.v)[at + i];
                  }
                  if (!(fabsf(x) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                }
              }
            }
          }
          if (live && whole) {
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = nan ? NAN : __uint_as_float(o[2 * i]) * inv, y = nan ? NAN : __uint_as_float(o[2 * i + 1]) * inv;
              h[i] = pack2<S::kBf16>(x, y);
            }
            uint4* const out = reinterpret_cast<uint4*>(p.out + (out_row + col) * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              part[(col / 4 + i) * kTreeTile] =
                  make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                              __uint_as_float(o[4 * i + 3]));
          }
        }
        if (!whole && live && c0 == 0)
          reinterpret_cast<float4*>(slot + kTreeUnitRows * D)[urow] = make_float4(st.m, st.ml, nan ? NAN : st.l, 0.f);
      }
      tc_fence_before();
      named_barrier_sync<2, 256>();  // the states, and the notes on the segment's rows, have been read
      if (threadIdx.x < 8) c->bad[s & 7][threadIdx.x] = 0;
      if (threadIdx.x == 0) c->bad_page[s & 7] = 0;
      mbar_arrive(&c->o_free);
      tau += tiles;
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);

  // What the merge has to join, as far as this CTA begins it: its last unit, if it does not finish it.
  if (threadIdx.x == 0) {
    TreeJoin join = {0, 0, 0, 0};
    TreeCursor walk;
    walk.begin(p, c->start_b, c->start_off, end - begin);
    while (walk.next(p, &seg)) {
      if (seg.t0 == 0 && seg.t1 < seg.kt) {
        const int ctas = min((int)gridDim.x, total);
        const int64_t last_tile = (int64_t)end - seg.t1 + seg.kt - 1;  // of the unit, among all tiles
        join.token0 = seg.token0;
        join.rows = seg.count;
        join.g = seg.g;
        join.last = (int)(((last_tile + 1) * ctas + total - 1) / total) - 1;
      }
    }
    joins[blockIdx.x] = join;
  }
  // Sequences that are refused: NaN rows.
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    int none = 0;
    const TreeSeq x = tree_sequence(p, b, &none);
    if (x.state >= 0) continue;
    const uint32_t n = (uint32_t)S::kNaN * 0x10001u;
    uint4* const out = reinterpret_cast<uint4*>(p.out + (int64_t)x.first * p.n_head * D * 2);
    for (int64_t i = threadIdx.x; i < (int64_t)x.n * p.n_head * (D / 8); i += kThreads) out[i] = make_uint4(n, n, n, n);
  }
}

}  // namespace da
