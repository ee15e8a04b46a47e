// Bookkeeping of a paged cache on the device: taking, sharing and releasing
// pages. Everything is whole numbers in an order that the header fixes, so that
// equal calls give equal states.
//
// Every call is one thread-block cluster: the steps (release, collect, take)
// need a barrier over all threads, and the cluster's is in hardware, without
// counters in memory or a promise that CTAs run at the same time. The bytes (a table
// entry, a count and a list entry for each page) are few; what a call
// costs is the chain of dependent loads (length, entry, count) and barriers. A
// resize that moves few pages (a step's drafts), which only the lengths say, is
// therefore left to the first CTA alone.
//
// Measured on one GB300, device time inside a graph: an empty resize 2.5 us; 64
// sequences give their drafts' pages back and take others in two calls, 8.6 us; 256
// sequences of up to 8192 rows end and begin, 24 us.
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "page_params.h"

namespace da {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kAtOnce = 4;  // entries of a lane on their way at once: a call's time is its chain of loads
constexpr int kClusterMax = 8;  // the portable size

__device__ __forceinline__ void cluster_sync() {
  cluster_arrive_release();
  cluster_wait_acquire();
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_load(const int* local, uint32_t rank) {
  uint32_t addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void report(int32_t* err_flag, int bits) {
  if (bits && err_flag) atomicOr(err_flag, bits);
}

// Threads for each of n sequences (of a pass over at most kThreads): a power of two.
__device__ __forceinline__ int team_of(int ctas, int n) {
  return 1 << (31 - __clz(ctas * kThreads / max(1, min(n, kThreads))));
}

// Sum of v over the threads before this one; in *all and *all_other the sums
// of v and `other` over all of them. Every thread takes part.
struct ScanArea {
  int v[kWarps], other[kWarps];
};
__device__ __forceinline__ int scan_threads(int v, int other, ScanArea& area, int* all, int* all_other) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  other = __reduce_add_sync(0xffffffffu, other);
  __syncthreads();  // (the last call's sums have been read)
  if (lane == 31) {
    area.v[warp] = sum;
    area.other[warp] = other;
  }
  __syncthreads();
  const int w = lane < kWarps ? area.v[lane] : 0;
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  *all = __reduce_add_sync(0xffffffffu, w);
  *all_other = __reduce_add_sync(0xffffffffu, lane < kWarps ? area.other[lane] : 0);
  return before + sum - v;
}

// Pages of a sequence before and after, and its number among the pages taken;
// of the kThreads sequences that a pass looks at.
struct Span {
  int held, wanted, rank;
};

// The sequences [first, first + kThreads): their spans into shared memory;
// returns the pages they take, and adds those they release to *released.
__device__ __forceinline__ int find_spans(const PoolParams& p, int first, int taken, Span* spans, ScanArea& area,
                                          int* released, int* errors) {
  const int b = first + threadIdx.x, most = p.max_pages << p.page_shift, size = 1 << p.page_shift;
  Span s = {0, 0, 0};
  if (b < p.B) {
    const int h = p.a[b], w = p.b[b];
    if (h < 0 || h > most || w < 0 || w > most) {
      *errors |= kErrKvLen;
    } else {
      s.held = (h + size - 1) >> p.page_shift;
      s.wanted = (w + size - 1) >> p.page_shift;
    }
  }
  int take, drop;
  s.rank = taken + scan_threads(max(0, s.wanted - s.held), max(0, s.held - s.wanted), area, &take, &drop);
  *released += drop;
  spans[threadIdx.x] = s;
  __syncthreads();
  return take;
}

// A page whose count has just become zero is marked by a count of kFreed (or
// near it, where it is released once too often in the same call) until it is listed.
constexpr int kFreed = INT32_MIN / 2;
__device__ __forceinline__ bool just_freed(int count) { return count < kFreed / 2; }

// Pages that a resize releases and takes at most for it to be the first CTA's alone.
constexpr int kSoloReleases = kThreads, kSoloTakes = 4 * kThreads;

__global__ void __launch_bounds__(kThreads) resize_kernel(const PoolParams p, int ctas) {
  __shared__ Span spans[kThreads];
  __shared__ ScanArea area;
  __shared__ int listed;
  __shared__ __align__(16) int freed[kSoloReleases + 4];  // the first CTA alone: pages that became free
  const int lane = threadIdx.x % 32;
  int cta = ctas > 1 ? (int)cluster_rank() : 0;
  pdl_wait();
  pdl_trigger();
  int32_t* const counts = p.pool + kPoolHeader;
  int32_t* const list = counts + p.num_pages;
  int errors = 0, released = 0, taken = 0;
  const int free_now = __ldcg(p.pool);
  const int free0 = min(max(free_now, 0), p.num_pages);
  if (free0 != free_now) errors |= kErrPool;
  bool solo = false;
  if (p.B <= kThreads) {
    taken = find_spans(p, 0, 0, spans, area, &released, &errors);
    solo = released <= kSoloReleases && taken <= kSoloTakes;  // (the same in every CTA)
    if (solo) {
      if (cta > 0) return;
      ctas = 1;
    }
  }
  auto barrier = [&]() {
    if (ctas > 1) cluster_sync(); else __syncthreads();
  };
  if (threadIdx.x == 0) listed = 0;
  barrier();  // every CTA has read the free pages
  // as many threads for a sequence as there are for each of a pass
  const int thread = cta * kThreads + threadIdx.x, team = team_of(ctas, p.B), mine = thread / team, at0 = thread % team;
  // releases
  for (int first = 0; first < p.B; first += kThreads) {
    if (p.B > kThreads) taken += find_spans(p, first, taken, spans, area, &released, &errors);
    if (mine < min(kThreads, p.B - first)) {
      const Span s = spans[mine];
      int32_t* const row = p.table + (int64_t)(first + mine) * p.max_pages;
      for (int j0 = s.wanted + at0; j0 < s.held; j0 += team * kAtOnce) {
        int id[kAtOnce], before[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int j = j0 + k * team;
          id[k] = j < s.held ? row[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          const int j = j0 + k * team;
          if (j < s.held) row[j] = -1;
          before[k] = 2;  // (nothing to do)
          if (id[k] >= 0 && id[k] < p.num_pages) {
            before[k] = atomicSub(counts + id[k], 1);
          } else if (id[k] != -1) {
            errors |= kErrPage;
          }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          if (before[k] == 1) {
            if (solo) {
              freed[atomicAdd(&listed, 1)] = id[k];
            } else {
              atomicAdd(counts + id[k], kFreed);
            }
          } else if (before[k] < 1) {
            atomicAdd(counts + id[k], 1);
            errors |= kErrPool;
          }
        }
      }
    }
    if (first + kThreads < p.B) __syncthreads();
  }
  int top = free0;
  if (solo) {
    if (released > 0) {
      __syncthreads();
      // in rising order: a page's place is the number of smaller ones
      const int n = listed, id = (int)threadIdx.x < n ? freed[threadIdx.x] : 0;
      if (threadIdx.x < 4) freed[n + threadIdx.x] = INT32_MAX;
      __syncthreads();
      int place = 0;
      if (threadIdx.x / 32 * 32 < n) {
#pragma unroll 4
        for (int i = 0; i < n; i += 4) {
          const int4 x = *reinterpret_cast<const int4*>(freed + i);
          place += (x.x < id) + (x.y < id) + (x.z < id) + (x.w < id);
        }
      }
      if ((int)threadIdx.x < n && free0 + place < p.num_pages) list[free0 + place] = id;
      if (free0 + n > p.num_pages) errors |= kErrPool;
      top = min(free0 + n, p.num_pages);
      __syncthreads();
    }
  } else if (released > 0) {
    barrier();
    // each CTA lists its part of the pool
    const int per = ((p.num_pages + ctas - 1) / ctas + kThreads - 1) / kThreads * kThreads;
    const int lo = min(p.num_pages, cta * per), hi = min(p.num_pages, lo + per);
    int found = 0;
#pragma unroll 4
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) found += just_freed(__ldcg(counts + i));
    int all, none;
    scan_threads(0, found, area, &none, &all);
    int at = free0;
    if (ctas > 1) {
      if (threadIdx.x == 0) listed = all;
      cluster_sync();
      const int n = lane < ctas ? cluster_load(&listed, lane) : 0;
      at += __reduce_add_sync(0xffffffffu, lane < cta ? n : 0);
      all = __reduce_add_sync(0xffffffffu, n);
    }
    for (int i0 = lo; i0 < hi; i0 += kThreads) {
      const int id = i0 + threadIdx.x, count = id < hi ? __ldcg(counts + id) : 0;
      const bool is = just_freed(count);
      int here;
      const int place = at + scan_threads(is, 0, area, &here, &none);
      if (is) {
        counts[id] = 0;
        if (place < p.num_pages) list[place] = id; else errors |= kErrPool;
      }
      at += here;
    }
    top = min(free0 + all, p.num_pages);
    barrier();
  }
  if (taken > 0) {
    int rank0 = 0, none = 0;
    for (int first = 0; first < p.B; first += kThreads) {
      if (p.B > kThreads) {
        __syncthreads();
        rank0 += find_spans(p, first, rank0, spans, area, &none, &none);
      }
      if (mine < min(kThreads, p.B - first)) {
        const Span s = spans[mine];
        int32_t* const row = p.table + (int64_t)(first + mine) * p.max_pages;
        for (int j0 = s.held + at0; j0 < s.wanted; j0 += team * kAtOnce) {
          int id[kAtOnce];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const int rank = s.rank + j0 + k * team - s.held;
            id[k] = j0 + k * team < s.wanted && rank < top ? __ldcg(list + top - 1 - rank) : -1;
          }
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const int j = j0 + k * team, rank = s.rank + j - s.held;
            if (j >= s.wanted) break;
            if (rank >= top) {
              errors |= kErrFull;
            } else if (id[k] < 0 || id[k] >= p.num_pages) {
              errors |= kErrPool;
              id[k] = -1;
            } else {
              atomicAdd(counts + id[k], 1);
            }
            row[j] = id[k];
          }
        }
      }
    }
  }
  if (cta == 0 && threadIdx.x == 0) p.pool[0] = top - min(taken, top);
  report(p.err_flag, errors);
  if (ctas > 1 && released > 0) cluster_sync();  // shared memory that other CTAs read is there until they have
}

// One cluster. Every CTA finds which forks are valid and how many pages those
// before each one take (bits of the children in shared memory); the warps then
// copy table rows.
__global__ void __launch_bounds__(kThreads) fork_kernel(const PoolParams p, int ctas, int words) {
  extern __shared__ uint32_t bits[];  // [words] children, [words] children of more than one fork
  __shared__ ScanArea area;
  struct Fork {
    int parent, child, rows, rank;  // rows -1: skipped
    int last;                       // the parent's part-filled page (-1: none inside the pool)
  };
  __shared__ Fork forks[kThreads];
  const int cta = ctas > 1 ? (int)cluster_rank() : 0;
  for (int i = threadIdx.x; i < 2 * words; i += kThreads) bits[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  int32_t* const counts = p.pool + kPoolHeader;
  const int32_t* const list = counts + p.num_pages;
  int errors = 0;
  const int free_now = __ldcg(p.pool);
  const int free0 = min(max(free_now, 0), p.num_pages);
  if (free0 != free_now) errors |= kErrPool;
  for (int i = threadIdx.x; i < p.n; i += kThreads) {
    const int c = p.b[i];
    if (c >= 0 && c < p.B && (atomicOr(bits + (c >> 5), 1u << (c & 31)) >> (c & 31) & 1))
      atomicOr(bits + words + (c >> 5), 1u << (c & 31));
  }
  __syncthreads();
  const int thread = cta * kThreads + threadIdx.x, team = team_of(ctas, p.n), my_fork = thread / team, at0 = thread % team;
  const int size = 1 << p.page_shift;
  int taken = 0;
  for (int first = 0; first < p.n; first += kThreads) {
    const int mine = first + threadIdx.x;
    Fork f = {0, 0, -1, 0, -1};
    if (mine < p.n) {
      f.parent = p.a[mine];
      f.child = p.b[mine];
      if (f.parent < 0 || f.parent >= p.B || f.child < 0 || f.child >= p.B ||
          (bits[words + (f.child >> 5)] >> (f.child & 31) & 1) || (bits[f.parent >> 5] >> (f.parent & 31) & 1)) {
        errors |= kErrSequence;
      } else {
        f.rows = __ldcg(p.kv_len + f.parent);
        if (f.rows < 0 || f.rows > p.max_pages << p.page_shift) {
          errors |= kErrKvLen;
          f.rows = -1;
        }
      }
    }
    int need = 0, all, none;
    if (f.rows > 0 && (f.rows & (size - 1))) {
      // (no page is taken for rows that cannot be copied: the child must not hold a page of somebody else's)
      f.last = p.table[(int64_t)f.parent * p.max_pages + (f.rows >> p.page_shift)];
      need = f.last >= 0 && f.last < p.num_pages;
      if (!need) {
        f.last = -1;
        errors |= kErrPage;
      }
    }
    f.rank = taken + scan_threads(need, 0, area, &all, &none);
    taken += all;
    if (need && f.rank >= free0) {
      errors |= kErrFull;
      f.rows = -1;
    }
    forks[threadIdx.x] = f;
    __syncthreads();
    if (my_fork < min(kThreads, p.n - first)) {
      const Fork k = forks[my_fork];
      const int full = k.rows >> p.page_shift, rest = k.rows & (size - 1);
      const int32_t* const from = p.table + (int64_t)k.parent * p.max_pages;
      int32_t* const to = p.table + (int64_t)k.child * p.max_pages;
      if (k.rows > 0) {
        for (int j0 = at0; j0 < full; j0 += team * kAtOnce) {
          int id[kAtOnce];
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) id[k] = j0 + k * team < full ? from[j0 + k * team] : 0;
#pragma unroll
          for (int k = 0; k < kAtOnce; ++k) {
            const int j = j0 + k * team;
            if (j >= full) break;
            to[j] = id[k];
            if (id[k] >= 0 && id[k] < p.num_pages) atomicAdd(counts + id[k], 1); else errors |= kErrPage;
          }
        }
      }
      if (at0 == 0) {
        int src = -1, dst = -1, rows = 0;
        if (k.rows > 0 && rest) {
          if (k.last >= 0) {
            dst = list[free0 - 1 - k.rank];
            if (dst < 0 || dst >= p.num_pages) {
              errors |= kErrPool;
              dst = -1;
            } else {
              atomicAdd(counts + dst, 1);
              src = k.last;
              rows = rest;
            }
          }
          to[full] = dst;
        }
        const int at = first + my_fork;
        p.copies[at] = src;
        p.copies[p.n + at] = dst;
        p.copies[2 * (int64_t)p.n + at] = rows;
        if (k.rows >= 0) p.kv_len[k.child] = k.rows;
      }
    }
    __syncthreads();
  }
  if (ctas > 1) cluster_sync();  // every CTA has read the free pages
  if (cta == 0 && threadIdx.x == 0) p.pool[0] = free0 - min(taken, free0);
  report(p.err_flag, errors);
}

__global__ void __launch_bounds__(256) init_kernel(int32_t* pool, int num_pages) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < kPoolHeader) pool[i] = i == 0 ? num_pages : 0;
  if (i < num_pages) {
    pool[kPoolHeader + i] = 0;
    pool[kPoolHeader + num_pages + i] = i;
  }
}

// CTAs of a call: one where its table entries are few (no cluster barriers),
// else a cluster.
constexpr int64_t kOneCtaEntries = 4096;

template <typename K, typename... A>
cudaError_t launch_cluster(K* kernel, int ctas, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = ctas;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_pool_init(int32_t* pool, int num_pages, cudaStream_t stream) {
  const int n = std::max(num_pages, kPoolHeader);
  init_kernel<<<(n + 255) / 256, 256, 0, stream>>>(pool, num_pages);
  return cudaGetLastError();
}

cudaError_t launch_pool_resize(const PoolParams& p, cudaStream_t stream) {
  const int ctas = (int64_t)p.B * p.max_pages <= kOneCtaEntries && p.num_pages <= kOneCtaEntries ? 1 : kClusterMax;
  return launch_cluster(resize_kernel, ctas, 0, stream, p, ctas);
}

cudaError_t launch_pool_fork(const PoolParams& p, cudaStream_t stream) {
  const int ctas = (int64_t)p.n * p.max_pages <= kOneCtaEntries ? 1 : kClusterMax;
  const int words = (p.B + 31) / 32;  // (at most 16 KiB of bits)
  return launch_cluster(fork_kernel, ctas, (size_t)words * 8, stream, p, ctas, words);
}

}  // namespace da
