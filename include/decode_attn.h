/*
 * decode_attn.h — C ABI of the GB300 (sm_103a) decode-attention library.
 *
 * One autoregressive decode step of one attention layer over a STATIC,
 * preallocated KV cache: the new key/value row is written in place at
 * position_id, and a single query token per head attends to the active prefix
 * [0, kv_len) of the cache only, with kv_len = position_id + 1. Grouped-query
 * heads are served straight from their shared KV head (no expansion).
 *
 * The operation follows:
 *  - VoxCPM issue #395, "MiniCPM4 MiniCPMAttention.forward_step Attention
 *    Performance Fix", section 3 (attend to the slice [0, position_id] only;
 *    position 0 attends to one row and returns V[0]) and section 4.1 (the
 *    patched forward_step: in-place write key_cache[:, :, position_id, :],
 *    then SDPA on the slice with enable_gqa=True);
 *  - fish-speech issue #1310, "Optimize native AR decoding by attending only
 *    to the active KV-cache prefix", section 2 (the cache keeps its physical
 *    max_seq_len size; only k[:, :, :kv_len], v[:, :, :kv_len] are consumed);
 *  - Cuda-Compute-OSS issue #343, "one-token decode fast path", section
 *    "Proposed implementation" (softmax(q K^T / sqrt(d)) V, max-subtracted
 *    softmax accumulated in fp32, result cast back to the input dtype).
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers to contiguous row-major arrays
 *    owned by the caller, 16-byte aligned. The library never allocates,
 *    frees or synchronises; work is enqueued on `stream` (a cudaStream_t;
 *    NULL is the legacy default stream) and the call returns at once.
 *  - Layouts: q and out [B, n_head, head_dim]; k_cache and v_cache
 *    [B, n_kv_head, capacity, head_dim]; k_new and v_new
 *    [B, n_kv_head, head_dim]; kv_len and position_ids int32 [B].
 *    Query head h reads KV head h / (n_head / n_kv_head).
 *  - dtype is DA_F16 or DA_BF16 and applies to q, out and both caches.
 *    Arithmetic is fp32; out is rounded to nearest even.
 *  - Supported: head_dim in {64, 128}; n_head / n_kv_head in {1, 2, 4, 8}.
 *  - Errors the host can see (null pointers, bad sizes, misalignment, a
 *    small workspace, an unsupported shape) return a negative da_status
 *    before anything is enqueued. Facts only the device knows (a kv_len
 *    outside [1, capacity], a position outside [0, capacity)) never fault:
 *    the affected output rows become NaN, the affected cache write is
 *    skipped, and the DA_DEVERR_* bit is OR-ed into *err_flag (a device
 *    int32, may be NULL). A launch failure returns DA_ERR_CUDA.
 */
#ifndef DECODE_ATTN_H_
#define DECODE_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DA_API __attribute__((visibility("default")))
#else
#define DA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { DA_F16 = 0, DA_BF16 = 1 } da_dtype;

typedef enum {
  DA_OK = 0,
  DA_ERR_NULL = -1,        /* a required pointer is NULL */
  DA_ERR_SHAPE = -2,       /* a size is out of range or inconsistent */
  DA_ERR_UNSUPPORTED = -3, /* valid but not built: head_dim, group size or page size */
  DA_ERR_WORKSPACE = -4,   /* workspace NULL or smaller than required */
  DA_ERR_CUDA = -5,        /* a CUDA runtime call or launch failed */
  DA_ERR_ALIGN = -6,       /* a pointer is not 16-byte aligned (int32 and scale arrays: 4-byte) */
  DA_ERR_DTYPE = -7        /* unknown dtype code */
} da_status;

/* Bits OR-ed into *err_flag by the kernels. */
#define DA_DEVERR_KV_LEN 1u   /* some kv_len[b] outside [1, capacity]: rows of b are NaN */
#define DA_DEVERR_POSITION 2u /* some position_ids[b] outside [0, capacity): write skipped */
#define DA_DEVERR_TIMEOUT 4u  /* a pipeline wait hit its time limit: rows are NaN */
#define DA_DEVERR_WORKSPACE 8u /* the workspace counters were not zero: rows of the group are NaN */
#define DA_DEVERR_PAGE 16u /* a page id in use lies outside [0, num_pages): rows are NaN, writes skipped */
#define DA_DEVERR_TOKENS 32u /* a sequence's range of packed tokens is not valid, or too long: skipped, or rows are NaN */
#define DA_DEVERR_SEQUENCE 64u /* a fork's parent or child is no sequence, or one that another fork writes: skipped */
#define DA_DEVERR_FULL 128u /* the pool has too few free pages: entries are -1, forks skipped */
#define DA_DEVERR_POOL 256u /* a pool's counts or list of free pages are not consistent */

/* Human-readable name of a da_status value (static string). */
DA_API const char* da_status_string(int status);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
DA_API int da_version(void);

/*
 * Split plan of the decode kernel, a pure host computation (no CUDA call):
 * the number of KV splits S per (sequence, KV head) group for B sequences,
 * n_kv_head KV heads, head_dim and a bound max_kv_len on the active length,
 * on a GPU with num_sms multiprocessors holding ctas_per_sm decode CTAs each,
 * where one thread-block cluster of up to cluster_max CTAs per group can be
 * resident. Flat plan: S is as many splits as fit one wave of resident CTAs
 * (two waves when B > 1, since most sequences of a batch are shorter than the
 * bound), at most one per tile of max_kv_len rows and at most 128; the
 * partials go through the workspace (*cluster_size = 1). Cluster plans, where
 * the S splits of a group form one cluster of *cluster_size = S CTAs that
 * merge their partial softmax states through distributed shared memory:
 * (a) one sequence whose clusters of c = min(cluster_max, 16) CTAs cover every
 * SM (B * n_kv_head * c >= num_sms) over at least 2c tiles: S = c;
 * (b) a short prefix: S = min(c, num_sms / (B * n_kv_head), tiles /
 * ctas_per_sm rounded up) when each split then streams at most 4 tiles, and
 * no split at all (S = 1) when that S is below 2.
 * (*cluster_size is written when non-NULL.) Each sequence b then splits its
 * own kv_len[b] rows evenly over at most S CTAs, in whole tiles.
 * Returns S >= 1, or a negative da_status.
 */
DA_API int decode_attn_plan_splits(int B, int n_kv_head, int head_dim, int max_kv_len, int num_sms,
                                   int ctas_per_sm, int cluster_max, int* cluster_size);

/*
 * Bytes of scratch memory decode_attn_fwd / decode_step_fwd need for these
 * sizes on the current device, for any max_kv_len_hint <= capacity.
 * Returns 0 when no scratch is needed (one cluster serves each group), or
 * (size_t)-1 for invalid sizes or a failed device query. Otherwise the
 * workspace starts with a 4 KiB region of 32-bit arrival counters (one per
 * sequence and KV head), followed by fp32 per-cluster partials
 * [B, n_head, S / cluster, head_dim + 2]. It must be zero-filled once before
 * its first use (decode_attn_workspace_init, or any memset); every call that
 * completes leaves it ready for the next call of any shape. Calls that
 * overlap on one workspace can leave a counter non-zero: a later call then
 * merges that group early or writes NaN rows with DA_DEVERR_WORKSPACE. After
 * a DA_DEVERR_TIMEOUT or DA_DEVERR_WORKSPACE, or an overlap, zero it again.
 */
DA_API size_t decode_attn_workspace_size(int B, int n_head, int n_kv_head, int head_dim, int capacity);

/* Zero-fill a workspace on `stream` (cudaMemsetAsync; allocates nothing). */
DA_API int decode_attn_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * The split count S that decode_attn_fwd / decode_step_fwd will use for
 * these arguments on the current device, and (when cluster_size is non-NULL)
 * the cluster size. S == 1: one CTA per group writes out directly; S equal
 * to the cluster size: one cluster per group merges in distributed shared
 * memory, no workspace; S larger: one partial per cluster goes through the
 * workspace and the last CTA of each group merges them, in the same launch.
 * The plan is decode_attn_plan_splits with this device's occupancy (the
 * largest cluster size of which one cluster per group is co-resident).
 * Returns S >= 1 or a negative da_status.
 */
DA_API int decode_attn_splits_for(int B, int n_head, int n_kv_head, int head_dim, int capacity,
                                  int max_kv_len_hint, int dtype, int* cluster_size);

/* Kernels decode_attn_kernel_for reports. */
#define DA_KERNEL_CUDA_CORES 0        /* scores on the CUDA cores (every group size) */
#define DA_KERNEL_TENSOR_CORES 1      /* >= 4 query heads per KV head: scores on the tensor cores, one CTA per SM */
#define DA_KERNEL_TENSOR_CORES_PAIRED 2 /* the same with two CTAs per SM (one CTA per group filling the GPU) */

/*
 * The decode kernel that decode_attn_fwd / decode_step_fwd / the layers call
 * (rotary == 0) or decode_step_rope_fwd (rotary != 0) will launch for these
 * arguments on the current device (for the layers call pass layers * B as
 * B). With four or more query heads per KV head the scores of a K tile,
 * q K^T, are a small dense product: the library runs it on the tensor cores
 * when each CTA streams more than 4 tiles or when the groups fill the GPU one
 * CTA each, and on the CUDA cores otherwise (shorter per-tile path). Every
 * kernel computes the same softmax(q K^T * scale) V within the stated
 * tolerance (the operation of decode_attn_fwd: Cuda-Compute-OSS issue #343,
 * "Proposed implementation"); results of different kernels may differ in
 * the last bits. Sizes are validated as in decode_attn_fwd (DA_ERR_SHAPE,
 * DA_ERR_UNSUPPORTED, DA_ERR_DTYPE before any device query). Returns a
 * DA_KERNEL_* value or a negative da_status.
 */
DA_API int decode_attn_kernel_for(int B, int n_head, int n_kv_head, int head_dim, int capacity,
                                  int max_kv_len_hint, int dtype, int rotary);

/*
 * Profiling hook. When both are non-NULL, every later decode_attn_fwd /
 * decode_step_fwd call made by this host thread records event_before (a
 * cudaEvent_t) on its stream immediately before its split-KV decode kernel
 * and event_after immediately after it, so that cudaEventElapsedTime gives
 * that kernel's device time. Under stream capture the records become graph
 * nodes. NULL, NULL turns the hook off. Returns DA_OK.
 */
DA_API int da_set_timing_events(void* event_before, void* event_after);

/*
 * Ordering promise for the decode calls of this host thread (default off).
 * Every decode kernel waits, by programmatic dependent launch, for the
 * kernel before it on the stream to complete before it reads its inputs.
 * With on != 0 the caller promises, for every later call of this thread with
 * B == 1 and max_kv_len_hint > 0, that no kernel that may still be running
 * when the call's kernel starts writes the cache rows the call will read:
 * rows [0, max_kv_len_hint) of k_cache and v_cache for decode_attn_fwd, rows
 * [0, max_kv_len_hint - 1) for the fused steps (whose last row comes from
 * k_new and v_new). The kernel then copies those rows of its first tiles into
 * shared memory before that wait; q, the lengths, k_new, v_new and the rotary
 * tables are still read after it. A decode loop meets the promise when the
 * only kernels between two calls on the same caches complete before the next
 * one starts: for instance the previous layer's call and the projections
 * (kernels on this stream release their dependents only after their own wait,
 * as this library's do). Back-to-back calls on the SAME caches (one layer,
 * nothing in between) do not: the first writes row position into the rows the
 * second reads. Breaking the promise gives wrong results, never a fault.
 * Returns DA_OK.
 */
DA_API int da_set_prefix_ready(int on);

/*
 * Failure-detection test hook. With slot >= 0, every later decode call made
 * by this host thread leaves ring slot `slot` of the first split of sequence
 * 0, KV head 0 unfilled: that CTA's pipeline waits run into their time limit
 * (about one second), the CTA publishes NaN and the call sets
 * DA_DEVERR_TIMEOUT; nothing faults and the context stays usable. Zero the
 * workspace afterwards (as after any DA_DEVERR_TIMEOUT). slot < 0 turns the
 * hook off (the default). A tree attention call leaves out that copy of its
 * first CTA in the same way. Returns DA_OK.
 */
DA_API int da_test_skip_slot(int slot);

/*
 * In-place append: k_cache[b, g, position_ids[b], :] = k_new[b, g, :] and the
 * same for V, for every sequence b and KV head g, copied bit for bit.
 * (VoxCPM issue #395, section 4.1.) A position outside [0, capacity) skips
 * that sequence and sets DA_DEVERR_POSITION.
 */
DA_API int kvcache_append(void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                   const int32_t* position_ids, int B, int n_kv_head, int head_dim, int capacity,
                   int dtype, int32_t* err_flag, void* stream);

/*
 * Decode attention over the active prefix:
 *   out[b, h, :] = softmax_j(scale * <q[b, h, :], K[b, g, j, :]>) V[b, g, j, :]
 * for j in [0, kv_len[b]) and g = h / (n_head / n_kv_head). Cache rows at or
 * beyond kv_len[b] are never read. kv_len is a DEVICE array, so no host
 * synchronisation is needed; max_kv_len_hint (> 0) is an optional host bound
 * on max_b kv_len[b] that only sizes the launch (<= 0 means capacity). A
 * kv_len above the hint but within capacity is still computed correctly.
 * workspace/workspace_bytes: caller-owned device scratch of at least
 * decode_attn_workspace_size(...) bytes (may be NULL when that is 0); calls
 * that share one workspace must not overlap on the GPU.
 * (Cuda-Compute-OSS issue #343, "Proposed implementation"; VoxCPM issue
 * #395, section 4.1.)
 */
DA_API int decode_attn_fwd(const void* q, const void* k_cache, const void* v_cache, const int32_t* kv_len,
                    int B, int n_head, int n_kv_head, int head_dim, int capacity, float scale,
                    void* out, void* workspace, size_t workspace_bytes, int max_kv_len_hint,
                    int dtype, int32_t* err_flag, void* stream);

/*
 * One fused decode step: the append of kvcache_append followed by
 * decode_attn_fwd with kv_len[b] = position_ids[b] + 1, in a single pass
 * over the cache. The attended row position_ids[b] is taken from k_new/v_new
 * and also written into the cache. Same arguments, layouts and error
 * behaviour as the two calls it replaces (VoxCPM issue #395, section 4.1:
 * write at position_id, then attend over [0, position_id]).
 */
DA_API int decode_step_fwd(const void* q, void* k_cache, void* v_cache, const void* k_new,
                    const void* v_new, const int32_t* position_ids, int B, int n_head,
                    int n_kv_head, int head_dim, int capacity, float scale, void* out,
                    void* workspace, size_t workspace_bytes, int max_kv_len_hint, int dtype,
                    int32_t* err_flag, void* stream);

/*
 * decode_step_fwd with the rotary position embedding the patched
 * forward_step applies to the query and the new key before the append
 * (VoxCPM issue #395, section 4.1: apply_rotary_pos_emb(query_states,
 * key_states, cos, sin), then the write at position_id and the attention).
 * q and k_new are the vectors before rotation; for sequence b with
 * p = position_ids[b], every query head and the new key row become
 *   x * cos[p] + rotate_half(x) * sin[p],  rotate_half(x) = [-x[D/2:], x[:D/2]]
 * with each product and the sum rounded to fp32 (no fused multiply-add) and
 * the result rounded to nearest even in the storage type; the rotated key row
 * is what the cache receives. v_new is appended unchanged.
 *   rope_cos, rope_sin  device fp32 tables [rope_rows, head_dim], row p
 *                       holding the embedding of position p; 16-byte
 *                       aligned; rope_rows >= capacity (else DA_ERR_SHAPE)
 * Everything else as decode_step_fwd. NULL tables give DA_ERR_NULL.
 */
DA_API int decode_step_rope_fwd(const void* q, void* k_cache, void* v_cache, const void* k_new,
                    const void* v_new, const float* rope_cos, const float* rope_sin, int rope_rows,
                    const int32_t* position_ids, int B, int n_head, int n_kv_head, int head_dim,
                    int capacity, float scale, void* out, void* workspace, size_t workspace_bytes,
                    int max_kv_len_hint, int dtype, int32_t* err_flag, void* stream);

/*
 * decode_step_fwd for `layers` layers of one model in one call: layer l
 * reads q[l], k_new[l], v_new[l] and appends to and attends over its own
 * caches k_cache[l], v_cache[l], writing out[l]:
 *   q, out          [layers, B, n_head, head_dim]
 *   k_cache, v_cache [layers, B, n_kv_head, capacity, head_dim]
 *   k_new, v_new    [layers, B, n_kv_head, head_dim]
 * all contiguous; position_ids [B] (the same step for every layer).
 * Every layer's inputs are given at once, so no layer depends on another:
 * the stacks are one batch of layers * B sequences (sequence l * B + b has
 * position position_ids[b]) and the whole call is ONE launch of the decode
 * kernel, with no per-layer launch cost. For a caller that holds every
 * layer's inputs at once (replays, benchmarks, several independent models or
 * requests stacked on a leading axis); in a model whose layer l + 1 query
 * depends on layer l's output, call decode_step_fwd per layer instead.
 * Results equal decode_step_fwd on the flattened [layers * B, ...] batch with
 * position_ids repeated per layer, bit for bit.
 *   workspace   at least decode_attn_workspace_size(layers * B, n_head,
 *               n_kv_head, head_dim, capacity) bytes
 * Validation as decode_step_fwd, all of it before the launch: an invalid
 * argument enqueues nothing, and a launch failure (DA_ERR_CUDA) leaves every
 * layer untouched. layers < 0 or layers * B > 65535 gives DA_ERR_SHAPE,
 * layers == 0 does nothing.
 */
DA_API int decode_step_layers_fwd(const void* q, void* k_cache, void* v_cache, const void* k_new,
                    const void* v_new, const int32_t* position_ids, int layers, int B, int n_head,
                    int n_kv_head, int head_dim, int capacity, float scale, void* out, void* workspace,
                    size_t workspace_bytes, int max_kv_len_hint, int dtype, int32_t* err_flag, void* stream);

/*
 * KV-head partition of one attention layer over `world` ranks (one GPU
 * each), a pure host computation. Every (sequence, KV head) group is
 * independent (its G = n_head / n_kv_head query heads read only that KV
 * head), so rank r can own a contiguous block of KV heads with their query
 * heads and run the decode calls of this header on its block alone, with no
 * exchange of data: its caches are [B, n_kv_local, capacity, head_dim] for KV
 * heads [kv_head0, kv_head0 + n_kv_local), its q and out [B, n_head_local,
 * head_dim] for query heads [head0, head0 + n_head_local) (n_head_local =
 * G * n_kv_local), and the ranks' outputs laid side by side on the head axis,
 * in rank order, are the layer's output. KV heads are dealt as evenly as
 * possible: the first n_kv_head % world ranks hold one more; a rank holds
 * none when world > n_kv_head. (fish-speech issue #1310, section 2: the GQA
 * head map h -> h / G; the pages run on one GPU, so this partition is this
 * library's own.) Returns DA_OK, DA_ERR_SHAPE for inconsistent sizes or a
 * rank outside [0, world), DA_ERR_NULL for a NULL output pointer.
 */
DA_API int decode_attn_shard_heads(int n_head, int n_kv_head, int world, int rank, int* kv_head0,
                                   int* n_kv_local, int* head0, int* n_head_local);

/* Size of the library-owned scratch array used by
 * decode_attn_fwd_static_scratch (1 MiB per GPU that loads the library). */
#define DA_STATIC_SCRATCH_BYTES (1u << 20)

/*
 * decode_attn_fwd for callers that must not allocate GPU memory. This entry
 * point is an addition of this library; the pages have no counterpart.
 *
 * Some callers only receive input and output buffers from the framework that
 * hosts them (a plugin inside an inference server or a real-time audio
 * engine, for instance) and are not allowed to call cudaMalloc, or cannot
 * reach the memory pool that owns the device memory. This variant takes the
 * same arguments as decode_attn_fwd minus the workspace: its split partials
 * live in a file-scope device array of DA_STATIC_SCRATCH_BYTES that the
 * library holds on every GPU that loads it, until the process exits. Nothing
 * is allocated or freed by the call.
 *
 * - The first call on a device that needs scratch looks up that array's
 *   device address (cudaGetSymbolAddress, with that device current) and keeps
 *   it for the life of the process; make that first call before any stream
 *   capture on the device (a first call made while `stream` is capturing
 *   returns DA_ERR_CUDA). A device reset (cudaDeviceReset) is not supported
 *   afterwards.
 * - Arguments whose split plan needs more scratch than
 *   DA_STATIC_SCRATCH_BYTES (decode_attn_workspace_size-style need for this
 *   call's max_kv_len_hint) are rejected with DA_ERR_SHAPE before anything is
 *   enqueued; use decode_attn_fwd with your own workspace for those.
 * - Every call on a device shares the one array and leaves its partials in
 *   it. A call that needs scratch first zero-fills its own arrival counters
 *   on `stream` (a cudaMemsetAsync of 4 * B * n_kv_head bytes), and its
 *   kernels write every partial they later read, so each call is correct
 *   whatever an earlier call left in the array. Calls that overlap on the GPU
 *   (different streams without ordering, or different host threads) race on
 *   the array: their outputs may be wrong, NaN (with DA_DEVERR_WORKSPACE) or
 *   left unwritten. Keep such calls ordered; the first ordered call after an
 *   overlap is correct again, with nothing to reset.
 * Otherwise identical to decode_attn_fwd, including results bit for bit.
 */
DA_API int decode_attn_fwd_static_scratch(const void* q, const void* k_cache, const void* v_cache,
                                          const int32_t* kv_len, int B, int n_head, int n_kv_head,
                                          int head_dim, int capacity, float scale, void* out,
                                          int max_kv_len_hint, int dtype, int32_t* err_flag,
                                          void* stream);

/* ------------------------------------------------------------------------
 * Paged caches, 8-bit caches and sliding windows. These entry points are
 * additions of this library; the pages it follows have no counterpart. They
 * keep its conventions (device pointers, contiguous row-major, nothing
 * allocated or synchronised, device facts reported in *err_flag) with these
 * layouts:
 *   k_pages, v_pages  [num_pages, n_kv_head, page_size, head_dim], page_size
 *                     a power of two in [16, 256]; a pool that sequences of
 *                     any length share
 *   page_table        int32 [B, max_pages]: rows [i * page_size, (i + 1) *
 *                     page_size) of sequence b are page page_table[b, i].
 *                     Entries of pages that a call does not touch are not
 *                     looked at and may hold anything. Sequences may share
 *                     pages that are only read; a page that two sequences of
 *                     one call append to ends up with unspecified rows.
 * and, for pages in 8 bits (e4m3: sign, four exponent, three mantissa bits, no
 * infinities),
 *   k_scale, v_scale  fp32 [num_pages, n_kv_head]: element x of a page and KV
 *                     head stands for x * scale.
 * max_pages * page_size stays below 2^31 - 512. The attentions (paged or over a
 * static cache) take at most 65535 sequences and 65535 KV heads, and B *
 * n_kv_head times the 16-row tiles of a longest sequence below 2^37. (Else
 * DA_ERR_SHAPE.) Arrays that a call writes overlap no other argument, but for
 * q_out, which may be q itself.
 */

/*
 * Append new rows to a paged cache, with the rotary embedding on the way. The
 * rows are packed: k_new and v_new [tokens, n_kv_head, head_dim]. Sequence b
 * owns tokens [token_start[b], token_start[b + 1]) (int32 [B + 1], rising),
 * and its first one has position position_ids[b]; token_start NULL means one
 * token per sequence (tokens == B, else DA_ERR_SHAPE). Tokens before
 * token_start[0] and from token_start[B] on (padding) are left alone, and so
 * are their q_out rows. With tables (rope_cos, rope_sin fp32 [rope_rows,
 * head_dim], as in decode_step_rope_fwd) the key row at position p becomes
 * k * cos[p] + rotate_half(k) * sin[p], products and sum rounded to fp32 and
 * the result once to the storage type; without (both NULL) it is copied. V is
 * copied. q [tokens, n_head, head_dim] (NULL: none) is rotated the same way
 * into q_out, which may be q itself; it needs the tables.
 * A sequence whose positions do not all lie in [0, max_pages * page_size) and
 * [0, rope_rows) is skipped whole and sets DA_DEVERR_POSITION (its q_out rows
 * become NaN); rows of a page id outside the pool are skipped and set
 * DA_DEVERR_PAGE. Only the appended rows of a page are written. k_pages and
 * v_pages are two arrays (else DA_ERR_SHAPE).
 */
DA_API int kvcache_append_paged(void* k_pages, void* v_pages, const void* k_new, const void* v_new, const void* q,
                    void* q_out, const float* rope_cos, const float* rope_sin, int rope_rows,
                    const int32_t* page_table, const int32_t* position_ids, const int32_t* token_start, int B,
                    int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages,
                    int dtype, int32_t* err_flag, void* stream);

/*
 * kvcache_append_paged into pages of e4m3 (dtype is that of k_new, v_new, q
 * and q_out). For every page and KV head that gets rows, with K and V apart:
 *   peak  = largest finite |x| among the page's new rows (fp32, the rotated
 *           key before any rounding)
 *   scale = the smallest power of two >= peak / 448, at least 2^-100; and at
 *           least the page's present scale when rows before the first new one
 *           lie in the page (a page filled from its first row on starts anew).
 *           A present scale is finite and not negative, a power of two or not
 *   x is stored as e4m3(x / scale), nearest even; NaN and infinities as NaN.
 * Where the scale grows, the page's earlier rows are rounded to the new one
 * (a power of two: only exponents move, bits are lost below 2^-9 of the new
 * scale alone). Rows behind the new ones are left as they were. Appending the
 * same rows at the same positions again changes nothing.
 */
DA_API int kvcache_append_paged_q8(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const void* k_new,
                    const void* v_new, const void* q, void* q_out, const float* rope_cos, const float* rope_sin,
                    int rope_rows, const int32_t* page_table, const int32_t* position_ids,
                    const int32_t* token_start, int B, int tokens, int n_head, int n_kv_head, int head_dim,
                    int num_pages, int page_size, int max_pages, int dtype, int32_t* err_flag, void* stream);

/*
 * Bytes of scratch that one call of decode_attn_paged_fwd,
 * decode_attn_paged_q8_fwd or decode_attn_window_fwd needs on the current
 * device: it depends on the heads alone, not on the batch, the lengths or the
 * pages. Zero-fill it once before its first use (decode_attn_workspace_init);
 * every call that completes leaves it ready for the next, whatever its sizes.
 * Calls that share a workspace must not overlap on the GPU. Returns
 * (size_t)-1 for invalid sizes or a failed device query.
 */
DA_API size_t decode_attn_paged_workspace_size(int n_head, int n_kv_head, int head_dim);

/*
 * Decode attention over a paged cache. Row j of sequence b is visible when
 *   j < kv_len[b] and (window == 0 or j >= kv_len[b] - window or j < sinks)
 * (the last `window` rows, the query's own among them, and the first `sinks`
 * ones), and out[b, h, :] = softmax_j(scale <q[b, h], K_j>) V_j over those
 * rows, fp32 arithmetic, rounded once. (Over fp16 and 8-bit caches a softmax
 * weight keeps 22 bits, and what lies above 2^-38 of the largest one of its
 * head; over bf16 caches all 24. Over 8-bit pages a bf16 query keeps what lies
 * above 2^-25 of its head's largest element.) Rows that are not visible are not
 * read; NaN among the visible ones reaches the heads that read it, and an
 * infinite element of V makes that element of its heads' outputs infinite or
 * NaN (a weight reaches V in pieces, and a piece may be zero or negative).
 * The weighted sums are held unnormalised: over bf16 and 8-bit caches kv_len
 * times the largest |V| stays below 2^120, or they may overflow.
 * kv_len[b] == 0 (an idle slot of a batch) gives a row of zeros;
 * kv_len[b] < 0 or > max_pages * page_size gives NaN and DA_DEVERR_KV_LEN; a
 * page id outside the pool gives NaN for the heads that would read it and
 * DA_DEVERR_PAGE. window >= 0, sinks >= 0, and sinks > 0 needs window > 0
 * (else DA_ERR_SHAPE). No length bound is needed: the launch does not depend
 * on the lengths, so a captured graph serves any of them. Equal calls give
 * equal bits. kv_len and page_table must not change while the call runs, and
 * out must not be q (DA_ERR_SHAPE).
 */
DA_API int decode_attn_paged_fwd(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                    const int32_t* kv_len, int B, int n_head, int n_kv_head, int head_dim, int num_pages,
                    int page_size, int max_pages, int window, int sinks, float scale, void* out, void* workspace,
                    size_t workspace_bytes, int dtype, int32_t* err_flag, void* stream);

/*
 * decode_attn_paged_fwd over pages of e4m3 with their scales: K_j and V_j are
 * the stored values times the scale of their page and KV head (any finite
 * scale; those of kvcache_append_paged_q8 are powers of two). dtype is that of
 * q and out.
 */
DA_API int decode_attn_paged_q8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                    const float* v_scale, const int32_t* page_table, const int32_t* kv_len, int B, int n_head,
                    int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int window, int sinks,
                    float scale, void* out, void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag,
                    void* stream);

/*
 * Decode attention with a sliding window and sinks over the static caches of
 * decode_attn_fwd: the visible rows are those of decode_attn_paged_fwd, with
 * window >= 1 (else DA_ERR_SHAPE), so a step reads at most window + sinks rows
 * however long the prefix is. kv_len[b] == 0 gives zeros; kv_len[b] < 0 or >
 * capacity gives NaN and DA_DEVERR_KV_LEN.
 */
DA_API int decode_attn_window_fwd(const void* q, const void* k_cache, const void* v_cache, const int32_t* kv_len,
                    int B, int n_head, int n_kv_head, int head_dim, int capacity, int window, int sinks, float scale,
                    void* out, void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag, void* stream);

/* ------------------------------------------------------------------------
 * Serving steps with drafted tokens, over the paged caches above (the same
 * conventions and layouts). A step takes pages for the drafts
 * (kvcache_resize_paged), appends them with rotary positions by their depth
 * (kvcache_append_paged_axes), verifies them in one pass over the cache
 * (decode_attn_tree_fwd), moves the accepted rows together
 * (kvcache_compact_paged) and gives the pages behind them back. No call needs
 * a length on the host, so that one captured graph serves every step.
 */

/*
 * kvcache_append_paged with rotary positions of their own: element pair (i, i +
 * head_dim / 2) of token t's key (and q) heads is rotated by row
 * rope_position_ids[a, t] of the tables, a = rope_axis[i], whatever row of the
 * cache the token goes to.
 *   rope_position_ids  int32 [axes, tokens], 1 <= axes <= DA_MAX_ROPE_AXES:
 *                      time, height and width of an image's patches, or one
 *                      axis with the depth of a drafted token
 *   rope_axis          int32 [head_dim / 2], 16-byte aligned, any order
 *                      (sections, interleaved); NULL: axis 0 for all
 * The tables are required. A token with a position (on any axis) outside [0,
 * rope_rows) is skipped whole (its q_out row becomes NaN) and sets
 * DA_DEVERR_POSITION; an entry of rope_axis outside [0, axes) sets it too and
 * counts as axis 0. position_ids alone decide where rows go; rope_rows does not
 * bound them. Everything else as in kvcache_append_paged (whose results it
 * has when every rope position is the token's position).
 */
#define DA_MAX_ROPE_AXES 4
DA_API int kvcache_append_paged_axes(void* k_pages, void* v_pages, const void* k_new, const void* v_new, const void* q,
                    void* q_out, const float* rope_cos, const float* rope_sin, int rope_rows,
                    const int32_t* rope_position_ids, const int32_t* rope_axis, int axes, const int32_t* page_table,
                    const int32_t* position_ids, const int32_t* token_start, int B, int tokens, int n_head,
                    int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int dtype,
                    int32_t* err_flag, void* stream);

/* kvcache_append_paged_axes into pages of e4m3, as kvcache_append_paged_q8. */
DA_API int kvcache_append_paged_q8_axes(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                    const void* k_new, const void* v_new, const void* q, void* q_out, const float* rope_cos,
                    const float* rope_sin, int rope_rows, const int32_t* rope_position_ids, const int32_t* rope_axis,
                    int axes, const int32_t* page_table, const int32_t* position_ids, const int32_t* token_start,
                    int B, int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size,
                    int max_pages, int dtype, int32_t* err_flag, void* stream);

/* Most tokens of one sequence in a call of decode_attn_tree_fwd. (More new tokens behind a prefix take a call
 * for each 256 of them, in order, each of which reads the prefix again.) */
#define DA_TREE_MAX_TOKENS 256

/* Bytes of scratch of one call of decode_attn_tree_fwd or
 * decode_attn_tree_q8_fwd on the current device; it depends on the heads alone.
 * Zero-fill it once before its first use; every call that completes leaves it
 * ready for the next, of any operator of this library whose workspace it is large
 * enough for (its counters lie in the first 4 KiB, as decode_attn_fwd's, and are zero
 * between calls), and the other way round. Calls that share it must not overlap on the GPU.
 * Returns (size_t)-1 for invalid sizes or a failed device query. */
DA_API size_t decode_attn_tree_workspace_size(int n_head, int n_kv_head, int head_dim);

/*
 * Attention of several new tokens of each sequence over a paged cache that
 * holds their rows already. q and out are packed, [tokens, n_head, head_dim];
 * sequence b owns tokens [token_start[b], token_start[b + 1]) (int32 [B + 1],
 * rising; NULL: one token per sequence), n_b of them, and they are its last
 * n_b rows: token i of it is row base_b + i, base_b = kv_len[b] - n_b. It sees
 * every row j < base_b, and of the new rows those of its mask: row base_b + i'
 * for i' in [0, n_b) where
 *   tree_mask == NULL   i' <= i (a chain of drafts)
 *   else                bit i' mod 64 of tree_mask[t, i' / 64] is set (int64
 *                       [tokens, mask_words], 1 <= mask_words <= 4; bits at
 *                       or past n_b do not matter): a tree's ancestors and
 *                       the token itself, or any other set
 *   out[t, h, :] = softmax_j(scale <q[t, h], K_j>) V_j over the rows seen
 * Products of the storage type, sums, maxima and exponentials in fp32; a
 * weight is rounded to the storage type, relative to its row's running
 * maximum (that of the first 128 rows, raised by whole powers of two: the weight of a
 * token's only row, or of a sink among them, is 1 and not rounded), before it reaches V (bf16, head_dim 128, sequences of at most 128 query
 * heads times tokens for each KV head: to 16 bits), and the output is rounded once. A token that sees
 * nothing gets a row of zeros. Rows that a token does not see do not reach
 * it, whatever they hold (NaN and infinities among them). Rows of q and out
 * that no sequence owns are left alone. Facts only the device knows:
 * kv_len[b] < n_b or > max_pages * page_size gives NaN rows and
 * DA_DEVERR_KV_LEN; n_b above DA_TREE_MAX_TOKENS or 64 * mask_words gives NaN
 * rows and DA_DEVERR_TOKENS; a token range that is not inside the packed
 * tokens is skipped and sets DA_DEVERR_TOKENS; a page id outside the pool
 * among the first ceil(kv_len / page_size) of a sequence gives NaN for its
 * tokens and DA_DEVERR_PAGE; a wait that hits its time limit gives NaN for some
 * units of tokens and DA_DEVERR_TIMEOUT; a workspace whose counters were not zero gives NaN
 * for the tokens that several CTAs share and DA_DEVERR_WORKSPACE, or joins their parts
 * early (as in decode_attn_workspace_size; zero the workspace after either). An infinite
 * element of V in a row that a token sees makes that element of its output infinite
 * or NaN. Scores, |scale <q, K_j>| of the rows seen, stay below 2^22 (32 bits leave half a power
 * of two open there, and a weight's type holds 2^16), and kv_len times the largest |V|
 * below 2^110, or a token's output may become NaN. Equal calls give equal bits. Lengths, table, tokens and masks must
 * not change while the call runs, and out must not overlap q (DA_ERR_SHAPE).
 * The pool has at most 2^31 - 1 rows of all KV heads, and B * n_kv_head * (n_head /
 * n_kv_head) times the 128-row tiles of a longest sequence, and 8 more, stay below
 * 2^31 (DA_ERR_SHAPE).
 */
DA_API int decode_attn_tree_fwd(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                    const int32_t* kv_len, const int32_t* token_start, const int64_t* tree_mask, int mask_words,
                    int B, int tokens, int n_head, int n_kv_head, int head_dim, int num_pages, int page_size,
                    int max_pages, float scale, void* out, void* workspace, size_t workspace_bytes, int dtype,
                    int32_t* err_flag, void* stream);

/* decode_attn_tree_fwd over pages of e4m3 with their scales (finite), as
 * decode_attn_paged_q8_fwd. dtype is that of q and out. The products are of fp16:
 * of a bf16 query, with 2^e the power of two at or below its head's largest element,
 * elements of 2^(e - 31) and more are exact, smaller ones are rounded to a multiple of
 * 2^(e - 38) (off by 2^(e - 39) at most); a weight, with the scale of its V row, keeps 11
 * bits above 2^-21 of its row's largest. Scales of V that a token sees are zero or lie
 * within 2^100 of one another. */
DA_API int decode_attn_tree_q8_fwd(const void* q, const void* k_pages, const void* v_pages, const float* k_scale,
                    const float* v_scale, const int32_t* page_table, const int32_t* kv_len,
                    const int32_t* token_start, const int64_t* tree_mask, int mask_words, int B, int tokens,
                    int n_head, int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, float scale,
                    void* out, void* workspace, size_t workspace_bytes, int dtype, int32_t* err_flag, void* stream);

/*
 * A pool's state, `pool`: int32 [DA_POOL_HEADER + 2 * num_pages]
 *   pool[0]                      number of free pages, f
 *   pool[1 .. DA_POOL_HEADER)    zero
 *   then [num_pages]             how many table entries hold each page
 *   then [num_pages]             the free pages, in entries [0, f)
 * The program may read it, or make it by itself (for a cache that exists). One
 * state serves the pools of all layers, which share page numbers. Calls on
 * one state must not overlap on the GPU. num_pages <= DA_POOL_MAX_PAGES.
 */
#define DA_POOL_HEADER 4
#define DA_POOL_MAX_PAGES (1 << 22)

/* A state whose pages are all free, listed in rising order (the last page is
 * taken first). */
DA_API int kvcache_pool_init(int32_t* pool, int num_pages, void* stream);

/*
 * Sequence b, whose first held_len[b] rows have pages, becomes one of
 * wanted_len[b] rows: table entries [ceil(wanted / page_size), ceil(held /
 * page_size)) are released (and become -1) where it shrinks, entries
 * [ceil(held / page_size), ceil(wanted / page_size)) get free pages where it
 * grows. Freeing a sequence is wanted 0, taking pages for new ones held 0.
 * First all releases: each lowers its page's count, and the pages whose count
 * becomes zero are put at the end of the list, in rising order. Then all
 * pages are taken from the end of the list, in the order of sequences and
 * rows (the first one gets the last entry), their counts raised by one. So
 * equal calls give equal states. Where the list runs out the entry becomes -1
 * and DA_DEVERR_FULL is set. A length outside [0, max_pages * page_size]
 * leaves the sequence as it was and sets DA_DEVERR_KV_LEN; a released entry
 * outside the pool sets DA_DEVERR_PAGE (-1: nothing); a page released more
 * often than it is counted, or a list with entries outside the pool, sets
 * DA_DEVERR_POOL. held_len and wanted_len int32 [B], may not overlap what the
 * call writes.
 */
DA_API int kvcache_resize_paged(int32_t* page_table, const int32_t* held_len, const int32_t* wanted_len,
                    int32_t* pool, int B, int num_pages, int page_size, int max_pages, int32_t* err_flag,
                    void* stream);

/*
 * Fork i (i < forks): sequence child[i] becomes a copy of sequence parent[i], n
 * = kv_len[parent[i]] rows. Their first floor(n / page_size) pages are shared
 * (the child's table entries are the parent's, their counts raised by one); a
 * page that is partly filled is not: the child gets one from the end of the
 * list of free pages (in the order of i), and copies[0, i] (the parent's page),
 * copies[1, i] (the child's) and copies[2, i] = n mod page_size say what
 * kvcache_copy_pages has to copy in every layer's pools (-1, -1, 0 where there
 * is nothing). kv_len[child[i]] becomes n; further entries of the child's table
 * row are left as they were. A child holds no pages before (release them with
 * kvcache_resize_paged). A fork is skipped, with copies -1, -1, 0, when parent or
 * child lie outside [0, B), when its child is another fork's child too, or its parent is
 * the child of any fork of the call (DA_DEVERR_SEQUENCE; a fork whose child another one names
 * as its parent is carried out, that other one is skipped), when the parent's length is outside [0,
 * max_pages * page_size] (DA_DEVERR_KV_LEN), or when it needs a page and none is
 * left (DA_DEVERR_FULL). A table entry outside the pool is shared without a count, or,
 * for a partly filled page, not copied: no page is taken, the child's entry becomes -1
 * and copies are -1, -1, 0. It sets DA_DEVERR_PAGE.
 *   parent, child int32 [forks]; copies int32 [3, forks]
 */
DA_API int kvcache_fork_paged(int32_t* page_table, int32_t* kv_len, const int32_t* parent, const int32_t* child,
                    int32_t* pool, int32_t* copies, int forks, int B, int num_pages, int page_size, int max_pages,
                    int32_t* err_flag, void* stream);

/*
 * Copy i (i < n): rows [0, copies[2, i]) of page copies[0, i] to page copies[1,
 * i], for every KV head of the K and V pools of `layers` layers (pools [layers,
 * num_pages, n_kv_head, page_size, head_dim] of elements of element_size bytes:
 * 2, or 1 with scales [layers, num_pages, n_kv_head], which are copied too; both
 * scales NULL: none). Rows behind the copied ones are left as they were (in 8
 * bits they then count under the new scale). A source or target below 0 skips
 * the entry, one past the pool, or a row count outside [0, page_size], too, and
 * sets DA_DEVERR_PAGE. A page that one entry writes and another one reads or
 * writes ends up with unspecified rows.
 */
DA_API int kvcache_copy_pages(void* k_pages, void* v_pages, float* k_scale, float* v_scale, const int32_t* copies,
                    int n, int layers, int num_pages, int n_kv_head, int page_size, int head_dim, int element_size,
                    int32_t* err_flag, void* stream);

/*
 * Move rows of sequences together: row keep[keep_start[b] + i] of sequence b goes to
 * row position_ids[b] + i, for i in [0, keep_start[b + 1] - keep_start[b]), in the K
 * and V pools of `layers` layers (as in kvcache_copy_pages, 16 bits). keep
 * (int32 [kept], packed; keep_start int32 [B + 1], rising) holds the rows of
 * accepted drafts, or what stays of a longer part: rising for each sequence,
 * never below the row it goes to. A sequence's rows from the first one on that
 * breaks this, or lies outside [0, max_pages * page_size), are not moved
 * (DA_DEVERR_POSITION), nor is a range that is not inside [0, kept]
 * (DA_DEVERR_TOKENS), nor rows from or to a page outside the pool (DA_DEVERR_PAGE).
 * Every other row is left as it was. Pages that rows move into belong to one
 * sequence (a shared one ends up with unspecified rows).
 */
DA_API int kvcache_compact_paged(void* k_pages, void* v_pages, const int32_t* page_table, const int32_t* keep,
                    const int32_t* keep_start, const int32_t* position_ids, int B, int kept, int layers,
                    int n_kv_head, int head_dim, int num_pages, int page_size, int max_pages, int32_t* err_flag,
                    void* stream);

/*
 * kvcache_compact_paged over pages of e4m3. A page that rows move into gets the
 * largest of its own scale and those of the pages the rows come from (finite, not
 * negative); rows of a smaller scale, the page's other rows among them (all
 * of them, those behind the new ones too), are rounded to it, e4m3(x * old /
 * new). Where no scale differs nothing but the moved rows changes.
 */
DA_API int kvcache_compact_paged_q8(void* k_pages, void* v_pages, float* k_scale, float* v_scale,
                    const int32_t* page_table, const int32_t* keep, const int32_t* keep_start,
                    const int32_t* position_ids, int B, int kept, int layers, int n_kv_head, int head_dim,
                    int num_pages, int page_size, int max_pages, int32_t* err_flag, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H_ */
