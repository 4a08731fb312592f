/*
 * hisparse.h -- C ABI of a GB300 (sm_103a) library for the decode hot path of
 * HiSparse ("HiSparse: Scaling Sparse-Attention Decoding with Hierarchical KV
 * Cache Management", as summarised on marsggbo.github.io, 2026-09-23).
 *
 * The method (summary §3): every request keeps its full per-layer KV history in
 * a host-DRAM pool (pinned; the authoritative copy).  The GPU holds only a
 * fixed B-slot hot buffer per (request, layer) with page-table and recency
 * metadata.  Each decode layer: the indexer hands over k logical positions;
 * RESOLVE looks them up in the hot buffer, fetches the misses from the host
 * pool into evicted slots and publishes the physical slot of every selected
 * position (§5); sparse attention reads exactly those slots (§3 step (4));
 * the new token's KV is written through to the host pool (§3 step (5)).
 *
 * Conventions for every call:
 *   - Pointers named d_* are device pointers (or device-visible managed memory)
 *     owned by the caller; the library never frees them.  Host pointers are
 *     named h_* or src/dst with the rule stated at the call.
 *   - Alignment of device arguments (the kernels move them with vector loads and
 *     stores): d_q, d_out, d_rec and d_kv 16 bytes, d_pos 8 bytes, d_topk and
 *     d_locs 4 bytes.  A misaligned pointer returns HS_ERR_ARG.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - Calls marked CAPTURABLE only enqueue kernels on `stream`: no allocation,
 *     no host synchronisation, no read of device data by the host.  They may be
 *     captured in a CUDA graph and replayed.  Each request of a pool is used from one
 *     stream at a time; disjoint request ranges (the *_range calls) may run on
 *     different streams concurrently.
 *   - Return value: HS_OK (0) or a negative hs_status.  Argument errors found on
 *     the host return at once and enqueue nothing.  Errors that only the device
 *     can see (a bad position in a top-k list, an append out of range, a timed
 *     out wait) set bits in the pool's device error word; the kernel skips the
 *     offending entry; hs_stats reports them and returns HS_ERR_DEVICE_FLAG.
 */
#ifndef HISPARSE_H
#define HISPARSE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct hs_pool hs_pool; /* opaque; owns all pool, buffer and metadata memory */

enum hs_status {
  HS_OK = 0,
  HS_ERR_CONFIG = -1,      /* hs_config rejected (see hs_pool_create) */
  HS_ERR_ALLOC_HOST = -2,  /* pinned host allocation failed */
  HS_ERR_ALLOC_DEV = -3,   /* device allocation failed */
  HS_ERR_ARG = -4,         /* a call argument is out of range or NULL */
  HS_ERR_CUDA = -5,        /* a CUDA runtime call failed */
  HS_ERR_DEVICE_FLAG = -6, /* hs_stats: a kernel recorded an error bit */
  HS_ERR_SCRATCH = -7      /* hs_sparse_attn_noalloc: the call needs more than its fixed scratch */
};

enum hs_policy {
  HS_POLICY_LRU = 0,          /* summary §4-§5: evict the least recently used, update in place */
  HS_POLICY_FIFO = 1,         /* §4: evict the earliest inserted */
  HS_POLICY_RANDOM = 2,       /* §4: evict at random (counter-based hash, reproducible) */
  HS_POLICY_SWAP_VANILLA = 3  /* §4: keep only the current top-k, no hot set */
};

enum hs_layout {
  HS_LAYOUT_MLA = 0, /* one shared latent of head_dim_qk bf16 per token; V = its first head_dim_v values */
  HS_LAYOUT_GQA = 1  /* per token num_kv_heads blocks of [K (head_dim_qk) | V (head_dim_v)] bf16 */
};

/* bits of the device error word */
enum hs_device_error {
  HS_DEVERR_RANGE = 1,    /* a top-k entry outside [0, capacity) other than -1 */
  HS_DEVERR_DUP = 2,      /* a top-k entry repeating an earlier one in the same list */
  HS_DEVERR_CLOCK = 4,    /* the 32-bit recency clock of a (request, layer) would wrap */
  HS_DEVERR_APPEND = 8,   /* an append position outside [shared_prefix, capacity), or on a host
                             page not reserved (hs_reserve) */
  HS_DEVERR_LOC = 16,     /* an attention slot index outside [0, rows) */
  HS_DEVERR_TIMEOUT = 32, /* a bounded wait inside a kernel gave up */
  HS_DEVERR_PAGE = 64,    /* a miss fetch read a position whose host page is not reserved (the
                             slot keeps its old contents) */
  HS_DEVERR_SLOTS = 128   /* a resolve or append on a (request, layer) whose device buffer holds
                             fewer than top_k slots (device_pool_slots > 0 and not reserved):
                             the call changed nothing for it and its locations are -1 */
};

typedef struct {
  int32_t num_requests;   /* R >= 1 */
  int32_t num_layers;     /* L >= 1 */
  int64_t capacity;       /* C: positions per (request, layer), prefill plus appends */
  int64_t shared_prefix;  /* positions [0, shared_prefix) are ONE history shared by all requests
                             (read-only for appends); 0 = every request owns its whole history */
  int32_t layout;         /* hs_layout */
  int32_t num_q_heads;    /* Hq */
  int32_t num_kv_heads;   /* GQA: KV heads per token (Hq % num_kv_heads == 0); MLA: 1 */
  int32_t head_dim_qk;    /* MLA 576, GQA 128 */
  int32_t head_dim_v;     /* MLA 512, GQA 128 */
  int32_t top_k;          /* k, 1 <= k <= buffer_slots, k <= 4096 (shared-memory hash) */
  int32_t buffer_slots;   /* B: hot-buffer slots per (request, layer), <= 16384 */
  int32_t policy;         /* hs_policy */
  uint64_t seed;          /* key of HS_POLICY_RANDOM */
  int32_t io_chunk_bytes; /* bytes one thread moves per batch of loads in a miss fetch:
                             16..128, a power of two dividing the record size (summary §5: the
                             per-thread transfer size of the swap-in is a tuned knob) */
  int32_t log_steps;      /* >0: keep per-step miss counts of the first log_steps resolves */
  int32_t fetch_in_attention; /* 0: hs_resolve copies the misses into their slots (summary §5).
                                 1: hs_resolve only decides; the next hs_sparse_attn of the layer
                                 reads the missing records straight from the host history while it
                                 gathers the resident ones from HBM, and writes them to their
                                 slots, so the host-link transfer overlaps the HBM-bound attention.
                                 Copies left pending when no attention follows are finished by the
                                 next hs_resolve or hs_append_writethrough of that layer.  Needs
                                 the GQA layout. */
  int32_t host_page_tokens;   /* positions per host page (summary §8, the memory layer allocates
                                 the host pool in pages): 0 = automatic (1024, or the largest power
                                 of two <= 1024 dividing shared_prefix); else a power of two that
                                 divides shared_prefix */
  int32_t host_on_demand;     /* 0: every page of [0, capacity) is reserved at pool creation.
                                 1: pages are reserved on demand: by hs_prefill_write for the
                                 positions it writes and by hs_reserve ahead of appends; a
                                 request's private pages return to the pool with hs_release. */
  int32_t buffer_page_slots;  /* slots per device buffer page: 0 = automatic (the smallest power of
                                 two >= 16 that cuts B into at most 64 pages); else a power of two
                                 with ceil(B / buffer_page_slots) <= 64 */
  int64_t device_pool_slots;  /* summary §8, the coordinator allocates and grows the per-request,
                                 per-layer device cache on demand.  0: every (request, layer) buffer
                                 holds all B slots from creation.  > 0: the device cache pool holds
                                 this many slots (rounded up to whole pages); a buffer holds only
                                 the pages hs_reserve gave it -- min(B, max(end, top_k)) slots
                                 rounded up to a page -- and
                                 resolve and append use its slots [0, that count) alone.  With the
                                 growth kept ahead of the positions a request uses, every result is
                                 identical to the full buffer's. */
  double host_to_device_ratio; /* > 0: the pinned host history may hold at most this many times the
                                  device cache pool's bytes; reservations beyond fail with
                                  HS_ERR_ALLOC_HOST.  0: no bound. */
  int32_t early_fetch;        /* summary §5 step 4 (the swap-in), started before the decision ends.
                                 0: each hs_resolve cluster fetches its misses once it has chosen
                                 the victims.  1: every hs_resolve launch also runs one cluster of
                                 fetch CTAs per request, which do the whole miss fetch.  From the
                                 launch's start they copy the records that look missing (from the
                                 slot each position was last installed in: a device map position
                                 -> slot, confirmed by the slot's tag) from the host history into
                                 a device scratch, up to about top_k / 4 per (request, layer).
                                 Once the deciding CTAs have chosen the victims, the fetch CTAs
                                 install every miss in its slot: from the scratch when they have
                                 it, else from the host.  Results are identical to mode 0.  Extra
                                 device memory per (layer, request): 4 x capacity bytes for the
                                 map, the scratch (about top_k / 4 records) and 4 x top_k bytes.
                                 Needs fetch_in_attention = 0. */
} hs_config;

/* Record size in bytes for a configuration (MLA: 2*head_dim_qk; GQA: 2*kv_heads*(qk+v)). */
int64_t hs_record_bytes(const hs_config* cfg);

/*
 * Create a pool on `cuda_device` (summary §3, §8 "memory layer").
 *   - Host history: pinned, device-mapped pages of host_page_tokens records, carved from large
 *     pinned slabs.  A device page table [R][L][ceil(capacity / page)] maps every (request, layer,
 *     position) to its page.  The pages of [0, shared_prefix) are one copy per layer, mapped into
 *     every request's table.
 *   - Hot buffers in HBM: one device cache pool of pages of buffer_page_slots slots x rec bytes; a
 *     device slot table [L][R][ceil(B / page)] maps each (layer, request, slot) to its page.  Tags
 *     [L][R][B] (-1 = empty), stamps (0 = empty), per-(request, layer) clock (starts at 1),
 *     counters and attention workspace.  All slots start empty.
 * With host_on_demand = 0 every host page is reserved here; else none is.  With
 * device_pool_slots = 0 every buffer gets all its pages here; else none does.  Synchronous, not
 * capturable.  Errors: HS_ERR_CONFIG, HS_ERR_ALLOC_HOST, HS_ERR_ALLOC_DEV, HS_ERR_CUDA.
 * Environment HS_FAULT=alloc_host|alloc_dev makes the named allocation fail (for tests).
 */
int hs_pool_create(const hs_config* cfg, int cuda_device, hs_pool** out);

/* Free everything the pool owns.  Synchronises the device.  NULL is accepted. */
int hs_pool_destroy(hs_pool* pool);

/* Cold start: empty every slot, reset clocks, counters, error word and step log.  CAPTURABLE. */
int hs_pool_reset(hs_pool* pool, void* stream);

/*
 * Prefill write (summary §3 step (1)): copy n records from `src` (host or device memory,
 * [n][rec] bytes) into the host history of (req, layer) at positions [pos0, pos0 + n).
 * Positions below shared_prefix go to the shared history whatever `req` is.  Reserves the pages
 * it writes (synchronously), then enqueues the copy on `stream`; the caller keeps `src` alive
 * until the stream reaches this point.  Writes only the host pool; the hot buffer is filled on
 * demand by hs_resolve (a device buffer grown on demand grows only by hs_reserve).
 * Errors: HS_ERR_ARG, HS_ERR_ALLOC_HOST, HS_ERR_CUDA.
 */
int hs_prefill_write(hs_pool* pool, int req, int layer, int64_t pos0, int64_t n, const void* src,
                     void* stream);

/*
 * Write-through append (summary §3 step (5)): for every request r, record d_rec[r] (bf16,
 * [R][rec] bytes, device) becomes position d_pos[r] (int64 [R], device) of (r, layer): it is
 * stored to the host history (16-byte stores through the device mapping) and into the hot
 * buffer -- in the slot already holding d_pos[r] if any, else the slot the policy would evict
 * first over all B slots -- with stamp = clock, clock += 1.  Positions outside
 * [shared_prefix, capacity) set HS_DEVERR_APPEND and are skipped.  CAPTURABLE.
 */
int hs_append_writethrough(hs_pool* pool, int layer, const int64_t* d_pos, const void* d_rec, void* stream);

/*
 * Fused RESOLVE (summary §5).  The summary runs one CTA per request; here a thread-block cluster
 * serves each request: every CTA of the cluster computes the whole decision below from the same
 * inputs, then writes its share of the slots and fetches its share of the misses, so one request's
 * host copies are spread over several SMs.  The cluster holds the largest of 8, 4 or 2 CTAs for
 * which every request's cluster fits on the GPU at once (fixed at hs_pool_create), else 1.
 * The decision: hash the k positions of d_topk[r]
 * (int32 [R][k], device; -1 = padding) in shared memory, probe all B slots for hits, choose
 * the m victims among the slots holding no selected position (smallest eviction key, then
 * lowest slot; victims in ascending slot order take the misses in top-k order), update the
 * recency stamps in place (hits to MRU in top-k order, misses after the hits), fetch each
 * missing record from the pinned host history with 16-byte loads straight into its slot,
 * and write d_locs[r][i] = slot of d_topk[r][i] (-1 for padding or invalid entries; int32
 * [R][k], device).  Updates hits/misses/host-byte counters.  With early_fetch = 1 a second cluster
 * per request does the whole miss fetch, starting at the launch's start (see hs_config).
 * CAPTURABLE.
 */
int hs_resolve(hs_pool* pool, int layer, const int32_t* d_topk, int32_t* d_locs, void* stream);

/*
 * hs_append_writethrough followed by hs_resolve for the same layer, fused into one kernel (the
 * append's slot choice and the resolve's decision are made by the same resolve cluster): results,
 * state and counters are identical to the two calls in sequence.  Arguments as for those calls.
 * CAPTURABLE.
 */
int hs_append_resolve(hs_pool* pool, int layer, const int64_t* d_pos, const void* d_rec, const int32_t* d_topk,
                      int32_t* d_locs, void* stream);

/*
 * Sparse attention over resolved slots (summary §3 step (4)): for request r and query head h,
 *   out[r][h] = sum_i softmax_i(scale * <q[r][h], K(row_i)>) V(row_i)
 * over the entries i with d_locs[r][i] >= 0, in top-k order, with K/V taken from the record
 * layout (MLA: K = the latent, V = its first head_dim_v values; GQA: KV head h/(Hq/Hkv)).
 * d_q: bf16 [R][Hq][head_dim_qk]; d_out: fp32 [R][Hq][head_dim_v]; both device.
 * kv_base == NULL: rows are the hot-buffer slots of `layer` (kv_rows ignored).  Otherwise
 * kv_base is a caller-owned device array [R][kv_rows][rec] and d_locs index its rows
 * (fully resident KV: used to check the exactness property).  A request with no valid entry
 * gets zeros.  Entries >= rows set HS_DEVERR_LOC and are skipped.  The reduction order
 * depends only on the top-k order, so the result is bit-identical whichever slots hold the
 * records.  Enqueued directly after hs_resolve / hs_append_resolve of the same layer on the same
 * stream (nothing of this pool in between), the attention of a request may start as soon as that
 * request's resolve is done, before the rest of the resolve; results are the same either way.
 * CAPTURABLE.
 */
int hs_sparse_attn(hs_pool* pool, int layer, const void* d_q, const int32_t* d_locs, const void* kv_base,
                   int64_t kv_rows, float scale, float* d_out, void* stream);

/* Size of the fixed device scratch that hs_sparse_attn_noalloc uses on every GPU (8 MiB + 64 KiB). */
#define HS_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u + 64u * 1024u)

/*
 * Sparse attention over caller-resident KV that allocates nothing.  The paper has no counterpart:
 * this is a convenience of this library for callers that must not call cudaMalloc at all, for
 * example code inside an inference engine whose own allocator owns all device memory, or a
 * process that must keep its device footprint fixed after start-up.  Creating a pool would
 * allocate the host history and the hot buffers; this call needs none of that.
 *
 * It computes exactly what hs_sparse_attn computes with a non-NULL kv_base, with the same
 * kernels and the same split plan, so the two give bit-identical outputs: for request r and query
 * head h, softmax(scale * <q, K(row)>)-weighted V over the rows d_locs[r][i] >= 0 of d_kv, in
 * top-k order.  Only these fields of *cfg are read: num_requests, layout, num_q_heads,
 * num_kv_heads, head_dim_qk, head_dim_v, top_k (pool settings such as fetch_in_attention are
 * ignored).
 *   d_q    : bf16 [R][Hq][head_dim_qk], device          d_locs : int32 [R][k], device
 *   d_kv   : bf16 [R][kv_rows][record], device, 16-byte aligned
 *   d_out  : fp32 [R][Hq][head_dim_v], device
 * The split partials live in one file-scope device array of HS_NOALLOC_SCRATCH_BYTES per GPU,
 * loaded with the library and held until the process exits.  A shape whose partials do not fit
 * returns HS_ERR_SCRATCH before anything is enqueued (about R * splits * Hq * (head_dim_v + 2) * 4
 * bytes; splits <= number of SMs / R).  Each call first clears the combine tickets and the error
 * word it uses and fills d_out with NaN.
 * The first call on a device (with that device current) looks up the scratch's device address
 * and raises the kernels' shared-memory limits; make that first call before any stream capture.
 * Every call on a device shares the one array and finds the previous call's leftovers there:
 * calls that may overlap on the GPU (different streams without ordering) race and corrupt each
 * other's results.  Rows outside [0, kv_rows) are skipped and not reported.  A bounded wait inside
 * a kernel that gives up (about a second without progress, a stalled GPU) leaves the affected
 * requests' outputs NaN; there is no pool whose error word could report it.
 * Errors: HS_ERR_ARG, HS_ERR_CONFIG, HS_ERR_SCRATCH, HS_ERR_CUDA.
 */
int hs_sparse_attn_noalloc(const hs_config* cfg, const void* d_q, const int32_t* d_locs, const void* d_kv,
                           int64_t kv_rows, float scale, float* d_out, void* stream);

/*
 * Request-range forms (summary §3: requests are independent; each one's layers stay in order).
 * They act on requests [r0, r0 + nreq) only; d_topk, d_locs, d_pos, d_rec, d_q and d_out hold
 * rows for those requests, the first row being request r0.  hs_resolve_range fuses the
 * write-through append when d_pos and d_rec are both non-NULL (both NULL: plain resolve).
 * hs_sparse_attn_range reads the hot buffer.  Calls on disjoint ranges touch disjoint state, so
 * two micro-batches of one pool can run on two streams and overlap one's host-link fetch with the
 * other's HBM-bound attention.  Errors: HS_ERR_ARG for an empty or out-of-range span.  CAPTURABLE.
 */
int hs_resolve_range(hs_pool* pool, int layer, int r0, int nreq, const int64_t* d_pos, const void* d_rec,
                     const int32_t* d_topk, int32_t* d_locs, void* stream);
int hs_sparse_attn_range(hs_pool* pool, int layer, int r0, int nreq, const void* d_q, const int32_t* d_locs,
                         float scale, float* d_out, void* stream);

typedef struct {
  uint64_t hits;
  uint64_t misses;
  uint64_t appends;
  uint64_t host_bytes;  /* bytes fetched from the host history by hs_resolve */
  uint32_t error_bits;  /* OR of all hs_device_error bits */
  uint32_t resolves;    /* hs_resolve calls counted on (request 0, layer 0) */
} hs_totals;

/*
 * Read the device counters (synchronises the device; not capturable).  Any output may be NULL.
 *   h_counters : uint64 [R][L][4]  (hits, misses, appends, host_bytes) per (request, layer)
 *   h_errors   : uint32 [R][L]     error bits per (request, layer)
 *   h_step_log : uint32 [log_steps][R][L] misses of the t-th resolve of (r, l)
 * reset != 0 zeroes the counters, error bits and step log afterwards (not the cache state).
 * Returns HS_ERR_DEVICE_FLAG when any error bit is set, after filling the outputs.
 */
int hs_stats(hs_pool* pool, hs_totals* totals, uint64_t* h_counters, uint32_t* h_errors, uint32_t* h_step_log,
             int reset);

/*
 * Inspection (synchronous, not capturable): copy the metadata of `layer` to host memory.
 *   h_tag: int32 [R][B]; h_stamp: uint32 [R][B]; h_clock: uint32 [R]; any may be NULL.
 */
int hs_read_state(hs_pool* pool, int layer, int32_t* h_tag, uint32_t* h_stamp, uint32_t* h_clock);

/* Inspection: copy the hot buffer of (req, layer), [B][rec] bytes, to host memory `dst`; slots
 * the buffer does not hold read as zeros. */
int hs_read_buffer(hs_pool* pool, int req, int layer, void* dst);

/* Inspection: copy n records of the host history of (req, layer) from position pos0 to `dst`;
 * positions on pages not reserved read as zeros. */
int hs_read_history(hs_pool* pool, int req, int layer, int64_t pos0, int64_t n, void* dst);

/*
 * Memory layer (summary §8: paged host pool and device cache pool, grown on demand): reserve the
 * host pages of (req, layer) that cover positions [0, end) -- layer = -1: every layer -- so that
 * appends up to `end` have somewhere to go, and (device_pool_slots > 0) grow its device buffer to
 * min(B, max(end, top_k)) slots rounded up to a page.  Pages of the shared prefix are reserved
 * once per layer.  Nothing is reserved when the call fails.  Synchronous (it updates the device
 * tables); call it outside captured graphs, before the decode steps that use those positions.
 * Errors: HS_ERR_ARG, HS_ERR_ALLOC_HOST, HS_ERR_ALLOC_DEV (device cache pool exhausted), HS_ERR_CUDA.
 */
int hs_reserve(hs_pool* pool, int req, int layer, int64_t end);

/*
 * End request `req` (every layer): its private host pages, and with device_pool_slots > 0 its
 * device buffer pages, return to the free lists for reuse by later reservations; the shared prefix
 * stays.  Its buffers are emptied (tags -1, stamps 0, clock 1, resolve count 0, error bits 0, no
 * copies pending), so a new request in this index starts cold; its counters are kept.  The
 * request's history reads as zeros afterwards.  Synchronises the device first.
 * Errors: HS_ERR_ARG, HS_ERR_CUDA.
 */
int hs_release(hs_pool* pool, int req);

/*
 * Test hook for the bounded waits (not for production use): the next launch of each kernel named in
 * `kernels` leaves one mbarrier arrival out, so that the wait for it gives up after its limit (about
 * one second) instead of completing.  The kernel then reports HS_DEVERR_TIMEOUT (hs_stats) and
 * returns; its outputs for that launch are undefined, and the cache state of a resolve that gave up
 * no longer matches its history (call hs_pool_reset).  The context stays usable.
 *   HS_STALL_ATTN    : the 64-head shared-latent tensor-core attention (the producers' arrival on
 *                      the first ring slot), consumed by the next launch of that kernel
 *   HS_STALL_RESOLVE : the resolve (the arrival that completes the early miss copies), consumed by
 *                      the next resolve launch that stages early copies
 *   HS_STALL_FETCH   : the resolve's fetch CTAs (early_fetch = 1): the deciding CTAs of the
 *                      launch's first request never signal that the victims are chosen, so that
 *                      request's fetch CTAs give up waiting and install nothing.  Consumed by the
 *                      next resolve launch with fetch CTAs.
 *   HS_STALL_TREE    : hs_pool_tree_attn on the tensor cores (an arrival of one CTA's first tile),
 *                      consumed by the next hs_pool_tree_attn; the cache is not touched, so no reset
 *                      is needed
 * Host-side only (takes effect at launch, also when the launch is captured).  Errors: HS_ERR_ARG.
 */
enum { HS_STALL_ATTN = 1, HS_STALL_RESOLVE = 2, HS_STALL_FETCH = 4, HS_STALL_TREE = 8 };
int hs_debug_stall_next(hs_pool* pool, int kernels);

/*
 * Speculative decoding over a cache: the T drafted tokens ("nodes") of a request form a tree that hangs
 * from its last token.  Three operators go round in a loop: append the drafts' records (rotated) behind
 * the context, attend all nodes at once over the context and each other, keep the accepted path.  The
 * summary has no counterpart; they stand beside hs_append_writethrough, hs_sparse_attn and
 * hs_sparse_attn_noalloc.
 *
 * They work on a cache that the caller keeps in device memory in pages, or (hs_pool_tree_attn) on a
 * pool's hot buffers.  Records have the layouts of hs_config; of the hs_config these calls read only
 * num_requests (<= 65535), layout, num_q_heads, num_kv_heads, head_dim_qk and head_dim_v (head dims:
 * multiples of 8, at most 576).  No call allocates or synchronises; all are CAPTURABLE.  `stream`
 * belongs to kv->cuda_device; the current device does not matter.
 */
typedef struct {
  void* d_pages;          /* bf16 [num_pages][page_tokens][record], 16-byte aligned */
  const int32_t* d_table; /* [num_requests][max_pages]: position p of request r is row p % page_tokens of
                             page d_table[r][p / page_tokens].  NULL: request r owns the pages
                             [r * max_pages, (r + 1) * max_pages) in order */
  int64_t num_pages;      /* num_pages * page_tokens <= 2^31 - 1 */
  int32_t page_tokens;    /* >= 1, any number */
  int32_t max_pages;      /* pages of a request: positions [0, max_pages * page_tokens), at
                             most 2^31 - 65536 */
  uint32_t* d_err;        /* device word that errors only the device sees are OR'ed into, or NULL */
  int32_t cuda_device;
} hs_paged_kv;

/*
 * Rotation tables.  The angle of position a for rotary pair j is a * inv_freq[j]; h_turns[j] =
 * inv_freq[j] / (2 pi) mod 1 as a 64-bit binary fraction, correctly rounded, so that a * h_turns[j] mod
 * 2^64 is the angle in turns with an error of a * 2^-65: far positions turn as exactly as near ones.  Host
 * arrays of n; errors: HS_ERR_ARG (NULL, n < 0, a frequency that is not below 2^32 in magnitude).
 */
int hs_rope_turns(const double* h_inv_freq, int n, uint64_t* h_turns);

typedef struct {
  int32_t num_tokens;         /* N >= 0 rows of the token arrays */
  const int32_t* d_cu;        /* [num_requests + 1] ascending: tokens [cu[r], cu[r+1]) belong to request r;
                                 tokens outside [cu[0], cu[num_requests]) are padding: nothing is read or
                                 written for them */
  const int64_t* d_start;     /* [num_requests]: token t of request r is stored at position start[r] + t - cu[r] */
  const int64_t* d_rope_pos;  /* [N] position whose angle a token gets (a drafted node: its depth), or NULL:
                                 the position where it is stored */
  const void* d_k;            /* bf16 [N][num_kv_heads][head_dim_qk]; MLA: the latent */
  int64_t k_token_stride, k_head_stride; /* in values; strides and addresses: multiples of 16 bytes */
  const void* d_v;            /* GQA: bf16 [N][num_kv_heads][head_dim_v]; MLA: NULL */
  int64_t v_token_stride, v_head_stride;
  const uint64_t* d_turns;    /* [rotary_dim / 2] of hs_rope_turns, device; NULL when rotary_dim = 0 */
  int32_t rotary_dim;         /* rotated values of a head, a multiple of 16; 0: nothing is rotated */
  int32_t rotary_offset;      /* the first of them in K, a multiple of 8 (MLA: usually head_dim_v) */
  int32_t interleaved;        /* 0: value j turns with j + rotary_dim / 2; 1: value 2j with 2j + 1 */
  const void* d_q;            /* bf16 [N][num_q_heads][q_dim], or NULL: no queries */
  int64_t q_token_stride, q_head_stride;
  void* d_q_out;              /* the queries rotated; may be d_q itself with the same strides */
  int64_t q_out_token_stride, q_out_head_stride;
  int32_t q_dim;              /* head_dim_qk (rotated at rotary_offset, the rest copied) or rotary_dim
                                 (all of it rotated) */
} hs_append_args;

/*
 * Append to a paged cache with the rotation applied on the way: every token's key (its rotary part
 * turned by its position) and value become the record at its position; queries are turned in the same
 * launch.  Records of a call go to distinct positions by construction; pages that two requests share
 * must not be written by two of them in one call.  A position outside [0, max_pages * page_tokens) sets
 * HS_DEVERR_APPEND, a table entry outside [0, num_pages) HS_DEVERR_PAGE; that record is skipped (its
 * query is still rotated).  The sines and cosines are within 1e-6 for positions below 2^40, products
 * and sums are 32-bit, results are rounded once to bf16.  Errors: HS_ERR_ARG, HS_ERR_CONFIG, HS_ERR_CUDA.
 */
int hs_append_rotated(const hs_config* cfg, const hs_paged_kv* kv, const hs_append_args* args, void* stream);

#define HS_MAX_TREE_NODES 256

typedef struct {
  const void* d_q;         /* bf16 [num_requests][nodes][num_q_heads][head_dim_qk], 16-byte aligned */
  const int64_t* d_len;    /* [num_requests] context length; node j is the record at position len + j */
  const int32_t* d_locs;   /* NULL: the context is every position [0, len).  Else [num_requests][top_k]
                              positions, -1 = padding, in any order: only those */
  int32_t top_k;           /* with d_locs: 1 .. 2^31 - 65536; ignored without */
  const uint64_t* d_mask;  /* [num_requests][nodes][ceil(nodes / 64)]: bit j of node i's words is set when
                              i sees node j (itself included).  Any pattern is accepted */
  const int32_t* d_nodes;  /* [num_requests] nodes in use (0 .. nodes), or NULL: all of them.  Output rows
                              behind them are left as they were */
  int32_t nodes;           /* T, 1 .. HS_MAX_TREE_NODES */
  float scale;             /* magnitude below 2.35e38: scale * log2(e) is a finite 32-bit number */
  void* d_out;             /* bf16 [num_requests][nodes][num_q_heads][head_dim_v], 16-byte aligned; apart from d_q */
  void* d_workspace;       /* hs_tree_attn_workspace bytes, 16-byte aligned; used by this call alone until
                              it is done: calls that may overlap need one each */
  int64_t workspace_bytes;
} hs_tree_args;

/* Bytes of workspace a tree attention of `nodes` nodes needs on `cuda_device`, whatever the lengths (0 is
 * possible); negative: an hs_status. */
int64_t hs_tree_attn_workspace(const hs_config* cfg, int nodes, int cuda_device);

/*
 * Attention of a tree of drafted tokens over a paged cache: for request r, node i and query head h,
 *   out[r][i][h] = sum_e softmax_e(scale * <q[r][i][h], K(e)>) V(e)
 * over the context's entries and the nodes j that i sees.  How often a context record is read: heads of 64 or 128
 * (keys and values alike, G <= 128 query heads a KV head) once for every two tiles of floor(128 / G) nodes; latents of
 * 576 values (512 of them V) once for every 128 (node, query head) rows; both run on the tensor cores.  Any other shape
 * runs on CUDA cores and reads a record once for every node and query head: 3 to 11 times the time of plain
 * matrix products on batches (80-value heads, 16 requests x 8 nodes over 2048 listed positions: 4.1 ms, where
 * 128-value heads take 41 us).  Nothing visible gives zeros.  What a node does not see has no
 * influence on it, whatever its values (NaN and infinities included).  What it does see counts however small its
 * weight, even one that is 0 (a score of -infinity) or rounds to it: an infinite or NaN value makes that dim of the
 * output infinite or NaN, a NaN score the whole row.  A row whose visible scores are all -infinity
 * gives zeros where the values are finite.  Positions outside
 * [0, max_pages * page_tokens) set HS_DEVERR_LOC, bad table entries HS_DEVERR_PAGE: such
 * entries are not seen.  A len < 0 sets HS_DEVERR_LOC and leaves neither context nor nodes (a list is still
 * read); a node count outside [0, nodes] sets it and is clamped.  Scores, softmax sums and accumulators
 * are 32-bit; the weights enter the value product as bf16 for the shapes on the tensor cores, and the
 * output is rounded once to bf16.  The order of the sums depends on the lengths alone: equal calls give
 * equal bits.  A bounded wait inside a kernel that gives up (about a second without progress, a stalled GPU) sets
 * HS_DEVERR_TIMEOUT and leaves d_out undefined; the cache is only read, and the next call works.  With d_err NULL
 * nothing reports that, nor any other error of the device's.
 * Errors: HS_ERR_ARG, HS_ERR_CONFIG, HS_ERR_SCRATCH (workspace too small), HS_ERR_CUDA.
 */
int hs_tree_attn(const hs_config* cfg, const hs_paged_kv* kv, const hs_tree_args* args, void* stream);

/*
 * The same over the hot buffers of a layer: args->d_locs are the slots that hs_resolve published
 * ([num_requests][cfg.top_k]; args->top_k and d_len are ignored), shared by all nodes of a request, and
 * d_draft (bf16 [num_requests][nodes][record], device, 16-byte aligned) holds the nodes' records, which
 * are in no pool yet.  Slots outside the buffer set HS_DEVERR_LOC (hs_stats).  Pools with
 * fetch_in_attention = 1 are refused (HS_ERR_CONFIG): their misses are copied by hs_sparse_attn alone.
 */
int hs_pool_tree_attn(hs_pool* pool, int layer, const hs_tree_args* args, const void* d_draft, void* stream);

/*
 * Keep the accepted path of a tree: for i in [0, count[r]) the record at position len[r] + i becomes the
 * one that was at position len[r] + path[r][i] before the call.  d_path int32 [num_requests][path_len],
 * node numbers with path[r][i] >= i (the nodes of a path ascend, so this holds for every tree whose
 * parents come first); another entry sets HS_DEVERR_LOC and is skipped, as is one whose position is
 * outside the cache; a count outside [0, path_len] sets HS_DEVERR_LOC and is clamped.  Pages that two requests
 * share must not hold records that this call moves or overwrites.  d_len int64, d_count int32
 * [num_requests].  Errors: HS_ERR_ARG, HS_ERR_CONFIG, HS_ERR_CUDA.
 */
int hs_keep_path(const hs_config* cfg, const hs_paged_kv* kv, const int64_t* d_len, const int32_t* d_path, int path_len,
                 const int32_t* d_count, void* stream);

/* Host memory of the pool: pages mapped in some table, pages on the free list, pinned bytes held. */
int hs_host_usage(hs_pool* pool, int64_t* pages_in_use, int64_t* pages_free, int64_t* bytes_pinned);

/* Device cache pool: pages held by some buffer, pages free, slots per page. */
int hs_device_usage(hs_pool* pool, int64_t* pages_in_use, int64_t* pages_free, int64_t* page_slots);

#ifdef __cplusplus
}
#endif

#endif /* HISPARSE_H */
