/*
 * dkv.h — C ABI of the zero-copy host-resident KV-cache attention library.
 *
 * The method is DirectKV ("No Buffer, No Bottleneck: Efficient Zero-Copy KV
 * Cache Offloading for Long-Context LLMs").  Its pieces, as the pages
 * describe them:
 *   - KV Cache Manager: K/V tensors live in pinned host memory allocated with
 *     cudaHostAlloc and are read by GPU kernels through zero-copy pointers;
 *     once written they stay there across decode iterations ("Paper Notes:
 *     DirectKV", System Architecture, KV Cache Manager).
 *   - Attention Fusion Engine: one kernel computes the K/V projection of the
 *     new token(s), keeps the fresh K/V on chip and runs attention over the
 *     host-resident cache (same page, System Architecture and Key Ideas (2)).
 *     Prefill iterates over HBM-resident Q for each host K/V tile; decode
 *     iterates over all cached K/V for the single new query (same page,
 *     System Architecture, prefill/decode strategies).
 *   - CPU-memory-aware tiling: a host K/V tile is fetched once and reused by
 *     every query tile and head that needs it (same page, Key Ideas (1)).
 *   - Kernel Adaptor: picks a precompiled kernel by dtype, head dim, tile and
 *     phase (same page, System Architecture, Kernel Adaptor).
 * The attention computed is softmax(Q.K^T / sqrt(d)).V with K = X.Wk,
 * V = X.Wv (same page, Fundamental Underlying Technologies, Kernel Fusion).
 *
 * Conventions for every call:
 *   - Shapes: B batch, T new tokens per sequence, H hidden, Hq query heads,
 *     Hkv KV heads (Hq a multiple of Hkv; query head h uses KV head
 *     h / (Hq/Hkv)), D head dim.
 *   - x is [B, T, H]; Wq is [H, Hq*D]; Wk and Wv are [H, Hkv*D]; out is
 *     [B, T, Hq, D]; all row-major, all in the cache's dtype, all DEVICE
 *     pointers owned by the caller.
 *   - The K cache and the V cache are each [B][Hkv][max_tokens][D] in pinned,
 *     mapped host memory owned by the library (dense caches; paged caches
 *     hold pools of pages, layered caches one such pair per layer, see
 *     their allocators).  Elements are the dtype, or 8-bit E4M3 for caches
 *     allocated with that format.
 *   - A stream argument is a cudaStream_t passed as void* (NULL = the legacy
 *     default stream).  Work is enqueued; nothing waits for the GPU unless
 *     the call says so.
 *   - No call throws.  Argument, capacity and support errors return before
 *     anything is enqueued and leave the cache unchanged.  dkv_last_error()
 *     gives a thread-local detail string for the last failure.
 */
#ifndef DKV_H
#define DKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DKV_OK = 0,
    DKV_ERR_INVALID_ARG = 1,      /* null pointer, bad size, bad handle */
    DKV_ERR_UNSUPPORTED = 2,      /* no precompiled kernel for (dtype, D, G), or a
                                     call that this kind of cache does not serve */
    DKV_ERR_CAPACITY = 3,         /* length + T would exceed max_tokens, or a row
                                     of a paged cache has no page */
    DKV_ERR_NO_MAPPED_MEMORY = 4, /* the device cannot map host memory */
    DKV_ERR_ALLOC = 5,            /* pinned host or device allocation failed */
    DKV_ERR_CUDA = 6,             /* a CUDA runtime call failed */
    DKV_ERR_TIMEOUT = 7           /* a bounded device-side wait gave up */
} dkv_status;

typedef enum { DKV_BF16 = 0, DKV_FP16 = 1 } dkv_dtype;

typedef struct dkv_cache dkv_cache; /* opaque; tagged so a stale handle is rejected */

/* What the cache stores per K/V element: the dtype itself (2 bytes), or 8-bit
 * E4M3 (OCP 8-bit floating point; 1 sign, 4 exponent, 3 mantissa bits; no
 * infinities; largest finite 448), unscaled and saturating.  E4M3 halves the
 * bytes the attention reads across the host link (the FP8 KV cache that
 * "KV Offloading and Transfer" lists among the cheaper things to do first,
 * in section 6, When it's worth it; not part of DirectKV's pages).  New
 * rows are the fp32 projection sums rounded once to E4M3 (to nearest, ties
 * to even, saturating); decode only, bf16 activations only. */
typedef enum {
    DKV_KV_NATIVE = 0,
    DKV_KV_E4M3 = 1,
    /* 4-bit E2M1 codes (OCP FP4: 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign) with one
     * E4M3 scale per 16 elements: 9/16 byte an element.  Paged caches only, pages
     * of 16 to 4096 tokens, both dtypes.  A page of one KV head is one run of
     * bytes: page_tokens rows of head_dim/2 code bytes (element 2i in the low
     * four bits of byte i), then page_tokens rows of head_dim/16 scale bytes;
     * a pool is [num_pages][n_kv_heads][page_tokens * head_dim * 9 / 16].  Served by
     * dkv_qkv_append and dkv_paged_attend; the calls that project, decode or
     * prefill through the cache handle return UNSUPPORTED for it. */
    DKV_KV_E2M1 = 2
} dkv_kv_format;

/* Everything a cache can be: dense (page_tokens 0), paged (page_tokens > 0,
 * one layer), layered (layers > 1, dense), in either element format.
 * layers 0 counts as 1. */
typedef struct {
    int batch, n_kv_heads, head_dim, max_tokens;
    dkv_dtype dtype;
    dkv_kv_format kv_format;
    int layers;
    int page_tokens, num_pages, max_pages_per_seq;
} dkv_cache_desc_t;

/* Sizes of what a cache holds (the pages' memory accounting: zero bytes of
 * HBM staging; "Paper Notes: DirectKV", Experiments, GPU memory). */
typedef struct {
    size_t host_pinned_bytes;  /* K + V caches in pinned, mapped host memory */
    size_t device_workspace_bytes; /* library-owned HBM for q, fresh K/V, partials */
    size_t device_staging_bytes;   /* HBM copies of the cache: always 0 */
    int batch, n_kv_heads, head_dim, max_tokens, dtype;
    int page_tokens;        /* paged caches: rows per page; 0 for a dense cache */
    int num_pages;          /* paged caches: pages in each of the K and V pools */
    int max_pages_per_seq;  /* paged caches: page-table entries per sequence */
    int layers;             /* layered caches: layers held (1 otherwise) */
    int kv_format;          /* dkv_kv_format of the K/V elements */
    int numa_node_wanted;   /* host NUMA node attached to the cache's GPU (-1: unknown) */
    int numa_node;          /* node holding the cache's first page (-1: unknown) */
} dkv_cache_info_t;

/* Allocate a K cache and a V cache of [batch][n_kv_heads][max_tokens][head_dim]
 * elements each with cudaHostAlloc(Mapped | Portable) and obtain their device
 * aliases with cudaHostGetDevicePointer (KV Cache Manager, "Paper Notes:
 * DirectKV", System Architecture).  Sequence lengths start at 0.  The current
 * CUDA device is the one the cache serves.  Host contents are zeroed.
 * Errors: INVALID_ARG (null out, non-positive size, dtype), UNSUPPORTED
 * (head_dim not 64 or 128), NO_MAPPED_MEMORY (device cannot map host
 * memory), ALLOC. */
dkv_status dkv_cache_alloc(dkv_cache** out, int batch, int n_kv_heads, int head_dim,
                           int max_tokens, dkv_dtype dtype);

/* The general allocator behind dkv_cache_alloc, dkv_cache_alloc_layered and
 * dkv_cache_alloc_paged, which also takes the element format.  An E4M3 cache
 * serves dkv_decode / dkv_decode_layer / dkv_decode_unfused / captured steps
 * (its host views hold uint8 E4M3 bits); dkv_prefill, dkv_decode_staged,
 * dkv_prefill_staged and dkv_attend_naive return UNSUPPORTED for it.  Errors: as the three
 * allocators, plus INVALID_ARG for an unknown format, UNSUPPORTED for E4M3
 * with fp16 activations, for E2M1 in a cache that is not paged or has pages of
 * fewer than 16 tokens, or for a paged cache of several layers. */
dkv_status dkv_cache_alloc_ex(dkv_cache** out, const dkv_cache_desc_t* desc);

/* A layered cache: one pinned allocation each for K and V holding `layers`
 * caches of [batch][n_kv_heads][max_tokens][head_dim] back to back, the
 * (layers, batch, heads, tokens, head_dim) host tensor of a whole model
 * ("DirectKV Guide: Zero-Copy KV Offloading on GH200 & GB200", Production
 * Engineering Playbook (1)).  Layers share the sequence lengths: a token's
 * calls go layer 0 .. layers-1 (dkv_decode_layer / dkv_prefill_layer), each
 * appending at the current length, and the lengths advance with the call for
 * the last layer.  dkv_decode / dkv_prefill refuse a layered cache
 * (INVALID_ARG); the measurement baselines need a one-layer cache.
 * Errors: as dkv_cache_alloc, plus INVALID_ARG for layers outside [1, 1024]. */
dkv_status dkv_cache_alloc_layered(dkv_cache** out, int layers, int batch, int n_kv_heads,
                                   int head_dim, int max_tokens, dkv_dtype dtype);

/* A paged cache: K and V pools of [num_pages][n_kv_heads][page_tokens][head_dim]
 * elements each in pinned, mapped host memory, addressed through a per-
 * sequence page table (the KV cache pages that the GPU kernels dereference in
 * place, "DirectKV Guide: Zero-Copy KV Offloading on GH200 & GB200", The
 * DirectKV Architecture (Zero-Copy Page Management) and End-to-End
 * Implementation (the page manager, 16-token pages)).  Logical row t of
 * sequence b lives in pool page table[b][t / page_tokens], row t % page_tokens.
 * Every decode / prefill call works on paged caches exactly as on dense ones;
 * a sequence holds at most max_pages_per_seq * page_tokens rows (its
 * max_tokens).  The page table starts empty (every entry -1).
 * Errors: as dkv_cache_alloc, plus INVALID_ARG when page_tokens is not a power
 * of two in [1, 4096] or num_pages / max_pages_per_seq is not positive. */
dkv_status dkv_cache_alloc_paged(dkv_cache** out, int batch, int n_kv_heads, int head_dim,
                                 int page_tokens, int num_pages, int max_pages_per_seq,
                                 dkv_dtype dtype);

/* Replace a paged cache's page table: table is host memory of
 * [batch][max_pages_per_seq] int32 pool page indices, -1 for none.  The
 * library keeps a host copy (each call checks that the rows it reads and
 * appends, [0, len + T) of every sequence, sit on pages: CAPACITY otherwise)
 * and a device copy, written after the cache's last stream has finished.
 * Pages may be shared between sequences for reading; the caller must not
 * let two sequences append into the same page row.
 * Errors: INVALID_ARG (dense cache, entry outside [-1, num_pages)), CUDA. */
dkv_status dkv_cache_set_page_table(dkv_cache* cache, const int32_t* table);

/* Release the pinned caches and the device workspace.  The caller must make
 * sure no enqueued work still uses the cache.  A handle already freed (or
 * never returned by dkv_cache_alloc) gives INVALID_ARG. */
dkv_status dkv_free(dkv_cache* cache);

/* The host NUMA node sysfs reports for a PCI device, given its bus id as
 * cudaDeviceGetPCIBusId prints it ("0000:1B:00.0"), read from
 * <sysfs_root>/bus/pci/devices/<id>/numa_node (sysfs_root null or "": /sys);
 * -1 when unknown, absent or malformed.  Every cache allocation pins its pages
 * with the calling thread's memory policy preferring the node of the current
 * GPU (so each replica's cache sits next to its own host link; "Paper Notes:
 * DirectKV", System Architecture, KV Cache Manager), then restores the policy;
 * DKV_NUMA=0 in the environment turns that off.  dkv_cache_info reports the
 * node wanted and the node the first page landed on. */
int dkv_pci_numa_node(const char* pci_bus_id, const char* sysfs_root);

/* Allocates and touches one page of ordinary host memory with the calling
 * thread's policy preferring `node`, as the cache allocation does, and
 * returns the node it landed on (-1 if unknown).  Needs no GPU. */
int dkv_numa_probe(int node);

/* Host addresses of the two caches ([B][Hkv][max_tokens][D] each), for
 * filling prefixes and reading back appended rows.  The host must not touch
 * rows that enqueued work reads or writes until that work has finished. */
dkv_status dkv_cache_host_ptrs(dkv_cache* cache, void** k_host, void** v_host);

/* Device aliases of the same two caches (zero-copy pointers). */
dkv_status dkv_cache_device_ptrs(dkv_cache* cache, void** k_dev, void** v_dev);

/* Set / read the per-sequence lengths (cached rows per sequence), len[B].
 * Set: INVALID_ARG if a length is negative, CAPACITY if above max_tokens. */
dkv_status dkv_cache_set_lengths(dkv_cache* cache, const int32_t* len);
dkv_status dkv_cache_get_lengths(const dkv_cache* cache, int32_t* len);

dkv_status dkv_cache_info(const dkv_cache* cache, dkv_cache_info_t* info);

/* Reserve the device workspace for calls with up to n_q_heads query heads and
 * up to max_new_tokens new tokens per sequence, so that later calls allocate
 * nothing.  Without it the first call of a larger shape grows the workspace
 * (a cudaMalloc on the calling thread, after synchronising the cache's last
 * stream). */
dkv_status dkv_cache_reserve(dkv_cache* cache, int n_q_heads, int max_new_tokens);

/* One decode step (T = 1) for every sequence: q = x.Wq, k = x.Wk, v = x.Wv
 * (fp32 accumulation in sequential order over H, rounded to the dtype), the
 * new k, v appended at row len[b] of the host cache, then softmax attention
 * of the Hq query heads over keys 0..len[b] of their KV head (the new token
 * included), written to out [B, 1, Hq, D].  Lengths advance by 1 when the
 * call is enqueued.  One cooperative launch of the fused kernel plus a
 * split-KV combine launch.  With an E4M3 cache the new k, v are the fp32
 * sums rounded once to E4M3 and the attention reads the decoded E4M3 rows.
 * Errors: INVALID_ARG (also for a layered cache: use dkv_decode_layer),
 * UNSUPPORTED (dtype, D, Hq/Hkv), CAPACITY, ALLOC (workspace growth), CUDA.
 * Device-side wait timeouts are reported by dkv_sync_status. */
dkv_status dkv_decode(dkv_cache* cache, const void* x, const void* wq, const void* wk,
                      const void* wv, int hidden, int n_q_heads, void* out, void* stream);

/* dkv_decode for one layer of a layered cache (layer 0 of any other cache):
 * x, W and out are that layer's; the append goes to the layer's cache at the
 * current length, and the lengths advance after the last layer.  Errors: as
 * dkv_decode, plus INVALID_ARG for a layer outside [0, layers). */
dkv_status dkv_decode_layer(dkv_cache* cache, int layer, const void* x, const void* wq,
                            const void* wk, const void* wv, int hidden, int n_q_heads, void* out,
                            void* stream);

/* Capture one whole decode step (every layer in order, then the lengths
 * advance by one) into a CUDA graph held by the cache, so that a step costs
 * one graph launch instead of two launches per layer.  x, wq, wk, wv, out are
 * host arrays of `layers` device pointers (as dkv_decode_layer takes them);
 * the graph keeps those pointers and the kernel configuration chosen now, and
 * reads the sequence lengths from device memory at run time, so every launch
 * appends at the lengths of its own step.  Captures on a stream of the
 * library's own; replaces an earlier capture.  A later call that needs a
 * larger workspace (a longer prefill, say) discards the capture, since the
 * graph holds workspace addresses; dkv_step_graph_launch then returns
 * INVALID_ARG until the step is captured again.  Errors: as dkv_decode, CUDA
 * (the capture or instantiation failed). */
dkv_status dkv_step_graph_capture(dkv_cache* cache, int hidden, int n_q_heads,
                                  const void* const* x, const void* const* wq,
                                  const void* const* wk, const void* const* wv,
                                  void* const* out);

/* Launch the captured step on `stream`: checks capacity (CAPACITY if a
 * sequence is full), publishes the host lengths to the device first if they
 * changed outside graph steps (one synchronisation), then launches and
 * advances the host lengths.  INVALID_ARG if nothing was captured. */
dkv_status dkv_step_graph_launch(dkv_cache* cache, void* stream);

/* One prefill (chunked-prefill) call: T new tokens per sequence at rows
 * [len[b], len[b]+T).  Query t of sequence b (absolute position len[b]+t)
 * attends causally to keys 0..len[b]+t.  Q = x.Wq is written to HBM first
 * (Q is HBM-resident, "Paper Notes: DirectKV", System Architecture, prefill
 * strategy); the fused kernel then holds each host K/V chunk stationary in
 * shared memory, computing the fresh K/V rows of chunks in the new region
 * in place and appending them to the host cache, and runs every query tile
 * of the KV head against it; a combine launch merges the per-chunk partial
 * results.  out is [B, T, Hq, D].  Lengths advance by T when enqueued.
 * Errors as dkv_decode, plus UNSUPPORTED for an E4M3 cache. */
dkv_status dkv_prefill(dkv_cache* cache, const void* x, int T, const void* wq, const void* wk,
                       const void* wv, int hidden, int n_q_heads, void* out, void* stream);

/* dkv_prefill for one layer of a layered cache (layer 0 of any other cache);
 * the lengths advance by T after the last layer. */
dkv_status dkv_prefill_layer(dkv_cache* cache, int layer, const void* x, int T, const void* wq,
                             const void* wk, const void* wv, int hidden, int n_q_heads, void* out,
                             void* stream);

/* Synchronise the stream, then return and clear the device status word that
 * bounded waits write (DKV_ERR_TIMEOUT), or DKV_ERR_CUDA if the stream
 * reported an error.  The word stays set until this call reads it: the
 * combine kernels of every decode or prefill enqueued while it is set write
 * NaN outputs instead of merging partials that were never written. */
dkv_status dkv_sync_status(dkv_cache* cache, void* stream);

/* Tuning overrides for ablations; 0 keeps the adaptor's choice.
 *   splits       decode: key-range splits per (sequence, KV head)
 *   tile_n       keys per host tile (decode) or per stationary chunk (prefill)
 *   stages       decode ring depth m */
dkv_status dkv_cache_set_tuning(dkv_cache* cache, int splits, int tile_n, int stages);

/* Test hook for the failure-detection path: while enabled, the producer
 * warps of every dkv_decode on this cache never signal their first host tile
 * (and the loader of every dkv_prefill never signals its chunk's host rows),
 * so a bounded wait expires after about one second; the kernel drains its own
 * copies and returns, and dkv_sync_status reports DKV_ERR_TIMEOUT.  The output
 * of such a call is NaN; the cache rows before the append are untouched and
 * the context stays usable. */
dkv_status dkv_cache_debug_withhold(dkv_cache* cache, int enable);

const char* dkv_status_str(dkv_status s);
const char* dkv_last_error(void);

/* Projection Y[M,N] = X[M,K] . W[K,N] on the tensor cores (the Q projection
 * step of dkv_prefill, q = x.Wq; "Paper Notes: DirectKV", Fundamental
 * Underlying Technologies, Kernel Fusion).  Row-major device tensors in
 * `dtype`, fp32 accumulation, one rounding to the dtype.  K must be a
 * multiple of 8 and N of 64; rows past M and columns past N are not
 * touched.  The caller owns all three buffers. */
dkv_status dkv_project(const void* x, const void* w, void* y, int M, int K, int N,
                       dkv_dtype dtype, void* stream);

/* ---- measurement kernels (internal baselines and link probes) ----------- */

/* Stream `bytes` (a multiple of 16) from `src` (a device pointer: a mapped
 * host alias for the link, HBM for the HBM rate) with 16-byte loads across
 * the whole GPU; the folded sum goes to sink[0] (device, 16 bytes) so the
 * loads cannot be elided.  The plain zero-copy streaming kernel whose rate is
 * the host-link denominator of the roofline. */
dkv_status dkv_probe_read(const void* src, size_t bytes, void* sink, void* stream);

/* Write `bytes` (a multiple of 16) of a pattern to `dst` with 16-byte stores. */
dkv_status dkv_probe_write(void* dst, size_t bytes, void* stream);

/* Launch floor: an empty kernel (it reads and writes nothing) launched
 * cooperatively with `grid` CTAs of `threads` threads (a multiple of 32, at
 * most 1024) and `smem_bytes` of dynamic shared memory (at most 227 KB).
 * Timed with CUDA events around it, it gives what launch and completion add
 * to a kernel's measured time.  INVALID_ARG for another shape; a grid that
 * cannot be co-resident is reported as a CUDA error. */
dkv_status dkv_probe_launch(int grid, int threads, int smem_bytes, void* stream);

/* Naive untiled zero-copy decode attention (the pages' "naive zero-copy"
 * baseline, "Paper Notes: DirectKV", Experiments, CPU-aware tiling): one CTA
 * per (sequence, query head, split) reads its KV head's rows straight from
 * the host cache with no shared-memory tile and no reuse across the heads of
 * a group.  It attends q (HBM, [B, Hq, D], the dtype) over keys 0..len[b]-1
 * of the cache as it stands (no projection, no append) into out [B, Hq, D].
 * Dense caches only (UNSUPPORTED for a paged cache). */
dkv_status dkv_attend_naive(dkv_cache* cache, const void* q, int n_q_heads, void* out,
                            void* stream);

/* Separate-kernel baseline (the unfused design the pages compare against,
 * "Paper Notes: DirectKV", Experiments & Results, Fused kernel (Fig. 13), and
 * Key Ideas (2)): the same
 * decode as dkv_decode split into two launches, a projection that writes q to
 * HBM and appends the fresh K/V rows to the host cache, then an attention
 * launch that reads every row, the appended one included, back across the
 * link.  Same arguments, results and errors as dkv_decode. */
dkv_status dkv_decode_unfused(dkv_cache* cache, const void* x, const void* wq, const void* wk,
                              const void* wv, int hidden, int n_q_heads, void* out,
                              void* stream);

/* Copy-to-HBM-then-attend baseline (swap-style staging, "Paper Notes:
 * DirectKV", Motivation): cudaMemcpyAsync the cached rows [0, len[b]) of
 * every (sequence, KV head) into the caller's HBM buffers k_stage, v_stage
 * (each [B][Hkv][max_tokens][D]) and run the same fused decode as dkv_decode
 * reading the prefix from HBM (the append still goes to the host cache).
 * Dense caches only (UNSUPPORTED for a paged cache). */
dkv_status dkv_decode_staged(dkv_cache* cache, const void* x, const void* wq, const void* wk,
                             const void* wv, int hidden, int n_q_heads, void* out,
                             void* k_stage, void* v_stage, void* stream);

/* The same baseline for prefill: cudaMemcpyAsync the cached rows [0, len[b])
 * of every (sequence, KV head) into the caller's HBM buffers k_stage,
 * v_stage (each [B][Hkv][max_tokens][D], device memory the caller owns), then
 * run the same fused prefill as dkv_prefill reading the cached prefix from
 * HBM; the T new rows are still appended to the host cache and the lengths
 * advance by T.  Same arguments, results and errors as dkv_prefill, plus
 * INVALID_ARG for a null staging buffer and UNSUPPORTED for a paged, layered
 * or E4M3 cache. */
dkv_status dkv_prefill_staged(dkv_cache* cache, const void* x, int T, const void* wq,
                              const void* wk, const void* wv, int hidden, int n_q_heads,
                              void* out, void* k_stage, void* v_stage, void* stream);

/* Naive untiled zero-copy prefill (measurement baseline for the pages'
 * CPU-memory-aware tiling, "Paper Notes: DirectKV", Key Ideas (1) and
 * Experiments & Results, Fig. 12).  Same computation, results and append
 * as dkv_prefill, from the same fused kernel, but every (Q tile, chunk)
 * pair gets its own CTA, in the order a Q-stationary kernel streams the
 * chunks, so each chunk of cached rows crosses the host link once per Q tile
 * that sees it instead of once.  The outputs are bit-identical to
 * dkv_prefill's.  Errors as dkv_prefill, plus UNSUPPORTED for a layered or
 * E4M3 cache. */
dkv_status dkv_prefill_naive(dkv_cache* cache, const void* x, int T, const void* wq,
                             const void* wk, const void* wv, int hidden, int n_q_heads,
                             void* out, void* stream);

/* Kernel timing for measurement: when enabled, each dkv_decode / dkv_prefill
 * records a pair of CUDA events on its stream around its main fused kernel
 * (not the projection or combine launches).  dkv_cache_last_kernel_ms waits
 * for the last recorded pair and returns its elapsed time in milliseconds;
 * INVALID_ARG if timing is off or nothing was recorded yet. */
dkv_status dkv_cache_kernel_timing(dkv_cache* cache, int enable);
dkv_status dkv_cache_last_kernel_ms(dkv_cache* cache, float* ms);

/* ---- decode without any allocation -------------------------------------- */

/* The paper has no counterpart to this call; it exists for callers that may
 * not allocate GPU memory at all (code running inside an allocator or
 * memory-pool callback, plug-ins whose host runtime owns every device
 * allocation, services that must hold a fixed memory budget after start-up).
 *
 * Same computation as dkv_decode on caller-owned buffers: q/k/v projection of
 * x, append of the new k, v at row lengths[b] of k_cache / v_cache, attention
 * over rows 0..lengths[b], result in out [B, 1, Hq, D].  k_cache and v_cache
 * are device-accessible pointers to [batch][n_kv_heads][max_tokens][head_dim]
 * caches (normally the mapped aliases of pinned host memory, e.g. from
 * dkv_cache_device_ptrs); lengths is a host array [batch] that this call
 * reads but does not advance.  All tensors are in `dtype`.
 *
 * It calls no cudaMalloc, cudaFree or allocating library routine.  Its
 * scratch (8 MiB: q and fresh K/V workspace, split-KV partials, status word)
 * is a fixed __device__ array that every GPU loading the library holds until
 * the process exits; a shape whose scratch would exceed 8 MiB even with one
 * key-range split is rejected with DKV_ERR_CAPACITY.  Every call on a device
 * shares that array, so calls whose work overlaps on the GPU (other streams,
 * other threads) race and must be serialised by the caller.  The first call
 * on each device looks up the array's device address (cudaGetSymbolAddress)
 * with that device current; make that first call before any stream capture.
 * The address is looked up again on every call (the lookup allocates
 * nothing), so a context that was reset and recreated is served correctly.
 * A device-side wait that gives up (DKV_ERR_TIMEOUT) is recorded in the
 * scratch status word, which every call clears first, and makes the call's
 * outputs NaN; dkv_decode_noalloc_status reads it.
 * Errors: INVALID_ARG, UNSUPPORTED, CAPACITY, CUDA, before anything is
 * enqueued. */
dkv_status dkv_decode_noalloc(const void* x, const void* wq, const void* wk, const void* wv,
                              void* k_cache, void* v_cache, const int32_t* lengths, int batch,
                              int hidden, int n_q_heads, int n_kv_heads, int head_dim,
                              int max_tokens, dkv_dtype dtype, void* out, void* stream);

/* Status of the last dkv_decode_noalloc on the current device, without any
 * allocation: synchronises `stream`, copies the scratch status word into a
 * host variable, clears it if set, and returns DKV_OK or the recorded error
 * (DKV_ERR_TIMEOUT); DKV_ERR_CUDA if the stream reported an error.  Call it
 * after the dkv_decode_noalloc it should report on and before the next one
 * (which clears the word). */
dkv_status dkv_decode_noalloc_status(void* stream);

/* Test hook for the no-allocation path (process-wide): while enabled, the
 * producers of every dkv_decode_noalloc withhold their first tile's signal so
 * that the consumers' bounded wait expires after about a second; the call's
 * outputs are NaN and dkv_decode_noalloc_status reports DKV_ERR_TIMEOUT. */
dkv_status dkv_decode_noalloc_debug_withhold(int enable);

/* ---- the device-side step over a 4-bit paged cache ------------------------ */

/* A decoder that normalises and rotates its queries and keys cannot use the
 * fused projection of dkv_decode / dkv_prefill.  These three calls serve it on
 * caller-owned buffers, with lengths, page tables and slots that live on the
 * device, so that a whole step (plan, append, attend for each layer) can be captured
 * in a CUDA graph and replayed without the host knowing a length:
 *
 *   dkv_step_plan      lengths and new-token counts -> pages, row starts,
 *                      positions and slots
 *   dkv_qkv_append     head norms and rotation of q and k; k and v into the
 *                      slots of an E2M1 pool
 *   dkv_paged_attend   softmax attention of ragged query rows over the pool
 *
 * A step has `rows` token rows: sequence b's new tokens are rows row_start[b] ..
 * row_start[b+1]-1, and rows behind the last sequence are padding (slot -1):
 * nothing of them is written.  Pools are device-accessible pointers: HBM, or
 * the mapped alias of pinned host memory (dkv_cache_device_ptrs of a
 * DKV_KV_E2M1 cache), which is then read across the host link (see dkv_paged_attend for
 * how often).
 * Nothing here allocates, synchronises or keeps state between calls; errors
 * return before anything is enqueued.  Calls that may overlap on the GPU need
 * outputs and workspaces of their own. */

#define DKV_MAX_STEP_BATCH 1024 /* sequences of a step */

/* Plan one step on the GPU.  All pointers are device memory of int32.
 *   lengths    [batch]  cached rows per sequence
 *   new_tokens [batch]  rows the step adds (0: none); below 0: the sequence has
 *                       ended, its pages go back and its length becomes 0
 *   page_table [batch][max_pages]  pool pages of each sequence's rows; the
 *                       entries of newly taken pages are written (entries past a
 *                       sequence's length are never read)
 *   free_pages [num_pages]  stack of unused pages, free_count[0] of them valid.
 *                       Pages released are pushed in order of sequence and
 *                       page; the k-th page taken, in that order too, is the k-th
 *                       from the top.
 * Written: row_start [batch + 1]; row_pos, row_slot [max_rows] (position and slot
 * = page * page_tokens + offset of each row, a slot of -1 where the table or the stack holds a page
 * outside [0, num_pages); 0 and -1 behind the last);
 * kv_len [batch], the lengths with the new rows; free_left [1]; report [4] =
 * {status, rows, pages taken, longest kv_len}.
 * All or nothing: where the pages, the rows (max_rows) or a sequence's table
 * (max_pages) do not suffice, report[0] is DKV_ERR_CAPACITY, every row is padding,
 * kv_len = lengths, free_left = free_count, and table and stack stay as they were.
 * kv_len may be `lengths` and free_left may be `free_count` (update in place); other
 * buffers must not overlap.
 * Errors: INVALID_ARG (null pointer; batch outside [1, DKV_MAX_STEP_BATCH];
 * page_tokens not a power of two in [1, 4096]; max_pages, num_pages or max_rows not
 * positive, or above 2^30 rows), CUDA. */
dkv_status dkv_step_plan(const int32_t* lengths, const int32_t* new_tokens, int32_t* page_table,
                         int32_t* free_pages, const int32_t* free_count, int batch, int max_pages,
                         int page_tokens, int num_pages, int max_rows, int32_t* row_start,
                         int32_t* row_pos, int32_t* row_slot, int32_t* kv_len, int32_t* free_left,
                         int32_t* report, void* stream);

/* Norm, rotation and append of one step's projected rows.
 *   q [rows][n_q_heads][head_dim], k and v [rows][n_kv_heads][head_dim], `dtype`;
 *     consecutive rows lie *_stride elements apart (one projection's output
 *     holds all three), heads of a row are contiguous.  q may be null (keys and
 *     values only), or k and v (queries only).
 *   q_gamma, k_gamma [head_dim], `dtype`, or null: RMS norm of each head's row,
 *     x / sqrt(mean x^2 + eps) * gamma.  Values are never normalised.
 *   cos_sin [max_positions][rotary_dim] fp32, or null: rotary_dim/2 cosines, then
 *     rotary_dim/2 sines of each position; positions [rows] int32.  Pairs are
 *     (i, i + rotary_dim/2), or (2i, 2i + 1) with `interleaved`; elements from
 *     rotary_dim on are not rotated.  A position outside the table makes the
 *     row's q and k NaN.
 *   slots [rows] int32: where the row's k and v go in the pools (page * page_tokens
 *     + offset).  A slot outside [0, num_pages * page_tokens) marks padding:
 *     nothing of the row is written, q_out included.  Two rows of a call must not
 *     have the same slot.  Null slots and pools: no append, k_out and v_out
 *     take the rows rounded to `dtype`.
 *   k_scale, v_scale: the pools hold k / k_scale and v / v_scale.
 *   q_out [rows][n_q_heads][head_dim] (may be q if q is contiguous); k_out, v_out
 *     [rows][n_kv_heads][head_dim] or null: with pools, the values that the cache
 *     now holds (times the scale, rounded to `dtype`).
 * Arithmetic is fp32, each operation rounded once, the key norm's sum of squares in
 * two words.  A block of 16 takes the scale e4m3(max|y| / 6), saturating at 448, and
 * the codes e2m1(y / scale), both to nearest even, saturating; a block with a NaN
 * or an infinity gets a NaN scale and reads back as NaN.  Where max|y| is below 0.0059 the block's
 * scale, and so the block, is 0, and below 0.094 the scale is subnormal, with one to three bits: a
 * k_scale or v_scale below 1 brings the rows of a model with such small keys or values (V as
 * a rule) into range.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim not 64 or 128), CUDA. */
typedef struct {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const void *q_gamma, *k_gamma;
    const float* cos_sin;
    const int32_t *positions, *slots;
    void *k_pool, *v_pool;
    void *q_out, *k_out, *v_out;
    int rows, n_q_heads, n_kv_heads, head_dim;
    dkv_dtype dtype;
    int rotary_dim, max_positions, interleaved;
    int page_tokens, num_pages;
    float eps, k_scale, v_scale;
} dkv_append_t;
dkv_status dkv_qkv_append(const dkv_append_t* args, void* stream);

/* Attention of a step's query rows over an E2M1 pool: row i of sequence b (n_b =
 * row_start[b+1] - row_start[b] rows) attends to keys 0 .. kv_len[b] - n_b + i of its
 * sequence, through page_table [batch][max_pages]:
 *   o = v_scale * softmax(scale * q . k) . v
 * A null row_start means one row per sequence (a decode step).  kv_len counts the
 * rows' own keys, appended before.  A row that sees no key is zero with lse -infinity.
 * out [rows][n_q_heads][head_dim] in `dtype`; lse [rows][n_q_heads] fp32, or null:
 * the natural log of the sum of exp(scale * q . k).  Rows of no sequence are left as
 * they were.
 * max_rows: no sequence has more rows than this; it chooses the kernel, any lengths
 * on the device are then served.  It does so for the whole call: up to 32 packed rows
 * (max_rows * heads per KV head) a kernel for few rows, above that one for many, in which
 * a single token costs about three times as much (64 of them at 32768 keys beside a chunk of
 * 2048 rows: 2.4 ms, as two calls 1.3).  The few-row kernel reads a sequence's keys once
 * for all its packed rows, the many-row kernel once for each 256 of them: a pool in host
 * memory crosses the link that often (4096 rows with 4 heads per KV head: 64 times), so
 * chunks want their pages in HBM.
 * Lengths above max_pages * page_tokens are cut to that; a page index outside
 * [0, num_pages) counts as a page without keys.  K's scale (dkv_append_t.k_scale) belongs
 * into `scale`.
 * A NaN in a key or value reaches the rows that see it and no others.
 * q, k.v products run on fp16 tensor operands (cache values and fp16 queries exactly;
 * bf16 queries scaled by a power of two per row, where an element below 2^-27 of its row's
 * largest may lose bits; weights rounded to fp16, which costs 2^-11 of a weight, or 2^-32 of
 * the row's largest where a weight is below 2^-21 of it), sums and softmax statistics in
 * fp32 (one head over 2^24 keys: 2^-10 and less).  |scale * q . k| up to 2^21 is served; where it
 * is larger a row may become NaN.  The result does not depend on timing.
 * workspace: device memory of dkv_paged_attend_workspace bytes (0 for arguments
 * that dkv_paged_attend refuses), on a 256-byte boundary; its contents do not matter
 * before and after a call.
 * The kernel for more than 32 rows times heads per KV head waits on the device for its own
 * copies and products, for a second at most; where a wait gives up, the affected rows of out and
 * lse are NaN.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim not 64 or 128), CUDA. */
typedef struct {
    const void* q;
    long long q_stride;
    const void *k_pool, *v_pool;
    const int32_t *page_table, *kv_len, *row_start;
    void* out;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int batch, rows, max_rows, n_q_heads, n_kv_heads, head_dim;
    dkv_dtype dtype;
    int page_tokens, num_pages, max_pages;
    float scale, v_scale;
} dkv_attend_t;
dkv_status dkv_paged_attend(const dkv_attend_t* args, void* stream);
size_t dkv_paged_attend_workspace(int batch, int n_q_heads, int n_kv_heads, int head_dim,
                                  int max_rows);

/* 1: the stream is being captured into a graph, which then owns what its launches use; 0: it is
 * not; -1: the stream cannot say. */
int dkv_stream_capturing(void* stream);

/* Test hook (process-wide, off by default): with enable != 0 the many-row kernel of the calls that follow never
 * signals an item's outputs, so that its waits run out (some seconds). */
dkv_status dkv_paged_attend_debug_withhold(int enable);

/* ---- the same step over an 8-bit paged cache with block scales ------------------ */

/* A pool of E4M3 codes [num_pages][n_kv_heads][page_tokens][head_dim] (one byte an element, the layout of a
 * paged DKV_KV_E4M3 cache) with fp32 scales [num_pages][n_kv_heads][page_tokens / 16]: an element is its
 * code times the scale of its block, 16 consecutive tokens of a page and head.  Pages hold 16 to 4096 tokens.
 * Four significant bits where E2M1 has two, for less than twice the bytes; dkv_step_plan plans it, dkv_pages_* share and move
 * its pages (codes and scales are pools of one table).  Pools may be HBM or the mapped alias of pinned host
 * memory, scales too. */

/* Norm, rotation and append of one step's projected rows: dkv_append_t's arguments and arithmetic, keys and values
 * into blocks.  k, v, both pools, their scales and slots are needed; q may be null.
 * For the rows y of a call in one block: need = the smallest power of two with max|y| <= 448 need (2^-64 at least),
 * s = max(need, scale so far), where a block whose first token is among the rows (slot a multiple of 16) has no scale
 * so far, and one whose scale is not a positive finite number neither.  The block's scale becomes s; if it grew, codes that are
 * there become e4m3(code * old / s); the rows' codes are e4m3(y / s), to nearest even.  A NaN or an infinity becomes a
 * NaN of its element alone, and does not count for the scale.
 * The rows of one block must lie within 16 consecutive rows of the call (dkv_step_plan deals them one after another), and no
 * two may have one slot;
 * sequences that append to the same block must not share it (dkv_pages_fork sees to that, after a cut too).  A
 * sequence that is cut back and appended to again keeps its block's scale, which is then larger than it has to be, until
 * the block begins anew.
 * k_out, v_out [rows][n_kv_heads][head_dim] or null: the values that the cache now holds, rounded to `dtype` (an
 * infinity where E4M3 has rounded the type's largest numbers up beyond it).
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim not 64 or 128), CUDA. */
typedef struct {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    const void *q_gamma, *k_gamma;
    const float* cos_sin;
    const int32_t *positions, *slots;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    void *q_out, *k_out, *v_out;
    int rows, n_q_heads, n_kv_heads, head_dim;
    dkv_dtype dtype;
    int rotary_dim, max_positions, interleaved;
    int page_tokens, num_pages;
    float eps;
} dkv_block_append_t;
dkv_status dkv_block_append(const dkv_block_append_t* args, void* stream);

/* dkv_paged_attend over such a pool, with its arguments, kernels and limits (v_scale aside, which the blocks' scales
 * take the place of):
 *   o = softmax(scale * q . k) . v,  k and v the codes times their blocks' scales.
 * Scales of blocks that a row sees are K's from 2^-126 to 2^126, V's from 2^-64 (dkv_block_append writes none below; the sum
 * of the weights, in fp32, counts their inverses) to 2^126, and those of V that one row sees within 2^80 of one another.
 * |scale * q . k| up to 2^21 is served; scores of a row whose largest |scale * q| is below 2^-113 lose bits.
 * A weight is rounded to fp16, by 2^-11 of it, or by
 * 2^-32 of the row's largest where it is below 2^-21 of that.  Up to 32 packed rows (max_rows times heads per KV head), and
 * above in tiles with a scale that is not a power of two from 2^-15 to 2^7 times its piece's first, weights count times
 * their V scale there.
 * workspace: dkv_paged_attend_workspace bytes.  Errors: as dkv_paged_attend. */
typedef struct {
    const void* q;
    long long q_stride;
    const void *k_pool, *v_pool;
    const float *k_scales, *v_scales;
    const int32_t *page_table, *kv_len, *row_start;
    void* out;
    float* lse;
    void* workspace;
    size_t workspace_bytes;
    int batch, rows, max_rows, n_q_heads, n_kv_heads, head_dim;
    dkv_dtype dtype;
    int page_tokens, num_pages, max_pages;
    float scale;
} dkv_block_attend_t;
dkv_status dkv_block_attend(const dkv_block_attend_t* args, void* stream);

/* ---- the life of a cache's pages ------------------------------------------- */

/* Sequences share, move and give back pages on the GPU.  A pool's pages have no counters: the page
 * table says who holds what (the ceil(kv_len / page_tokens) first entries of a sequence's row), and a page that no
 * sequence holds is free.  Several rows may name one page; dkv_step_plan appends to a sequence's last,
 * partly filled page only, which dkv_pages_fork leaves to one row alone.  A sequence that is cut back (a smaller
 * kv_len) into a page that others hold goes through dkv_pages_fork, itself as its source, before anything is appended to
 * it: the fork sees the shorter length and gives it a copy.  The pages behind its new end are on no stack until
 * dkv_pages_compact.  A sequence that may share pages ends by
 * dkv_pages_fork (source -1): dkv_step_plan's release would put a shared page on the stack while others
 * hold it.  A table that serves several pools (layers; keys, values and their scales) takes one fork or
 * compaction and one dkv_pages_copy over all of them:
 *
 *   dkv_pages_fork     sequences go on as copies of others, or end
 *   dkv_pages_compact  the pages held move to the front of the pool
 *   dkv_pages_copy     the bytes that the two (or the caller) want moved
 *
 * workspace: device memory of dkv_pages_workspace bytes (0 for sizes that the calls refuse) on a 256-byte
 * boundary, for fork and compact; its contents do not matter before and after a call.  Nothing
 * allocates, synchronises or keeps state; all of it can be captured.  Calls that may overlap on the GPU need
 * outputs and workspaces of their own. */
size_t dkv_pages_workspace(int batch, int max_pages, int num_pages);

/* New sequence b becomes old sequence sources[b]: its length, and its pages.  Below 0: b ends (or stays
 * empty).  All int32 device memory.
 *   page_table [batch][max_pages], kv_len [batch]  before the call
 *   sources    [batch]  0 .. batch - 1, or below 0
 *   free_pages [num_pages], free_count [1]  the stack of dkv_step_plan
 * Full pages are shared.  Of the rows that go on with the same last page, filled in part, one keeps it (the lowest with
 * sources[b] = b, else the lowest), and none where a row that goes on has it as a full page (the others were cut back);
 * every other one takes a page from
 * the stack, in order of b, the k-th from the top, and has copies[b] = {the source's page, its own}.  Pages that were
 * held before and are not any more are pushed first, in ascending order.
 * Written: table_out [batch][max_pages] (the entries of pages held; others are left as they were), len_out [batch],
 * free_left [1], copies [batch][2] ({-1, -1}: nothing to copy), report [4] = {status, pages released, pages
 * taken, longest len_out}.
 * All or nothing: where the stack does not hold enough (or would hold more than num_pages), or a length is above
 * max_pages * page_tokens, report[0] is DKV_ERR_CAPACITY, and with a source of batch or more
 * DKV_ERR_INVALID_ARG; nothing is copied, and table_out, len_out (0 for a length below 0) and free_left are what came in.
 * A page index outside [0, num_pages) is handed on and never released.  Lengths below 0 count as 0.
 * table_out may be page_table, len_out kv_len and free_left free_count (in place); other buffers
 * must not overlap.  Errors: INVALID_ARG, CUDA. */
dkv_status dkv_pages_fork(const int32_t* page_table, const int32_t* kv_len, const int32_t* sources,
                          int32_t* free_pages, const int32_t* free_count, int batch, int max_pages,
                          int page_tokens, int num_pages, int32_t* table_out, int32_t* len_out,
                          int32_t* free_left, int32_t* copies, int32_t* report, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The pages that any sequence holds, `live` of them, move to pages 0 .. live - 1: the i-th of them from page
 * `live` on, in ascending order, goes to the i-th page below `live` that nobody holds.  Pages held by
 * something other than a row of the table count as free.
 * Written: table_out [batch][max_pages] (entries of pages held), moves [max_moves][2] = {from, to} in that order, {-1, -1} behind the
 * last (max_moves is num_pages / 2 at least, moves may be null where num_pages is 1), free_pages [num_pages]:
 * num_pages - 1 down to live, so that the lowest page is taken first, the rest left as it was; free_left [1]; report [4] = {status,
 * pages moved, live, longest kv_len}.  A page index outside [0, num_pages) is left as it is.
 * With a length above max_pages * page_tokens report[0] is DKV_ERR_CAPACITY, nothing moves, table_out is
 * page_table, and free_pages and free_left are not written.
 * The bytes move by dkv_pages_copy(moves), of every pool behind the table; until then the new table
 * must not be used.  table_out may be page_table; other buffers must not overlap.  Errors: INVALID_ARG, CUDA. */
dkv_status dkv_pages_compact(const int32_t* page_table, const int32_t* kv_len, int batch, int max_pages,
                             int page_tokens, int num_pages, int32_t* table_out, int32_t* free_pages,
                             int32_t* free_left, int32_t* moves, int max_moves, int32_t* report,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Page `to` of each pool's dst takes the bytes of page `from` of its src, for every {from, to} of pairs
 * [n_pairs][2] (device memory; n_pairs may be 0).  A pair with an index outside the pool is skipped.  src and dst may be one
 * pool, or two of different sizes, in HBM or in pinned host memory (pages leave for the host, or come back).
 * No page may be `to` of two pairs, nor `to` of one and `from` of another in the same pool.
 * pools is host memory; up to 64 pools of one alignment go in one launch.
 * Errors: INVALID_ARG (page_bytes not a multiple of 4 or above 2^30, a pool not on a 4-byte boundary), CUDA. */
typedef struct {
    const void* src;
    void* dst;
    size_t page_bytes;
    int src_pages, dst_pages;
} dkv_page_pool_t;
dkv_status dkv_pages_copy(const int32_t* pairs, int n_pairs, const dkv_page_pool_t* pools, int n_pools,
                          void* stream);

/* Number of kernel launches the last dkv_decode / dkv_prefill enqueued. */
int dkv_last_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* DKV_H */
