/*
 * oscar.h - C ABI of the GB300 (sm_103a) OSCAR INT2 rotated paged KV cache.
 *
 * OSCAR ("Offline Spectral Covariance-Aware Rotation for 2-bit KV Cache
 * Quantization", arXiv 2605.17757) keeps a paged KV cache in which the first
 * ("sink") and the most recent tokens stay BF16 and the middle history is
 * stored as INT2 after a fixed per-layer rotation R = U . H_Had . P_br and
 * clipping (gist.science technical summary, section 2.2 B; arXiv abstract).
 * This library is the serving hot path: the write into pages, the append that
 * evicts the oldest recent token into INT2, and the fused decode attention
 * over the mixed cache.  Calibration (computing R and the clip thresholds,
 * section 2.2 A) is offline and not part of this library.
 *
 * Conventions
 *  - Every call returns oscar_status (0 = OK).  oscar_last_error() gives a
 *    thread-local message for the last failing call on this thread.
 *  - Tensor arguments are DEVICE pointers owned by the caller unless stated
 *    otherwise.  The library keeps no pointer beyond the call, except the two
 *    pools registered at oscar_create.
 *  - Work is enqueued asynchronously on the caller's stream (cudaStream_t
 *    passed as void*; NULL = legacy default stream).  Argument errors are
 *    reported synchronously.  Device-side errors (a page id out of range, a
 *    bounded wait that timed out) set a status word read by
 *    oscar_check_status().
 *  - Row-vector convention: a rotated vector is y = x R, R is d x d float32
 *    row-major (R[i*d + j]), 16-byte aligned (OSCAR_ERR_INVALID otherwise).
 *    Every R_K / R_V argument holds one such matrix per layer call, or, when
 *    the configuration's rotation_per_kv_head is 1, n_kv_heads of them back to
 *    back ([n_kv_heads][d][d], kv head h at R + h*d*d).
 *  - bf16 tensors are uint16 bit patterns of bfloat16.
 *
 * Memory layout (all little-endian)
 *  INT2 page pool: [num_layers][num_pages][n_kv_heads][block], where one
 *  (layer, page, kv head) block of P = page_size tokens is
 *      K codes  [P][d/4] bytes | K (scale, zero) [P][d/32][2] bf16 |
 *      V codes  [P][d/4] bytes | V (scale, zero) [P][d/32][2] bf16
 *  (d = 128, P = 64: 6144 bytes).  History token t of a request lives in page
 *  block_table[b][t / P], slot t % P (absolute-position paging).
 *  K code row (d/4 bytes = d/16 32-bit words): for lane tig in 0..3,
 *  w in [0, d/64), slot x in 0..7, let P8 = 8w + x, g = P8>>2, kt = (P8>>1)&1,
 *  h = P8&1, c = 32g + 16kt + 8h + 2*tig; word tig*(d/64)+w holds channel c
 *  at bits 2x and channel c+1 at bits 16+2x.
 *  V code row (d/8 16-bit half-words): half-word hw, slot s in 0..7 at bits
 *  2s holds channel 64*(hw % (d/64)) + 8s + hw / (d/64).
 *  Quantiser (per token, kv head, group of 32 rotated channels): y clipped to
 *  [-clip, clip]; zero = bf16(min); scale = bf16((max-min)/3);
 *  code = clamp(rne((y - zero)/scale), 0, 3) (all zero if scale == 0);
 *  dequantised value zero + code*scale.
 *
 *  BF16 window slab: [num_layers][max_requests][n_kv_heads][2 (K,V)][S+W][d]
 *  bf16, unrotated.  Sink token t (< S) is at slot t; recent token t is at slot
 *  S + (t - S) mod W.  Token t of a sequence of length n is sink if t < S,
 *  recent if t >= max(S, n - W), history (INT2) otherwise.
 *
 *  BF16 paged pool (comparison kernel only): [num_layers][num_pages]
 *  [n_kv_heads][2 (K,V)][P][d] bf16, token t at block_table[b][t/P], slot t%P.
 */
#ifndef OSCAR_H_
#define OSCAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t oscar_status;
enum {
  OSCAR_OK = 0,
  OSCAR_ERR_INVALID = -1,     /* bad argument (null pointer, size, sink/recent mismatch) */
  OSCAR_ERR_OOM = -2,         /* page allocator exhausted */
  OSCAR_ERR_CUDA = -3,        /* a CUDA runtime call failed (message in oscar_last_error) */
  OSCAR_ERR_DEVICE = -4,      /* device status word set (bad page id, wait timeout) */
  OSCAR_ERR_UNSUPPORTED = -5  /* shape outside the supported set */
};

enum { OSCAR_DTYPE_F32 = 0, OSCAR_DTYPE_BF16 = 1 };

/* Device status bits reported by oscar_check_status (oscar_device_status). */
enum {
  OSCAR_DEV_BAD_PAGE = 1,     /* block table entry out of [0, num_pages) on a needed page */
  OSCAR_DEV_TIMEOUT = 2,      /* a bounded barrier wait gave up */
  OSCAR_DEV_BAD_LEN = 4,      /* seq_len / start_pos outside [0, max_pages*page_size] */
  OSCAR_DEV_BAD_SLOT = 8,     /* req_slot outside [0, max_requests) */
  OSCAR_DEV_BAD_VALUE = 16    /* an infinity or NaN among the K or V values of a quantised 8-bit page */
};

typedef struct {
  int32_t num_layers;
  int32_t n_q_heads;
  int32_t n_kv_heads;
  int32_t head_dim;          /* 64 or 128 */
  int32_t page_size;         /* 16, 32 or 64 */
  int32_t group_size;        /* 32 */
  int32_t sink;              /* S >= 0 */
  int32_t recent;            /* W >= 1 */
  int32_t max_requests;      /* window-slab slots */
  int32_t max_pages_per_req; /* block-table row capacity used for bounds checks */
  int32_t num_pages;         /* INT2 pages per layer */
  int32_t rotation_per_kv_head; /* 0: one R_K and one R_V per layer, shared by every kv head (the
                                   pages' fixed per-layer rotation): R_K, R_V are [d][d].  1: one
                                   rotation per (layer, kv head): R_K, R_V are [n_kv_heads][d][d],
                                   kv head h rotated by R[h] (a variant of ours; the clip thresholds
                                   stay per layer) */
} oscar_config;

typedef struct oscar_ctx oscar_ctx;

/* Thread-local message of the last failing call ("" if none). */
const char* oscar_last_error(void);

/* Library version string. */
const char* oscar_version(void);

/* Bytes of the INT2 page pool / BF16 window slab / one (page, kv head) block
 * for a configuration; 0 if the configuration is invalid. */
size_t oscar_int2_pool_bytes(const oscar_config* cfg);
size_t oscar_window_slab_bytes(const oscar_config* cfg);
size_t oscar_page_block_bytes(const oscar_config* cfg);

/* Validate cfg and create a context over caller-owned device buffers:
 * int2_pool (oscar_int2_pool_bytes) and window_slab (oscar_window_slab_bytes),
 * both 16-byte aligned (else OSCAR_ERR_INVALID).
 * The context keeps the raw pointers: both buffers must stay allocated until
 * oscar_destroy (and until any captured graph that uses them is destroyed).
 * Either pointer may be NULL for a host-only context (allocator calls work,
 * kernel calls return OSCAR_ERR_INVALID).  Creating a context with buffers
 * allocates a 4-byte device status word and max_requests x n_kv_heads int32
 * counters of the one-launch decode (zero between launches).  OSCAR_ERR_UNSUPPORTED for a shape
 * outside head_dim {64,128}, page_size {16,32,64}, group_size 32,
 * n_q_heads/n_kv_heads in {1,2,4,8}. */
oscar_status oscar_create(const oscar_config* cfg, void* int2_pool, void* window_slab, oscar_ctx** out);
oscar_status oscar_destroy(oscar_ctx* ctx);

/* ---------------------------------------------------------------- host page allocator
 * Source: the OSCAR serving path keeps the INT2 history in a paged cache that is
 * compatible with paged attention and prefix caching (gist.science technical
 * summary, section 2.2 B and section 3; arXiv abstract: fused kernels inside the
 * paged serving engines).  These calls are the page side of that cache: a page
 * is the unit a block table maps, and a refcount lets requests that share a
 * prefix share its pages.
 * Pages are shared by every layer (page id p addresses block p of each layer).
 * A freshly allocated page has refcount 1; a page returns to the free list
 * when its refcount drops to 0.  ids are host arrays.  Host-only: no device
 * work, no stream.  oscar_alloc_pages returns OSCAR_ERR_OOM (and allocates
 * nothing) when fewer than n pages are free; ref/unref of an id outside
 * [0, num_pages) or of a free page returns OSCAR_ERR_INVALID. */
oscar_status oscar_alloc_pages(oscar_ctx* ctx, int32_t n, int32_t* out_ids);
oscar_status oscar_ref_pages(oscar_ctx* ctx, const int32_t* ids, int32_t n);
oscar_status oscar_unref_pages(oscar_ctx* ctx, const int32_t* ids, int32_t n);
oscar_status oscar_page_refcount(oscar_ctx* ctx, int32_t id, int32_t* out_refcount);
oscar_status oscar_free_page_count(oscar_ctx* ctx, int32_t* out_n);

/* Copy the INT2 blocks of n pages of one layer to host memory (a test and
 * debugging aid; the cache itself is transient serving state).  host_dst
 * receives n x [n_kv_heads][block] bytes, page ids[i] at offset i x n_kv_heads
 * x block bytes (the layout above).  Synchronous: it waits for the copies (and
 * so for earlier work on the legacy default stream).  A page id outside
 * [0, num_pages) returns OSCAR_ERR_INVALID and copies nothing.  ids is a host
 * array. */
oscar_status oscar_read_pages(oscar_ctx* ctx, int32_t layer, const int32_t* ids, int32_t n, void* host_dst);

/* Pages a request of length n needs mapped: logical pages 0 .. (n_hist_end-1)/P
 * where n_hist_end = n - recent (0 if no history). */
int32_t oscar_pages_needed(const oscar_config* cfg, int32_t seq_len);

/* Fork request dst off request src at src's current length n (a branch point,
 * as for parallel sampling or a shared prompt).  Source: prefix caching over the
 * INT2 cache (gist.science technical summary, section 2.2 B: the serving kernel
 * stays compatible with prefix caching; section 3: prefix reuse is kept with the
 * compressed cache).  Host block-table rows: src_bt (read),
 * dst_bt (written, capacity max_pages_per_req; unused entries set to -1).
 * History pages that the prefix fills completely are shared (refcount + 1);
 * the page holding the end of the history, if partial, is copied into a newly
 * allocated page (copy-on-write) for every layer; the BF16 window slot of src
 * is copied to dst for every layer.  Copies are enqueued on stream. */
oscar_status oscar_fork_prefix(oscar_ctx* ctx, const int32_t* src_bt, int32_t* dst_bt, int32_t n,
                               int32_t src_slot, int32_t dst_slot, void* stream);

/* ---------------------------------------------------------------- write path
 * Varlen write (prefill or extend) of tokens [start_pos[b], start_pos[b]+len_b)
 * of each request b, len_b = cu_seqlens[b+1] - cu_seqlens[b]; total_tokens =
 * cu_seqlens[batch] (host value, sizes the grid).  K, V: [total_tokens]
 * [n_kv_heads][d] in dtype (OSCAR_DTYPE_BF16 or _F32).  Ring tokens that stop
 * being recent are first quantised from their stored BF16 values into INT2;
 * then each new token goes to the sink slot, the INT2 page (rotate by R_K / R_V
 * = y = x R, clip to [-clip, clip], quantise, pack), or the recent ring.
 * cu_seqlens [batch+1], start_pos [batch], req_slot [batch]: device int32.
 * block_table: device int32 [batch][bt_stride]; every page that receives a
 * history token must be mapped (else OSCAR_DEV_BAD_PAGE and the row is
 * skipped).  R_K, R_V: device float32 [d][d].  Source: rotation and clipping
 * of the history (summary section 2.2 A/B), fused write kernel (abstract). */
oscar_status oscar_write_kv(oscar_ctx* ctx, int32_t layer, const void* K, const void* V, int32_t dtype,
                            const int32_t* cu_seqlens, const int32_t* start_pos, int32_t batch,
                            int32_t total_tokens, const float* R_K, const float* R_V, float clip_K,
                            float clip_V, const int32_t* block_table, int32_t bt_stride,
                            const int32_t* req_slot, void* stream);

/* Same as oscar_write_kv for R = H_Had . P_br (U = I, the data-oblivious
 * Hadamard-only rotation): the rotation runs as a fast Walsh-Hadamard
 * transform instead of a dense product. */
oscar_status oscar_write_kv_hadamard(oscar_ctx* ctx, int32_t layer, const void* K, const void* V, int32_t dtype,
                                     const int32_t* cu_seqlens, const int32_t* start_pos, int32_t batch,
                                     int32_t total_tokens, float clip_K, float clip_V,
                                     const int32_t* block_table, int32_t bt_stride, const int32_t* req_slot,
                                     void* stream);

/* One decode-step append per request.  Source: the sink and most recent
 * tokens stay BF16 and the history is stored as INT2 after the rotation and
 * clipping (gist.science technical summary, section 2.2 B); so when a new token
 * arrives, the oldest recent token leaves the BF16 window and is written into
 * the INT2 history by the fused write path (arXiv abstract: fused write
 * kernel).  K_new, V_new [batch][n_kv_heads][d]
 * (dtype) is token seq_lens_before[b].  If seq_lens_before[b] - W >= S the
 * oldest recent token e = seq_lens_before[b] - W is first quantised from the
 * ring into page block_table[b][e / P] slot e % P; the new token then takes
 * its ring slot (or sink slot if seq_lens_before[b] < S).  The caller maps the
 * page of e beforehand (oscar_pages_needed(seq_lens_before + 1)). */
oscar_status oscar_append_step(oscar_ctx* ctx, int32_t layer, const void* K_new, const void* V_new, int32_t dtype,
                               const int32_t* seq_lens_before, int32_t batch, const float* R_K, const float* R_V,
                               float clip_K, float clip_V, const int32_t* block_table, int32_t bt_stride,
                               const int32_t* req_slot, void* stream);

/* Declare the clip thresholds a layer's INT2 history was written with, for a
 * cache filled outside this library (an uploaded image).  The write and append
 * calls declare theirs implicitly.  The decode kernels feed the history's BF16
 * scales and zeros to f16 tensor-core operands multiplied by 2^k, where k is the
 * largest exponent with clip * 2^k < 2^14 over every clip declared for the
 * layer (the smallest k is kept); INT2 decode of a layer with no declared clip
 * returns OSCAR_ERR_INVALID.  Clips must lie in [2^-86, 16384) (else
 * OSCAR_ERR_UNSUPPORTED, also from the write calls).  Host-only. */
oscar_status oscar_set_layer_clip(oscar_ctx* ctx, int32_t layer, float clip_K, float clip_V);

/* ---------------------------------------------------------------- decode
 * Bytes of decode workspace for batch requests of at most max_seq tokens. */
oscar_status oscar_decode_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq, size_t* bytes);

/* Fused decode attention over the mixed cache (summary section 2.2 B: unpack,
 * dequantise, inverse rotation and attention for the INT2 history; abstract:
 * fused decode kernel).  q: [batch][n_q_heads][d] (q_dtype); out:
 * [batch][n_q_heads][d] float32 (out_dtype F32) or bf16 (BF16).  seq_lens
 * [batch] (device) counts every cached token including the current one; query
 * head h reads kv head h / (n_q_heads / n_kv_heads); softmax scale 1/sqrt(d).
 * The query is rotated once (q' = q R_K) to score the INT2 history in the
 * rotated basis, history values accumulate in the rotated basis, and R_V^T is
 * applied once per output row; sink/recent tokens use q and accumulate
 * unrotated; both share one softmax.  sink/recent must equal the
 * configuration.  max_seq (host) bounds seq_lens and sizes the grid.
 * workspace: device scratch of oscar_decode_workspace_size bytes (256-byte
 * aligned); its contents need no initialisation.  The layer needs a declared
 * clip threshold (a write to it, or oscar_set_layer_clip).  R_K and R_V
 * (device float32 [d][d], the layer's fixed rotations) are read before the
 * kernels wait on the work queued ahead of them: they must not be written by
 * the kernel launched immediately before this call on the stream.
 *
 * Launches (oscar_set_decode_form).  Three kernels: q_rotate, split-K and
 * combine.  One kernel: its split CTAs form the rotated query themselves and
 * the last CTA of each (request, kv head) to finish (an atomic ticket on a
 * counter the context owns; no CTA waits on another) merges that pair's
 * partials and writes its output rows; before its dependency wait it only
 * prefetches into L2.  One-launch calls on one context share its counters: do
 * not run two of them concurrently on different streams (order them with
 * events).  After a failed launch, oscar_check_status also resets the
 * counters. */
oscar_status oscar_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int32_t q_dtype, void* out,
                               int32_t out_dtype, const int32_t* block_table, int32_t bt_stride,
                               const int32_t* seq_lens, const int32_t* req_slot, int32_t batch, int32_t max_seq,
                               int32_t sink, int32_t recent, const float* R_K, const float* R_V,
                               void* workspace, size_t ws_bytes, void* stream);

/* One decode step of a layer, fused: append each request's new token and
 * attend over the cache that includes it.  Equivalent to oscar_append_step
 * with seq_lens_before[b] = seq_lens[b] - 1 followed by oscar_decode_attn with
 * seq_lens on the same stream (identical cache contents and outputs), with the
 * same arguments as those two calls (K_new, V_new: [batch][n_kv_heads][d] in
 * kv_dtype; seq_lens [batch] device int32 counts the new token).  The query
 * rotation and the append run as one grid ("step_prep": rotation CTAs first,
 * then append CTAs; no rotation CTAs when the decode is one launch), launched
 * as a programmatic dependent of the preceding kernel; the split-K kernel is
 * its dependent and reads only the page the append may be writing after the
 * dependency resolves.  The caller maps the
 * page of the evicted token beforehand, as for oscar_append_step. */
oscar_status oscar_decode_step(oscar_ctx* ctx, int32_t layer, const void* K_new, const void* V_new, int32_t kv_dtype,
                               const void* q, int32_t q_dtype, void* out, int32_t out_dtype,
                               const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                               const int32_t* req_slot, int32_t batch, int32_t max_seq, int32_t sink, int32_t recent,
                               const float* R_K, const float* R_V, float clip_K, float clip_V, void* workspace,
                               size_t ws_bytes, void* stream);

/* Allocation-free variant of oscar_decode_attn (no counterpart in the OSCAR
 * paper; it exists for callers that cannot allocate device memory).
 *
 * Some callers cannot hand over a workspace: an engine whose device memory is
 * all owned and budgeted by its own allocator, a plugin that must not call
 * cudaMalloc (which can synchronise the device and stall other work), or a
 * serving loop that is forbidden from allocating after start-up.  This call
 * takes the same arguments as oscar_decode_attn minus workspace/ws_bytes and
 * uses scratch in a file-scope device array of 8 MiB that the library keeps on
 * every GPU that loads it, until the process exits.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *  - Limit: the scratch oscar_decode_workspace_size would report for
 *    (batch, max_seq) must be at most 8 MiB (for example batch 1 up to 128K
 *    tokens at 32 q heads); larger calls return OSCAR_ERR_INVALID with a
 *    message and launch nothing.
 *  - The first call on a device looks up the array's device address (with that
 *    device current); make that first call before any stream capture.
 *  - All calls share the one array and it keeps the last call's contents
 *    (nothing in it needs to start at zero).  Calls whose kernels overlap on
 *    the GPU (different streams, or different host threads) race on it:
 *    serialise them. */
oscar_status oscar_decode_attn_noalloc(oscar_ctx* ctx, int32_t layer, const void* q, int32_t q_dtype, void* out,
                                       int32_t out_dtype, const int32_t* block_table, int32_t bt_stride,
                                       const int32_t* seq_lens, const int32_t* req_slot, int32_t batch,
                                       int32_t max_seq, int32_t sink, int32_t recent, const float* R_K,
                                       const float* R_V, void* stream);

/* ---------------------------------------------------------------- extend
 * Extend (chunked prefill) attention over the mixed cache (summary section 2.2 B:
 * the serving kernel handles paged attention and prefix caching over the INT2
 * history; section 3: prefix reuse kept with the INT2 cache).  Request b holds
 * prefix_lens[b] cached tokens and brings len_b = cu_seqlens[b+1] - cu_seqlens[b]
 * new tokens at positions prefix_lens[b] + i.  Query token i of request b
 * attends to every cached token in the form the cache stores it at length
 * prefix_lens[b] (INT2 history dequantised and rotated back, sink and recent
 * tokens BF16) and, causally, to the chunk's tokens 0..i, whose keys and
 * values are the K_new / V_new rows themselves.  Call it before writing the
 * chunk (oscar_write_kv with start_pos = prefix_lens): the cache must hold
 * exactly prefix_lens[b] tokens of request b.
 *  q: [total_tokens][n_q_heads][d] BF16; K_new, V_new: [total_tokens]
 *  [n_kv_heads][d] BF16 (another q_dtype or kv_dtype: OSCAR_ERR_UNSUPPORTED;
 *  the BF16 tiles take the query exactly as a BF16 tensor-core operand);
 *  out: [total_tokens][n_q_heads][d] float32 or bf16 (out_dtype).  q, K_new,
 *  V_new and out 16-byte aligned.  cu_seqlens [batch+1], prefix_lens [batch],
 *  req_slot [batch]: device int32; total_tokens = cu_seqlens[batch] and
 *  max_chunk >= every len_b (host values, they size the grids; a request whose
 *  chunk they do not cover sets OSCAR_DEV_BAD_LEN and gets no output).
 *  block_table [batch][bt_stride] maps the history pages of each prefix (a
 *  missing one sets OSCAR_DEV_BAD_PAGE); R_K, R_V: the layer's rotations
 *  (device float32 [d][d]); the layer needs a declared clip threshold.
 *  n_q_heads / n_kv_heads must divide 128 and batch must not exceed 65535
 *  (else OSCAR_ERR_UNSUPPORTED).
 *  workspace: device scratch of at least oscar_extend_workspace_size(cfg,
 *  total_tokens) bytes (256-byte aligned, no initialisation); it holds q R_K for
 *  every query row and R_V as f16 hi / lo planes (one per kv head with
 *  rotation_per_kv_head) for the epilogue's y R_V^T on the tensor cores.  With
 *  oscar_extend_workspace_size_unpacked(cfg, total_tokens, batch, max_prefix,
 *  max_chunk) bytes or more, the unpacked-prefix form runs: a pre-pass forms
 *  every 64-key tile that the query tiles of a request share (its INT2 history
 *  tiles, dequantised; its BF16 window tiles; its chunk's own tiles) once per
 *  call into the workspace, and the attention CTAs of all the request's query
 *  tiles copy those tiles instead of each forming them from the pages and rows.
 *  The workspace holds the window and chunk tiles for this max_chunk and T INT2
 *  tiles per (request, kv head), T as many as fit; a request with more history
 *  tiles forms its own.  Both forms give identical outputs.  Softmax scale 1/sqrt(d), query
 *  head h reads kv head h / (n_q_heads / n_kv_heads).  Kernels on the stream:
 *  the pre-pass (unpacked form), the query rotation, then the tensor-core
 *  attention (timing name "extend"). */
oscar_status oscar_extend_workspace_size(const oscar_config* cfg, int32_t total_tokens, size_t* bytes);
/* Workspace of the unpacked-prefix form for batch requests whose prefixes hold at
 * most max_prefix tokens and whose chunks at most max_chunk (the max_chunk given
 * to oscar_extend_attn): the base size plus, per (request, kv head), one operand
 * tile (42 KB at d = 128, 26 KB at d = 64) per 64 positions of the INT2 history
 * (672 B per history token and kv head at d = 128, against the cache's 96 B: a
 * working copy for one call), of the BF16 window and of the chunk.  Negative
 * arguments: OSCAR_ERR_INVALID. */
oscar_status oscar_extend_workspace_size_unpacked(const oscar_config* cfg, int32_t total_tokens, int32_t batch,
                                                  int32_t max_prefix, int32_t max_chunk, size_t* bytes);
oscar_status oscar_extend_attn(oscar_ctx* ctx, int32_t layer, const void* q, int32_t q_dtype, const void* K_new,
                               const void* V_new, int32_t kv_dtype, void* out, int32_t out_dtype,
                               const int32_t* cu_seqlens, const int32_t* prefix_lens, int32_t batch,
                               int32_t total_tokens, int32_t max_chunk, const int32_t* block_table, int32_t bt_stride,
                               const int32_t* req_slot, const float* R_K, const float* R_V, void* workspace,
                               size_t ws_bytes, void* stream);

/* One chunked-prefill step of a layer: oscar_extend_attn followed by
 * oscar_write_kv of the same chunk (start_pos = prefix_lens), with the
 * arguments of those two calls on one stream (identical outputs and cache
 * contents).  The write runs after the attention has read the window slots and
 * pages it overwrites.  clip_K and clip_V are declared for the layer first, so
 * the first chunk of a fresh layer may use this call.  The caller maps the pages
 * that the chunk's history tokens (and the ring tokens it evicts) land in,
 * as for oscar_write_kv. */
oscar_status oscar_extend_step(oscar_ctx* ctx, int32_t layer, const void* q, int32_t q_dtype, const void* K_new,
                               const void* V_new, int32_t kv_dtype, void* out, int32_t out_dtype,
                               const int32_t* cu_seqlens, const int32_t* prefix_lens, int32_t batch,
                               int32_t total_tokens, int32_t max_chunk, const int32_t* block_table, int32_t bt_stride,
                               const int32_t* req_slot, const float* R_K, const float* R_V, float clip_K,
                               float clip_V, void* workspace, size_t ws_bytes, void* stream);

/* In-house comparison: standard split-K paged decode over an all-BF16 cache
 * (layout above), same grid and staging as the INT2 kernel.  bf16_pool points
 * at the whole [num_layers][num_pages]... pool; workspace from
 * oscar_bf16_decode_workspace_size. */
oscar_status oscar_bf16_decode_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq,
                                              size_t* bytes);
oscar_status oscar_bf16_decode_attn(oscar_ctx* ctx, int32_t layer, const void* bf16_pool, const void* q,
                                    int32_t q_dtype, void* out, int32_t out_dtype, const int32_t* block_table,
                                    int32_t bt_stride, const int32_t* seq_lens, int32_t batch, int32_t max_seq,
                                    void* workspace, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- 8-bit cache
 * A paged cache at 8 bits beside the INT2 one, for requests or models that need more
 * than 2 bits (no rotation, no clip threshold), with its own attention calls.  It
 * shares the context's page allocator and block tables: page id p addresses block p
 * of the 8-bit pool as it does in the INT2 pool.  Its pool spans every layer of the
 * context, and a fork carries a request in one of the two caches: a model that keeps
 * some layers at 2 bits and others at 8 takes a context for each kind, with page ids
 * of its own.
 *
 * Tokens.  Page j of a request holds tokens j*P .. j*P + P-1.  A page is quantised
 * when its last token arrives; the n % P tokens of the page that is not complete yet
 * are BF16 rows in the tail slab.  So what the cache holds at length n does not
 * depend on how the tokens arrived (one prompt, chunks or single tokens).  F32 rows
 * are rounded to BF16 on entry.
 *
 * 8-bit pool: [num_layers][num_pages][n_kv_heads][block], one (layer, page, kv head)
 * block of oscar_kv8_block_bytes bytes being
 *     K codes [P][d] | V codes [P][d] | K scale, V scale (float32), 8 unused bytes |
 *     K lo [d] | K hi [d] | unused bytes up to a multiple of 128
 * Token rows are d bytes in channel order, but the 16-byte chunks of each 128-byte
 * line of a code section are stored at place (chunk ^ turn), with turn = 4 (t & 1)
 * for K at d = 128, 0 for K at d = 64, and 2 ((t >> 1) & 3) for V, t being the chunk's
 * token in the page.
 *   OSCAR_KV8_INT8: byte = code + 128, code in [-127, 127], M = 127.  A uniform step
 *     per block: the closer format for values of even size.
 *   OSCAR_KV8_E4M3: byte = the 8-bit floating-point number (4 exponent, 3 mantissa
 *     bits), M = 448.  A relative step: for channels that differ much in size.
 * With m = max |x| over the block's finite values: scale = m / M (float32), code =
 * x M / m rounded to nearest even, dequantised value = code * scale.  A block with
 * m < 2^-100 is stored as zeros with scale 0.  An infinity saturates, a NaN is stored
 * as 0, and both set OSCAR_DEV_BAD_VALUE.  lo and hi are the smallest and largest K
 * code of each channel over the page's tokens (-0 as +0), for oscar_kv8_select_pages.
 *
 * Tail slab: [num_layers][max_requests][n_kv_heads][2 (K,V)][P][d] bf16, token t at
 * row t mod P.
 *
 * Row arguments (K, V, q) have heads x d adjacent elements per token and a stride in
 * elements between tokens, heads x d at least (a slice of a wider projection needs no copy;
 * 0: adjacent tokens, not one row for all of them); the address and the stride in bytes must be multiples of 16.  Every kernel call must be made
 * with the device current on which the buffers were bound (else OSCAR_ERR_INVALID),
 * takes at most 65535 requests (else OSCAR_ERR_UNSUPPORTED), needs no allocation and
 * can be captured into a graph (after one such call outside a capture).  Requests of one
 * call have distinct req_slots and write distinct pages.  Workspaces are scratch of the
 * one call, 256-byte aligned, with no initialisation; calls whose kernels may run at the
 * same time need a workspace each. */
enum { OSCAR_KV8_INT8 = 0, OSCAR_KV8_E4M3 = 1 };

/* Bytes of the 8-bit pool / tail slab / one block for a configuration (sink, recent
 * and group_size do not matter to them); 0 if the configuration is invalid. */
size_t oscar_kv8_pool_bytes(const oscar_config* cfg);
size_t oscar_kv8_tail_bytes(const oscar_config* cfg);
size_t oscar_kv8_block_bytes(const oscar_config* cfg);

/* Pages a request of length n needs mapped in the 8-bit cache: n / P, its complete
 * pages.  -1 for an invalid configuration or a negative length. */
int32_t oscar_kv8_pages_needed(const oscar_config* cfg, int32_t seq_len);

/* Bind an 8-bit cache (caller-owned device buffers of the sizes above, 16-byte
 * aligned) to a context, which may be one created without INT2 buffers.  Once per
 * context; the context keeps both pointers until oscar_destroy.  Allocates the 4-byte
 * status word if the context has none. */
oscar_status oscar_kv8_bind(oscar_ctx* ctx, int32_t format, void* pool, void* tail);

/* Varlen write (prefill or extend) of tokens [start_pos[b], start_pos[b]+len_b) of each
 * request b; cu_seqlens, start_pos, req_slot, block_table and total_tokens as for
 * oscar_write_kv.  K, V: [total_tokens][n_kv_heads][d] in dtype, tokens k_stride and
 * v_stride elements apart.  cu_seqlens must not decrease (else OSCAR_DEV_BAD_LEN, and rows
 * of other requests may be missing too).  The cache must hold exactly start_pos[b] tokens of
 * request b (its tail rows are read).  Every page that the chunk completes must be mapped (else
 * OSCAR_DEV_BAD_PAGE and that page is not stored). */
oscar_status oscar_kv8_write(oscar_ctx* ctx, int32_t layer, const void* K, int64_t k_stride, const void* V,
                             int64_t v_stride, int32_t dtype, const int32_t* cu_seqlens, const int32_t* start_pos,
                             int32_t batch, int32_t total_tokens, const int32_t* block_table, int32_t bt_stride,
                             const int32_t* req_slot, void* stream);

/* One token per request: K_new, V_new [batch][n_kv_heads][d] become token
 * seq_lens_before[b], row seq_lens_before[b] mod P of the tail; a request whose page it
 * completes has that page quantised (and needs it mapped).  Same cache contents as
 * oscar_kv8_write of the same tokens.  seq_lens_before[b] = -1 skips request b (a padded
 * batch); its length in the attention calls is then 0. */
oscar_status oscar_kv8_append(oscar_ctx* ctx, int32_t layer, const void* K_new, int64_t k_stride, const void* V_new,
                              int64_t v_stride, int32_t dtype, const int32_t* seq_lens_before, int32_t batch,
                              const int32_t* block_table, int32_t bt_stride, const int32_t* req_slot, void* stream);

/* Decode attention over the 8-bit cache: o = softmax(q K^T / sqrt(d)) V over the
 * seq_lens[b] / P complete pages and the seq_lens[b] mod P tail rows.  q: [batch]
 * [n_q_heads][d], requests q_stride elements apart; out: [batch][n_q_heads][d] adjacent,
 * 16-byte aligned; the other arguments as for oscar_decode_attn.  A request of length 0
 * (or of a bad length) gets zeros; a page that is not mapped is left out and sets
 * OSCAR_DEV_BAD_PAGE.  The output is a float32 evaluation's for finite scores of any size.  (A
 * query whose largest components meet keys of 0 only, while components below 2^-20 of them decide
 * the weights, takes 20 to 90 times the time.)  A NaN or an infinity in q or in a tail row makes
 * NaN of the outputs that depend on it (an infinite key or value of a tail row may count by its
 * limit). */
oscar_status oscar_kv8_decode_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq, size_t* bytes);
oscar_status oscar_kv8_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                   void* out, int32_t out_dtype, const int32_t* block_table, int32_t bt_stride,
                                   const int32_t* seq_lens, const int32_t* req_slot, int32_t batch, int32_t max_seq,
                                   void* workspace, size_t ws_bytes, void* stream);

/* Select the pages that sparse decode reads.  For a page p of a kv head,
 *     U_p = scale_p sum_c (a_c hi_pc - b_c lo_pc),
 *     a_c = sum_h max(q_hc, 0),  b_c = sum_h max(-q_hc, 0)  over the heads h that share it,
 * is the sum over those heads of an upper bound of q_h . k over the page's keys.
 * page_idx [batch][n_kv_heads][n_select] receives logical page indexes in ascending
 * order, -1 after the last: the first keep_first and the last keep_last complete pages
 * of the request, then those of the largest U_p, the lowest index first among equal
 * ones; every complete page when there are no more than n_select.  1 <= n_select,
 * keep_first + keep_last <= n_select.  Pages are ordered by U_p to about 48 bits (a NaN in q
 * counts as 0, an infinity leaves the choice open; a page that is not mapped comes last and sets
 * OSCAR_DEV_BAD_PAGE).  The list may
 * serve several calls (later tokens, other layers) as long as its pages are complete. */
oscar_status oscar_kv8_select_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq, size_t* bytes);
oscar_status oscar_kv8_select_pages(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                    const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                    int32_t batch, int32_t max_seq, int32_t keep_first, int32_t keep_last,
                                    int32_t n_select, int32_t* page_idx, void* workspace, size_t ws_bytes,
                                    void* stream);

/* oscar_kv8_decode_attn over the listed pages of each (request, kv head) and the tail
 * rows.  page_idx [batch][n_kv_heads][n_select] (device): complete pages of the request,
 * strictly ascending, negative entries after the last.  An entry that is out of order,
 * given twice or not a complete page sets OSCAR_DEV_BAD_PAGE and is left out, or counts
 * again where it is not next to its like: check the status before using the output. */
oscar_status oscar_kv8_sparse_workspace_size(const oscar_config* cfg, int32_t batch, int32_t n_select, size_t* bytes);
oscar_status oscar_kv8_sparse_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride,
                                          int32_t q_dtype, void* out, int32_t out_dtype, const int32_t* page_idx,
                                          int32_t n_select, const int32_t* block_table, int32_t bt_stride,
                                          const int32_t* seq_lens, const int32_t* req_slot, int32_t batch,
                                          void* workspace, size_t ws_bytes, void* stream);

/* Decode attention of requests that share a prefix: what oscar_kv8_decode_attn computes, with the shared pages of a
 * group read once for all of its requests (samples or beams of one prompt, conversations behind one
 * system prompt).  Group i holds requests group_starts[i] .. group_starts[i + 1] - 1 of the batch, and the first
 * shared_pages[i] entries of their block-table rows are the same pages (forks of n tokens share n / P).
 * group_starts [n_groups + 1], ascending from 0 to batch, and shared_pages [n_groups]: device int32; a group may hold one
 * request or none, and share no page.  A group's shared pages are found through the row of its first request that
 * is not empty.  max_shared (pages) bounds shared_pages and max_own (tokens) what the requests hold behind them
 * (host values, they size the grids and the workspace); the other arguments as for
 * oscar_kv8_decode_attn.  A request of length 0 (a padded batch) gets zeros; one that no group holds, that is shorter
 * than its group's shared pages or beyond the bounds gets zeros and sets OSCAR_DEV_BAD_LEN; a page that is not
 * mapped is left out and sets OSCAR_DEV_BAD_PAGE.
 * Next to oscar_kv8_decode_attn the shared part's weights have fewer bits: 22 for float32 outputs, and for BF16 ones 11 (a
 * weight is off by up to 2^-11 of itself, where the output's own rounding is 2^-8; some 6 to 8 % of the values come out
 * one BF16 step apart).  A caller who wants the nearest BF16 numbers asks for float32 and rounds.
 * The workspace size holds for every call of at most batch requests in at most n_groups groups with the same
 * max_shared and max_own: a program whose requests finish or whose groups end keeps its
 * workspace. */
oscar_status oscar_kv8_shared_workspace_size(const oscar_config* cfg, int32_t batch, int32_t n_groups, int32_t max_shared,
                                             int32_t max_own, size_t* bytes);
oscar_status oscar_kv8_shared_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                          void* out, int32_t out_dtype, const int32_t* group_starts,
                                          const int32_t* shared_pages, int32_t n_groups, int32_t max_shared,
                                          const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                          const int32_t* req_slot, int32_t batch, int32_t max_own, void* workspace,
                                          size_t ws_bytes, void* stream);

/* Fork n_dst requests off request src at its current length n in the 8-bit cache (parallel
 * sampling, beams, a shared prompt).  Host arrays: src_bt (n / P entries are read), dst_slots
 * [n_dst] (distinct, not src_slot), dst_bt [n_dst][max_pages_per_req] (written; unused entries
 * -1).  The n / P complete pages are shared (each refcount + n_dst); the n mod P tail rows are
 * copied to every destination slot, in every layer, by one kernel on stream.  On an error
 * nothing is forked.  Without a bound cache only the host part is done.  The allocator changes
 * at the call, so a stream that is being captured is refused.  It copies no
 * INT2 window, and oscar_fork_prefix neither 8-bit blocks nor tail rows: a request that is
 * forked keeps its tokens in one of the two caches. */
oscar_status oscar_kv8_fork(oscar_ctx* ctx, const int32_t* src_bt, int32_t n, int32_t src_slot,
                            const int32_t* dst_slots, int32_t n_dst, int32_t* dst_bt, void* stream);

/* The states of beams after a selection: request b * beams + j of the new batch continues request
 * b * beams + parents[b][j] of the old one (1 <= beams <= 64; -1: an empty request, of length 0 and with a row of -1).
 * new_block_table [batch * beams][bt_stride] and new_seq_lens [batch * beams] receive the parents' rows and lengths.
 * new_req_slot: a parent's first child (the lowest j) keeps its slot; every other beam, in ascending order of j,
 * takes the slot of an old beam without a child, in ascending order of those, and unless it is empty
 * its parent's seq_lens mod P tail rows are copied there in every layer (other rows of the slab stay as they are).  So
 * an item's slots are the same ones before and after, and a beam's tail moves only if its parent has
 * several children.  All arguments are device int32; the outputs must overlap neither the inputs nor one another (else
 * OSCAR_ERR_INVALID).  A parent out of range counts as -1 and sets OSCAR_DEV_BAD_SLOT; a slot out of range that a beam
 * keeps or takes sets OSCAR_DEV_BAD_SLOT and a parent's length out of range OSCAR_DEV_BAD_LEN, whether rows would be
 * copied or not: they are not copied, and the new arrays hold the slot or length as it was.  The call can be captured into a graph: it does not touch
 * the page allocator, whose refcounts follow with oscar_ref_pages of the parent's pages for every further child and
 * oscar_unref_pages of the pages of every beam without one, before the next page is allocated. */
oscar_status oscar_kv8_reorder(oscar_ctx* ctx, const int32_t* parents, int32_t batch, int32_t beams, const int32_t* block_table,
                               int32_t bt_stride, const int32_t* seq_lens, const int32_t* req_slot, int32_t* new_block_table,
                               int32_t* new_seq_lens, int32_t* new_req_slot, void* stream);

/* The next beams of a beam search.  Candidate (i, v) of a batch item continues beam i with token v and has
 *     key = scores[i] + ((x_v - m) - log sum_u e^(x_u - m)),  x = logits[i], m = max x,
 * the sum of log probabilities so far.  The n_out candidates of the largest keys, compared in 64 bits, in descending order; among
 * equal keys the lowest beam comes first, within a beam the larger logit (a small difference may be lost in a large score), then the lowest
 * token: out_scores [batch][n_out] (the keys, rounded to float32), out_tokens (v) and out_parents (i, as
 * oscar_kv8_reorder takes them), both int32.
 *  logits: rows [batch][beams][vocab] of dtype (BF16 or F32), row_stride elements apart (0: adjacent) and aligned to
 *  their elements only (16-byte aligned rows are read fastest).  scores: [batch][beams] float32; a beam at -infinity has no
 *  candidates (beams 1 .. of a first step).  finished [batch][beams] (bytes; NULL: none): a beam that is not 0 there has one candidate,
 *  (i, pad_token) with its score unchanged, and its logits are not read.
 * A candidate at -infinity (a masked token) is never taken: where there are fewer than n_out others,
 * the rest of the outputs is -infinity, -1, -1.  A NaN or +infinity among a beam's logits or as its score
 * leaves the beam out and sets OSCAR_DEV_BAD_VALUE.  Exponentials and their sums are float32's (the normaliser is good to
 * 10^-6): candidates of different beams whose keys differ by less may come in either order; equal rows and scores
 * are equal.  1 <= beams, n_out <= 64, vocab <= 2^24.  The context is any one with device buffers; the workspace's
 * rules are those of the 8-bit cache's calls; outputs and workspace must overlap neither the inputs nor one another
 * (else OSCAR_ERR_INVALID). */
oscar_status oscar_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t n_out, size_t* bytes);
oscar_status oscar_beam_select(oscar_ctx* ctx, const void* logits, int64_t row_stride, int32_t dtype, const float* scores,
                               const uint8_t* finished, int32_t pad_token, int32_t batch, int32_t beams, int32_t vocab,
                               int32_t n_out, float* out_scores, int32_t* out_tokens, int32_t* out_parents, void* workspace,
                               size_t ws_bytes, void* stream);

/* Move the allocated pages down to ids [0, live), live = pages in use, so that the rest of
 * the pools holds nothing: every allocated page with an id >= live moves to a free id below,
 * in every layer of the INT2 pool and of the bound 8-bit pool (not of a caller's BF16
 * comparison pool).  block_table [rows][bt_stride]
 * (device int32, adjacent rows; rows = 0 for none) is rewritten to the new ids; out_map [num_pages]
 * (host) gives every page's new id (-1 for a free one) for block tables on the host, and
 * *out_live receives live.  Refcounts move with their pages, and fresh pages are handed out from
 * live upwards.  The copies and the rewriting run on stream; every block table that maps a moved
 * page must be rewritten before its next use, and work on other streams that reads those pages
 * must be ordered around the call.  On an error no page has moved and block_table has its old
 * entries.  The allocator changes at the call, so a stream that is being captured is refused. */
oscar_status oscar_compact_pages(oscar_ctx* ctx, int32_t* block_table, int32_t rows, int32_t bt_stride,
                                 int32_t* out_map, int32_t* out_live, void* stream);

/* Self-test of the device-side failure path (no counterpart in the OSCAR
 * paper).  Every kernel bounds its mbarrier waits and, when one runs out, sets
 * OSCAR_DEV_TIMEOUT in the status word instead of trapping, so the context
 * stays usable.  This call launches one small kernel that waits on a barrier
 * nothing arrives on until limit_us microseconds (1 .. 1e6) have passed, then
 * sets OSCAR_DEV_TIMEOUT; oscar_check_status reports it and clears it. */
oscar_status oscar_selftest_wait_timeout(oscar_ctx* ctx, int32_t limit_us, void* stream);

/* ---------------------------------------------------------------- status, tracing
 * Synchronise stream, read and clear the device status word.  Returns
 * OSCAR_ERR_DEVICE (bits in *out_bits if non-NULL) if any kernel flagged an
 * error since the last check. */
oscar_status oscar_check_status(oscar_ctx* ctx, void* stream, int32_t* out_bits);

/* ---------------------------------------------------------------- decode launch form
 * How the INT2 decode calls (oscar_decode_attn, oscar_decode_step,
 * oscar_decode_attn_noalloc) launch: OSCAR_DECODE_AUTO (the library's choice
 * for the batch; the default), OSCAR_DECODE_THREE_KERNELS (query rotation,
 * split-K and combine kernels) or OSCAR_DECODE_ONE_LAUNCH (the one-kernel
 * form described at oscar_decode_attn whenever batch <= max_requests, three
 * kernels otherwise).  The forms agree within floating-point rounding (the
 * rotated query is summed in another order).  Host-only; OSCAR_ERR_INVALID
 * for any other value. */
#define OSCAR_DECODE_AUTO 0
#define OSCAR_DECODE_THREE_KERNELS 1
#define OSCAR_DECODE_ONE_LAUNCH 2
oscar_status oscar_set_decode_form(oscar_ctx* ctx, int32_t form);

/* Kernel timing for tracing: when enabled, the library brackets each launch
 * of the named kernel family with CUDA events on the launch stream.
 * oscar_kernel_time returns the summed milliseconds and launch count since the
 * last reset (synchronises the recorded events).  Names: "decode_splitk",
 * "decode_combine", "q_rotate", "step_prep", "append", "evict", "write", "bf16_prepare",
 * "bf16_decode", "bf16_combine", "extend", "selftest", "kv8_write", "kv8_append", "kv8_decode",
 * "kv8_combine" (not launched for contexts or selections of up to 512 tokens, 1024 at d = 64
 * and P >= 32), "kv8_select", "kv8_fork", "kv8_prefix", "kv8_reorder", "beam_units", "beam_pick", "copy_pages", "remap_table".  Launches recorded into a CUDA graph get external event-record nodes: replay the graph
 * once, then read; the events return to the library when read, so a graph
 * captured with timing on is replayed at most once.  With timing on, the decode
 * kernels are launched without programmatic dependent launch. */
oscar_status oscar_set_timing(oscar_ctx* ctx, int32_t enable);
oscar_status oscar_kernel_time(oscar_ctx* ctx, const char* name, double* out_ms, int32_t* out_launches);
oscar_status oscar_reset_timing(oscar_ctx* ctx);

/* Number of kernel launches this context has issued (all families). */
int64_t oscar_launch_count(oscar_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* OSCAR_H_ */
