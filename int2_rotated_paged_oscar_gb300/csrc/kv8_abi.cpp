// C ABI of the 8-bit paged cache and of the page moves (see include/oscar.h).
#include <algorithm>
#include <new>
#include <vector>

#include "kv8_internal.h"
#include "oscar_ctx.h"

using oscar::check_layer;
using oscar::check_workspace;
using oscar::cuda_fail;
using oscar::fail;
using oscar::Geom;
using oscar::Kv8DecodeArgs;
using oscar::Kv8SelectArgs;
using oscar::Kv8WriteArgs;
using oscar::LaunchScope;
using oscar::validate;

namespace {

constexpr int kMaxGrid = 65535;  // of the grid's second and third dimension

// The buffers were bound on one device and the kernels run on the current one.
oscar_status check_device(const oscar_ctx* ctx) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "current device");
  if (dev != ctx->device)
    return fail(OSCAR_ERR_INVALID, "the context's buffers are on device %d, the current device is %d", ctx->device, dev);
  return OSCAR_OK;
}

// The allocator changes at the call: a captured one would move pages by an old plan at every replay.
oscar_status check_not_capturing(void* stream, const char* name) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs) != cudaSuccess) {
    (void)cudaGetLastError();  // (the legacy stream during another one's capture: a launch there reports it)
    return OSCAR_OK;
  }
  if (cs != cudaStreamCaptureStatusNone) return fail(OSCAR_ERR_INVALID, "%s cannot be captured into a graph", name);
  return OSCAR_OK;
}

oscar_status need_kv8(oscar_ctx* ctx) {
  if (!ctx) return fail(OSCAR_ERR_INVALID, "context is null");
  if (!ctx->kv8_pool) return fail(OSCAR_ERR_INVALID, "no 8-bit cache is bound to the context (oscar_kv8_bind)");
  return check_device(ctx);
}

// Rows of heads x d elements, *stride elements apart (0: adjacent), read in 16-byte vectors.
oscar_status check_rows(const char* name, const void* p, int64_t* stride, int heads, int d, int dtype) {
  if (*stride == 0) *stride = (int64_t)heads * d;
  const long long row_stride = *stride;
  if (dtype != OSCAR_DTYPE_BF16 && dtype != OSCAR_DTYPE_F32) return fail(OSCAR_ERR_INVALID, "bad dtype %d of %s", dtype, name);
  const long long elem = dtype == OSCAR_DTYPE_BF16 ? 2 : 4;
  if (!p) return fail(OSCAR_ERR_INVALID, "%s is null", name);
  if (row_stride < (long long)heads * d)
    return fail(OSCAR_ERR_INVALID, "row stride %lld of %s is below the row's %d elements", row_stride, name, heads * d);
  if ((reinterpret_cast<uintptr_t>(p) & 15) || (row_stride * elem) % 16)
    return fail(OSCAR_ERR_INVALID, "%s and its row stride must be 16-byte aligned", name);
  return OSCAR_OK;
}

oscar_status check_batch(int32_t batch, int32_t bt_stride) {
  if (batch < 0 || bt_stride < 1) return fail(OSCAR_ERR_INVALID, "bad batch/bt_stride");
  if (batch > kMaxGrid) return fail(OSCAR_ERR_UNSUPPORTED, "batch %d exceeds %d", batch, kMaxGrid);
  return OSCAR_OK;
}

oscar_status write_rows(oscar_ctx* ctx, int32_t layer, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                        int32_t dtype, const int32_t* cu_seqlens, const int32_t* start_pos, int32_t batch,
                        int32_t total_tokens, const int32_t* block_table, int32_t bt_stride, const int32_t* req_slot,
                        void* stream, const char* name) {
  oscar_status st = need_kv8(ctx);
  if (st != OSCAR_OK) return st;
  if ((st = check_layer(ctx, layer)) != OSCAR_OK) return st;
  if ((st = check_batch(batch, bt_stride)) != OSCAR_OK) return st;
  if (total_tokens < 0) return fail(OSCAR_ERR_INVALID, "total_tokens %d is negative", total_tokens);
  if (batch == 0 || total_tokens == 0) return OSCAR_OK;
  if (!start_pos || !block_table || !req_slot) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  const Geom& g = ctx->g;
  if ((st = check_rows("K", K, &k_stride, g.Hkv, g.D, dtype)) != OSCAR_OK) return st;
  if ((st = check_rows("V", V, &v_stride, g.Hkv, g.D, dtype)) != OSCAR_OK) return st;
  Kv8WriteArgs a{};
  a.g = g;
  a.fmt = ctx->kv8_format;
  a.layer = layer;
  a.K = K;
  a.V = V;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.dtype = dtype;
  a.cu_seqlens = cu_seqlens;
  a.start_pos = start_pos;
  a.batch = batch;
  a.total_tokens = total_tokens;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.req_slot = req_slot;
  a.pool = ctx->kv8_pool;
  a.tail = ctx->kv8_tail;
  a.status = ctx->d_status;
  LaunchScope ls(ctx, name, stream);
  const int e = oscar::launch_kv8_write(a, stream, !ctx->timing);
  ls.done(e);
  if (e) return cuda_fail(e, "8-bit write launch");
  return OSCAR_OK;
}

constexpr int kMaxSelect = 1 << 24;

oscar_status check_select(int32_t n_select) {
  if (n_select < 1) return fail(OSCAR_ERR_INVALID, "n_select %d is below 1", n_select);
  if (n_select > kMaxSelect) return fail(OSCAR_ERR_UNSUPPORTED, "n_select %d exceeds %d", n_select, kMaxSelect);
  return OSCAR_OK;
}

// What the two attention calls and the selection have in common.
oscar_status check_query(oscar_ctx* ctx, int32_t layer, const void* q, int64_t* q_stride, int32_t q_dtype,
                         const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch) {
  oscar_status st = need_kv8(ctx);
  if (st != OSCAR_OK) return st;
  if ((st = check_layer(ctx, layer)) != OSCAR_OK) return st;
  if ((st = check_batch(batch, bt_stride)) != OSCAR_OK) return st;
  if (batch == 0) return OSCAR_OK;
  if (!block_table || !seq_lens) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  return check_rows("q", q, q_stride, ctx->g.Hq, ctx->g.D, q_dtype);
}

oscar_status check_max_seq(const oscar_ctx* ctx, int32_t max_seq) {
  if (max_seq < 0) return fail(OSCAR_ERR_INVALID, "max_seq %d is negative", max_seq);
  if ((long long)max_seq > (long long)ctx->g.max_pages_per_req * ctx->g.P)
    return fail(OSCAR_ERR_INVALID, "max_seq %d exceeds max_pages_per_req * page_size", max_seq);
  return OSCAR_OK;
}

oscar_status attend(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype, void* out,
                    int32_t out_dtype, const int32_t* page_idx, int32_t n_select, const int32_t* block_table,
                    int32_t bt_stride, const int32_t* seq_lens, const int32_t* req_slot, int32_t batch, int32_t max_seq,
                    void* workspace, size_t ws_bytes, void* stream) {
  oscar_status st;
  if (!req_slot || !out) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  if (out_dtype != OSCAR_DTYPE_BF16 && out_dtype != OSCAR_DTYPE_F32) return fail(OSCAR_ERR_INVALID, "bad out dtype");
  if (reinterpret_cast<uintptr_t>(out) & 15) return fail(OSCAR_ERR_INVALID, "out must be 16-byte aligned");
  if ((st = check_workspace(workspace)) != OSCAR_OK) return st;
  Kv8DecodeArgs a{};
  a.g = ctx->g;
  a.fmt = ctx->kv8_format;
  a.layer = layer;
  a.q = q;
  a.q_stride = q_stride;
  a.q_dtype = q_dtype;
  a.out = out;
  a.out_dtype = out_dtype;
  a.page_idx = page_idx;
  a.n_select = n_select;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.req_slot = req_slot;
  a.batch = batch;
  a.max_seq = max_seq;
  a.pool = ctx->kv8_pool;
  a.tail = ctx->kv8_tail;
  a.status = ctx->d_status;
  a.part = static_cast<float*>(workspace);
  a.wl = oscar::kv8_plan(ctx->g, batch, page_idx ? n_select : max_seq / ctx->g.P);
  if (ws_bytes < a.wl.total) return fail(OSCAR_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, a.wl.total);
  const bool pdl = !ctx->timing;
  {
    LaunchScope ls(ctx, "kv8_decode", stream);
    const int e = oscar::launch_kv8_decode(a, stream, pdl);
    ls.done(e);
    if (e) return cuda_fail(e, "8-bit decode launch");
  }
  if (a.wl.max_splits == 1) return OSCAR_OK;  // the one split of a request has written its output
  LaunchScope ls(ctx, "kv8_combine", stream);
  const int e = oscar::launch_kv8_combine(a, stream, pdl);
  ls.done(e);
  if (e) return cuda_fail(e, "8-bit combine launch");
  return OSCAR_OK;
}

}  // namespace

extern "C" {

size_t oscar_kv8_pool_bytes(const oscar_config* cfg) {
  Geom g;
  return validate(cfg, &g) == OSCAR_OK ? oscar::kv8_pool_bytes(g) : 0;
}

size_t oscar_kv8_tail_bytes(const oscar_config* cfg) {
  Geom g;
  return validate(cfg, &g) == OSCAR_OK ? oscar::kv8_tail_bytes(g) : 0;
}

size_t oscar_kv8_block_bytes(const oscar_config* cfg) {
  Geom g;
  return validate(cfg, &g) == OSCAR_OK ? oscar::kv8_geom(g).block_bytes() : 0;
}

int32_t oscar_kv8_pages_needed(const oscar_config* cfg, int32_t seq_len) {
  Geom g;
  if (validate(cfg, &g) != OSCAR_OK || seq_len < 0) return -1;
  return seq_len / g.P;
}

oscar_status oscar_kv8_bind(oscar_ctx* ctx, int32_t format, void* pool, void* tail) {
  if (!ctx) return fail(OSCAR_ERR_INVALID, "context is null");
  if (format != OSCAR_KV8_INT8 && format != OSCAR_KV8_E4M3) return fail(OSCAR_ERR_INVALID, "unknown 8-bit format %d", format);
  if (!pool || !tail) return fail(OSCAR_ERR_INVALID, "the pool and the tail slab are device buffers, not null");
  if ((reinterpret_cast<uintptr_t>(pool) | reinterpret_cast<uintptr_t>(tail)) & 15)
    return fail(OSCAR_ERR_INVALID, "the pool and the tail slab must be 16-byte aligned");
  if (ctx->kv8_pool) return fail(OSCAR_ERR_INVALID, "an 8-bit cache is bound to the context already");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "current device");
  if (ctx->d_status && dev != ctx->device)
    return fail(OSCAR_ERR_INVALID, "the context's buffers are on device %d, the current device is %d", ctx->device, dev);
  if (!ctx->d_status) {
    int* word = nullptr;
    e = cudaMalloc(&word, sizeof(int));
    if (e == cudaSuccess) e = cudaMemset(word, 0, sizeof(int));
    if (e != cudaSuccess) {
      if (word) cudaFree(word);
      return cuda_fail(e, "status word");
    }
    ctx->d_status = word;
    ctx->device = dev;
  }
  ctx->kv8_format = format;
  ctx->kv8_pool = static_cast<uint8_t*>(pool);
  ctx->kv8_tail = static_cast<uint16_t*>(tail);
  return OSCAR_OK;
}

oscar_status oscar_kv8_write(oscar_ctx* ctx, int32_t layer, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                             int32_t dtype, const int32_t* cu_seqlens, const int32_t* start_pos, int32_t batch,
                             int32_t total_tokens, const int32_t* block_table, int32_t bt_stride, const int32_t* req_slot,
                             void* stream) {
  if (batch > 0 && total_tokens > 0 && !cu_seqlens) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  return write_rows(ctx, layer, K, k_stride, V, v_stride, dtype, cu_seqlens, start_pos, batch, total_tokens, block_table,
                    bt_stride, req_slot, stream, "kv8_write");
}

oscar_status oscar_kv8_append(oscar_ctx* ctx, int32_t layer, const void* K_new, int64_t k_stride, const void* V_new,
                              int64_t v_stride, int32_t dtype, const int32_t* seq_lens_before, int32_t batch,
                              const int32_t* block_table, int32_t bt_stride, const int32_t* req_slot, void* stream) {
  return write_rows(ctx, layer, K_new, k_stride, V_new, v_stride, dtype, nullptr, seq_lens_before, batch, batch, block_table,
                    bt_stride, req_slot, stream, "kv8_append");
}

oscar_status oscar_kv8_decode_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq, size_t* bytes) {
  Geom g;
  const oscar_status st = validate(cfg, &g);
  if (st != OSCAR_OK) return st;
  if (!bytes || batch < 0 || max_seq < 0) return fail(OSCAR_ERR_INVALID, "bad arguments to workspace size");
  *bytes = oscar::kv8_plan(g, batch, max_seq / g.P).total;
  return OSCAR_OK;
}

oscar_status oscar_kv8_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype, void* out,
                                   int32_t out_dtype, const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                   const int32_t* req_slot, int32_t batch, int32_t max_seq, void* workspace, size_t ws_bytes,
                                   void* stream) {
  oscar_status st = check_query(ctx, layer, q, &q_stride, q_dtype, block_table, bt_stride, seq_lens, batch);
  if (st != OSCAR_OK) return st;
  if ((st = check_max_seq(ctx, max_seq)) != OSCAR_OK || batch == 0) return st;
  return attend(ctx, layer, q, q_stride, q_dtype, out, out_dtype, nullptr, 0, block_table, bt_stride, seq_lens, req_slot,
                batch, max_seq, workspace, ws_bytes, stream);
}

oscar_status oscar_kv8_select_workspace_size(const oscar_config* cfg, int32_t batch, int32_t max_seq, size_t* bytes) {
  Geom g;
  const oscar_status st = validate(cfg, &g);
  if (st != OSCAR_OK) return st;
  if (!bytes || batch < 0 || max_seq < 0) return fail(OSCAR_ERR_INVALID, "bad arguments to workspace size");
  *bytes = oscar::kv8_select_ws_bytes(g, batch, max_seq);
  return OSCAR_OK;
}

oscar_status oscar_kv8_select_pages(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                    const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch,
                                    int32_t max_seq, int32_t keep_first, int32_t keep_last, int32_t n_select,
                                    int32_t* page_idx, void* workspace, size_t ws_bytes, void* stream) {
  oscar_status st = check_query(ctx, layer, q, &q_stride, q_dtype, block_table, bt_stride, seq_lens, batch);
  if (st != OSCAR_OK) return st;
  if ((st = check_max_seq(ctx, max_seq)) != OSCAR_OK) return st;
  if ((st = check_select(n_select)) != OSCAR_OK) return st;
  if (keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > n_select)
    return fail(OSCAR_ERR_INVALID, "keep_first %d and keep_last %d: neither below 0, together at most n_select (%d)", keep_first,
                keep_last, n_select);
  if (batch == 0) return OSCAR_OK;
  if (!page_idx) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  if ((st = check_workspace(workspace)) != OSCAR_OK) return st;
  const size_t need = oscar::kv8_select_ws_bytes(ctx->g, batch, max_seq);
  if (ws_bytes < need) return fail(OSCAR_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, need);
  Kv8SelectArgs a{};
  a.g = ctx->g;
  a.fmt = ctx->kv8_format;
  a.layer = layer;
  a.q = q;
  a.q_stride = q_stride;
  a.q_dtype = q_dtype;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.batch = batch;
  a.max_seq = max_seq;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.n_select = n_select;
  a.page_idx = page_idx;
  a.pool = ctx->kv8_pool;
  a.status = ctx->d_status;
  a.ws = static_cast<uint8_t*>(workspace);
  a.max_pages = max_seq / ctx->g.P;
  LaunchScope ls(ctx, "kv8_select", stream);
  const int e = oscar::launch_kv8_select(a, stream, !ctx->timing);
  ls.done(e);
  if (e) return cuda_fail(e, "page selection launch");
  if (a.max_pages > n_select) ctx->launches++;  // the scope counts one: the scores have a kernel of their own
  return OSCAR_OK;
}

oscar_status oscar_kv8_sparse_workspace_size(const oscar_config* cfg, int32_t batch, int32_t n_select, size_t* bytes) {
  Geom g;
  const oscar_status st = validate(cfg, &g);
  if (st != OSCAR_OK) return st;
  if (!bytes || batch < 0) return fail(OSCAR_ERR_INVALID, "bad arguments to workspace size");
  const oscar_status ok = check_select(n_select);
  if (ok != OSCAR_OK) return ok;
  *bytes = oscar::kv8_plan(g, batch, n_select).total;
  return OSCAR_OK;
}

oscar_status oscar_kv8_sparse_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                          void* out, int32_t out_dtype, const int32_t* page_idx, int32_t n_select,
                                          const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                          const int32_t* req_slot, int32_t batch, void* workspace, size_t ws_bytes,
                                          void* stream) {
  oscar_status st = check_query(ctx, layer, q, &q_stride, q_dtype, block_table, bt_stride, seq_lens, batch);
  if (st != OSCAR_OK) return st;
  if ((st = check_select(n_select)) != OSCAR_OK || batch == 0) return st;
  if (!page_idx) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  return attend(ctx, layer, q, q_stride, q_dtype, out, out_dtype, page_idx, n_select, block_table, bt_stride, seq_lens,
                req_slot, batch, 0, workspace, ws_bytes, stream);
}

// ---------------------------------------------------------------- page management
oscar_status oscar_kv8_fork(oscar_ctx* ctx, const int32_t* src_bt, int32_t n, int32_t src_slot, const int32_t* dst_slots,
                            int32_t n_dst, int32_t* dst_bt, void* stream) {
  if (!ctx) return fail(OSCAR_ERR_INVALID, "context is null");
  const Geom& g = ctx->g;
  if (n < 0 || (long long)n > (long long)g.max_pages_per_req * g.P) return fail(OSCAR_ERR_INVALID, "prefix length %d out of range", n);
  const int full = n / g.P, rows = n % g.P;
  if (n_dst < 0 || n_dst > g.max_req) return fail(OSCAR_ERR_INVALID, "n_dst %d out of [0, %d]", n_dst, g.max_req);
  if ((full > 0 && !src_bt) || (n_dst > 0 && (!dst_slots || !dst_bt))) return fail(OSCAR_ERR_INVALID, "bad arguments to oscar_kv8_fork");
  if (src_slot < 0 || src_slot >= g.max_req) return fail(OSCAR_ERR_INVALID, "bad source slot %d", src_slot);
  if (n_dst == 0) return OSCAR_OK;
  try {
    std::vector<char> seen(g.max_req, 0);
    seen[src_slot] = 1;
    for (int i = 0; i < n_dst; ++i) {
      if (dst_slots[i] < 0 || dst_slots[i] >= g.max_req || seen[dst_slots[i]])
        return fail(OSCAR_ERR_INVALID, "destination slot %d is out of range, the source or given twice", dst_slots[i]);
      seen[dst_slots[i]] = 1;
    }
  } catch (const std::bad_alloc&) {
    return fail(OSCAR_ERR_OOM, "host allocation failed");
  }
  if (ctx->kv8_pool) {
    oscar_status st = check_device(ctx);
    if (st == OSCAR_OK) st = check_not_capturing(stream, "oscar_kv8_fork");
    if (st != OSCAR_OK) return st;
  }
  {
    std::lock_guard<std::mutex> lk(ctx->mu);
    for (int i = 0; i < full; ++i)
      if (src_bt[i] < 0 || src_bt[i] >= g.num_pages || ctx->refcount[src_bt[i]] <= 0)
        return fail(OSCAR_ERR_INVALID, "source page %d is not mapped to an allocated page", i);
    for (int i = 0; i < full; ++i) ctx->refcount[src_bt[i]] += n_dst;
  }
  int err = 0;
  if (ctx->kv8_pool && rows > 0) {
    for (int at = 0; at < n_dst && !err; at += oscar::kMostPairs) {
      LaunchScope ls(ctx, "kv8_fork", stream);
      err = oscar::launch_kv8_fork_tail(g, ctx->kv8_tail, src_slot, dst_slots + at, std::min(n_dst - at, oscar::kMostPairs), rows,
                                        stream);
      ls.done(err);
    }
  }
  if (err) {  // nothing was forked
    std::lock_guard<std::mutex> lk(ctx->mu);
    for (int i = 0; i < full; ++i) ctx->refcount[src_bt[i]] -= n_dst;
    return cuda_fail(err, "fork launch");
  }
  for (int k = 0; k < n_dst; ++k) {
    int32_t* row = dst_bt + (size_t)k * g.max_pages_per_req;
    for (int i = 0; i < g.max_pages_per_req; ++i) row[i] = i < full ? src_bt[i] : -1;
  }
  return OSCAR_OK;
}

oscar_status oscar_compact_pages(oscar_ctx* ctx, int32_t* block_table, int32_t rows, int32_t bt_stride, int32_t* out_map,
                                 int32_t* out_live, void* stream) {
  if (!ctx || !out_map || !out_live) return fail(OSCAR_ERR_INVALID, "bad arguments to oscar_compact_pages");
  if (rows < 0 || (rows > 0 && (!block_table || bt_stride < 1))) return fail(OSCAR_ERR_INVALID, "bad block table");
  const Geom& g = ctx->g;
  const bool device = ctx->pool || ctx->kv8_pool;
  if (rows > 0 && !device) return fail(OSCAR_ERR_INVALID, "context was created without device buffers");
  if (device) {
    oscar_status st = check_device(ctx);
    if (st == OSCAR_OK) st = check_not_capturing(stream, "oscar_compact_pages");
    if (st != OSCAR_OK) return st;
  }
  try {
    std::lock_guard<std::mutex> lk(ctx->mu);
    const int live = g.num_pages - (int)ctx->free_stack.size();
    std::vector<int32_t> src, dst;
    for (int i = 0; i < g.num_pages; ++i) {
      const bool used = ctx->refcount[i] > 0;
      if (used && i >= live) src.push_back(i);
      if (!used && i < live) dst.push_back(i);
    }
    std::vector<int32_t> stack;
    stack.reserve(g.num_pages);
    for (int i = g.num_pages - 1; i >= live; --i) stack.push_back(i);  // lowest id first
    // Every copy before any table entry changes, and the entries back to the old ids (dst is as ascending as src) when a later
    // launch fails: the old pages still hold, and the allocator has not changed.
    const int moves = (int)src.size();
    auto run = [&](int pass, const int* from, const int* to, int n) {
      LaunchScope ls(ctx, pass < 2 ? "copy_pages" : "remap_table", stream);
      const int e = pass == 0   ? oscar::launch_copy_pages(ctx->pool, g.L, g.num_pages, g.Hkv * g.block_bytes(), from, to, n, stream)
                    : pass == 1 ? oscar::launch_copy_pages(ctx->kv8_pool, g.L, g.num_pages, oscar::kv8_geom(g).page_bytes(), from, to, n, stream)
                                : oscar::launch_remap_table(block_table, rows, bt_stride, from, to, n, stream);
      ls.done(e);
      return e;
    };
    for (int pass = 0; pass < 3 && device; ++pass) {
      if (pass == 0 ? !ctx->pool : pass == 1 ? !ctx->kv8_pool : rows == 0) continue;
      for (int at = 0; at < moves; at += oscar::kMostPairs) {
        const int e = run(pass, src.data() + at, dst.data() + at, std::min(moves - at, oscar::kMostPairs));
        if (!e) continue;
        for (int back = 0; pass == 2 && back < at; back += oscar::kMostPairs)
          (void)run(2, dst.data() + back, src.data() + back, oscar::kMostPairs);
        return cuda_fail(e, "page move launch");
      }
    }
    for (int i = 0; i < g.num_pages; ++i) out_map[i] = ctx->refcount[i] > 0 ? i : -1;
    for (size_t i = 0; i < src.size(); ++i) {
      out_map[src[i]] = dst[i];
      ctx->refcount[dst[i]] = ctx->refcount[src[i]];
      ctx->refcount[src[i]] = 0;
    }
    ctx->free_stack.swap(stack);
    *out_live = live;
  } catch (const std::bad_alloc&) {
    return fail(OSCAR_ERR_OOM, "host allocation failed");
  }
  return OSCAR_OK;
}

}  // extern "C"
