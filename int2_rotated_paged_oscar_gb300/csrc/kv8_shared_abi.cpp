// C ABI of the 8-bit cache's requests that continue one prompt: attention with a shared prefix, reordering of beams
// (see include/oscar.h).
#include "beam_internal.h"
#include "kv8_checks.h"

using oscar::check_query;
using oscar::check_workspace;
using oscar::cuda_fail;
using oscar::fail;
using oscar::Geom;
using oscar::kMaxGrid;
using oscar::Kv8DecodeArgs;
using oscar::LaunchScope;
using oscar::need_kv8;
using oscar::overlap;
using oscar::ReorderArgs;
using oscar::validate;

namespace {

oscar_status check_groups(const Geom& g, int32_t n_groups, int32_t max_shared, int32_t max_own) {
  if (n_groups < 0 || max_shared < 0 || max_own < 0)
    return fail(OSCAR_ERR_INVALID, "n_groups %d, max_shared %d, max_own %d: none below 0", n_groups, max_shared, max_own);
  if (n_groups > kMaxGrid) return fail(OSCAR_ERR_UNSUPPORTED, "%d groups exceed %d", n_groups, kMaxGrid);
  if (max_shared > g.max_pages_per_req || (long long)max_own > (long long)g.max_pages_per_req * g.P)
    return fail(OSCAR_ERR_INVALID, "max_shared %d pages or max_own %d tokens exceed max_pages_per_req", max_shared, max_own);
  return OSCAR_OK;
}

}  // namespace

extern "C" {

oscar_status oscar_kv8_shared_workspace_size(const oscar_config* cfg, int32_t batch, int32_t n_groups, int32_t max_shared,
                                             int32_t max_own, size_t* bytes) {
  Geom g;
  oscar_status st = validate(cfg, &g);
  if (st != OSCAR_OK) return st;
  if (!bytes || batch < 0) return fail(OSCAR_ERR_INVALID, "bad arguments to workspace size");
  if ((st = check_groups(g, n_groups, max_shared, max_own)) != OSCAR_OK) return st;
  *bytes = oscar::kv8_shared_ws_bytes(g, batch, n_groups, max_shared, max_own);
  return OSCAR_OK;
}

oscar_status oscar_kv8_shared_decode_attn(oscar_ctx* ctx, int32_t layer, const void* q, int64_t q_stride, int32_t q_dtype,
                                          void* out, int32_t out_dtype, const int32_t* group_starts,
                                          const int32_t* shared_pages, int32_t n_groups, int32_t max_shared,
                                          const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                          const int32_t* req_slot, int32_t batch, int32_t max_own, void* workspace,
                                          size_t ws_bytes, void* stream) {
  oscar_status st = check_query(ctx, layer, q, &q_stride, q_dtype, block_table, bt_stride, seq_lens, batch);
  if (st != OSCAR_OK) return st;
  if ((st = check_groups(ctx->g, n_groups, max_shared, max_own)) != OSCAR_OK || batch == 0) return st;
  if (n_groups < 1) return fail(OSCAR_ERR_INVALID, "%d requests in no group", batch);
  if (!group_starts || !shared_pages) return fail(OSCAR_ERR_INVALID, "null tensor argument");
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
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.req_slot = req_slot;
  a.batch = batch;
  a.pool = ctx->kv8_pool;
  a.tail = ctx->kv8_tail;
  a.status = ctx->d_status;
  a.part = static_cast<float*>(workspace);
  a.wl = oscar::kv8_shared_plan(ctx->g, batch, n_groups, max_shared, max_own, &a.groups, &a.splits);
  a.groups.starts = group_starts;
  a.groups.shared = shared_pages;
  if (ws_bytes < a.wl.total) return fail(OSCAR_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, a.wl.total);
  const struct { const char* name; int (*launch)(const Kv8DecodeArgs&, void*, bool); } kernels[] = {
      {"kv8_decode", oscar::launch_kv8_decode}, {"kv8_prefix", oscar::launch_kv8_shared_prefix}, {"kv8_combine", oscar::launch_kv8_combine}};
  for (const auto& k : kernels) {
    if (k.launch == oscar::launch_kv8_shared_prefix && max_shared == 0) continue;
    LaunchScope ls(ctx, k.name, stream);
    const int e = k.launch(a, stream, !ctx->timing);
    ls.done(e);
    if (e) return cuda_fail(e, "shared-prefix decode launch");
  }
  return OSCAR_OK;
}

oscar_status oscar_kv8_reorder(oscar_ctx* ctx, const int32_t* parents, int32_t batch, int32_t beams, const int32_t* block_table,
                               int32_t bt_stride, const int32_t* seq_lens, const int32_t* req_slot, int32_t* new_block_table,
                               int32_t* new_seq_lens, int32_t* new_req_slot, void* stream) {
  oscar_status st = need_kv8(ctx);
  if (st != OSCAR_OK) return st;
  if (batch < 0 || beams < 1 || bt_stride < 1) return fail(OSCAR_ERR_INVALID, "bad batch/beams/bt_stride");
  if (beams > oscar::kMaxBeams) return fail(OSCAR_ERR_UNSUPPORTED, "%d beams: at most %d", beams, oscar::kMaxBeams);
  if ((long long)batch * beams > kMaxGrid)
    return fail(OSCAR_ERR_UNSUPPORTED, "%d x %d beams exceed %d", batch, beams, kMaxGrid);
  if (batch == 0) return OSCAR_OK;
  if (!parents || !block_table || !seq_lens || !req_slot || !new_block_table || !new_seq_lens || !new_req_slot)
    return fail(OSCAR_ERR_INVALID, "null tensor argument");
  const size_t rows = 4 * (size_t)batch * beams, table = rows * bt_stride;  // bytes
  const struct { const int32_t* p; size_t n; } of[] = {{new_block_table, table}, {new_seq_lens, rows}, {new_req_slot, rows},
                                                       {parents, rows}, {block_table, table}, {seq_lens, rows}, {req_slot, rows}};
  for (int o = 0; o < 3; ++o)
    for (int i = o + 1; i < 7; ++i)
      if (overlap(of[o].p, of[o].n, of[i].p, of[i].n))
        return fail(OSCAR_ERR_INVALID, "the new tables, lengths and slots must overlap neither the old ones nor one another");
  ReorderArgs a{};
  a.g = ctx->g;
  a.parents = parents;
  a.batch = batch;
  a.beams = beams;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.req_slot = req_slot;
  a.new_block_table = new_block_table;
  a.new_seq_lens = new_seq_lens;
  a.new_req_slot = new_req_slot;
  a.tail = ctx->kv8_tail;
  a.status = ctx->d_status;
  LaunchScope ls(ctx, "kv8_reorder", stream);
  const int e = oscar::launch_kv8_reorder(a, stream, !ctx->timing);
  ls.done(e);
  if (e) return cuda_fail(e, "reorder launch");
  return OSCAR_OK;
}

}  // extern "C"
