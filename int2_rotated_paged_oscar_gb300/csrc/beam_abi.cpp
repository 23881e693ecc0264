// C ABI of the choice of beams (see include/oscar.h).
#include "beam_internal.h"
#include "kv8_checks.h"

using oscar::BeamArgs;
using oscar::check_device;
using oscar::check_workspace;
using oscar::cuda_fail;
using oscar::fail;
using oscar::LaunchScope;
using oscar::overlap;

namespace {

oscar_status check_sizes(int32_t batch, int32_t beams, int32_t vocab, int32_t n_out) {
  if (batch < 0 || beams < 1 || vocab < 1 || n_out < 1)
    return fail(OSCAR_ERR_INVALID, "batch %d, beams %d, vocab %d, n_out %d", batch, beams, vocab, n_out);
  if (batch > 65535 || beams > oscar::kMaxBeams || vocab > oscar::kMaxVocab || n_out > oscar::kMaxCandidates)
    return fail(OSCAR_ERR_UNSUPPORTED, "batch %d, beams %d, vocab %d, n_out %d: at most 65535, %d, %d, %d", batch, beams, vocab,
                n_out, oscar::kMaxBeams, oscar::kMaxVocab, oscar::kMaxCandidates);
  return OSCAR_OK;
}

}  // namespace

extern "C" {

oscar_status oscar_beam_select_workspace_size(int32_t batch, int32_t beams, int32_t vocab, int32_t n_out, size_t* bytes) {
  const oscar_status st = check_sizes(batch, beams, vocab, n_out);
  if (st != OSCAR_OK) return st;
  if (!bytes) return fail(OSCAR_ERR_INVALID, "bad arguments to workspace size");
  *bytes = oscar::beam_ws_bytes(batch, beams, vocab);
  return OSCAR_OK;
}

oscar_status oscar_beam_select(oscar_ctx* ctx, const void* logits, int64_t row_stride, int32_t dtype, const float* scores,
                               const uint8_t* finished, int32_t pad_token, int32_t batch, int32_t beams, int32_t vocab,
                               int32_t n_out, float* out_scores, int32_t* out_tokens, int32_t* out_parents, void* workspace,
                               size_t ws_bytes, void* stream) {
  if (!ctx) return fail(OSCAR_ERR_INVALID, "context is null");
  if (!ctx->d_status) return fail(OSCAR_ERR_INVALID, "context was created without device buffers");
  oscar_status st = check_device(ctx);
  if (st != OSCAR_OK) return st;
  if ((st = check_sizes(batch, beams, vocab, n_out)) != OSCAR_OK) return st;
  if (dtype != OSCAR_DTYPE_BF16 && dtype != OSCAR_DTYPE_F32) return fail(OSCAR_ERR_INVALID, "bad dtype %d of logits", dtype);
  if (row_stride == 0) row_stride = vocab;
  if (row_stride > (1LL << 40)) return fail(OSCAR_ERR_UNSUPPORTED, "row stride %lld of logits", (long long)row_stride);
  if (row_stride < vocab) return fail(OSCAR_ERR_INVALID, "row stride %lld of logits is below the vocabulary %d", (long long)row_stride, vocab);
  if (finished && (pad_token < 0 || pad_token >= vocab)) return fail(OSCAR_ERR_INVALID, "pad_token %d out of [0, %d)", pad_token, vocab);
  if (batch == 0) return OSCAR_OK;
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  const size_t elem = dtype == OSCAR_DTYPE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % elem) return fail(OSCAR_ERR_INVALID, "logits must be aligned to its elements");
  const size_t rows = (size_t)batch * beams, out = 4 * (size_t)batch * n_out, read = ((rows - 1) * row_stride + vocab) * elem;
  if ((st = check_workspace(workspace)) != OSCAR_OK) return st;
  BeamArgs a{};
  const size_t need = oscar::beam_ws_bytes(batch, beams, vocab);
  if (ws_bytes < need) return fail(OSCAR_ERR_INVALID, "workspace too small: %zu < %zu bytes", ws_bytes, need);
  // what is written, then what is read
  const struct { const void* p; size_t n; } of[] = {{out_scores, out}, {out_tokens, out}, {out_parents, out}, {workspace, need},
                                                    {scores, 4 * rows}, {finished, rows}, {logits, read}};
  for (int o = 0; o < 4; ++o)
    for (int i = o + 1; i < 7; ++i)
      if (overlap(of[o].p, of[o].n, of[i].p, of[i].n))
        return fail(OSCAR_ERR_INVALID, "the outputs and the workspace must overlap neither the inputs nor one another");
  a.logits = logits;
  a.stride = row_stride;
  a.dtype = dtype;
  a.scores = scores;
  a.finished = finished;
  a.pad_token = pad_token;
  a.batch = batch;
  a.beams = beams;
  a.vocab = vocab;
  a.n_out = n_out;
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  a.status = ctx->d_status;
  a.part = static_cast<float*>(workspace);
  const bool pdl = !ctx->timing;
  {
    LaunchScope ls(ctx, "beam_units", stream);
    const int e = oscar::launch_beam_units(a, stream, pdl);
    ls.done(e);
    if (e) return cuda_fail(e, "beam selection launch");
  }
  LaunchScope ls(ctx, "beam_pick", stream);
  const int e = oscar::launch_beam_pick(a, stream, pdl);
  ls.done(e);
  if (e) return cuda_fail(e, "beam selection launch");
  return OSCAR_OK;
}

}  // extern "C"
