// Checks of arguments that the 8-bit cache's calls share.
#pragma once
#include "kv8_internal.h"
#include "oscar_ctx.h"

namespace oscar {

constexpr int kMaxGrid = 65535;  // of the grid's second and third dimension

// The buffers were bound on one device and the kernels run on the current one.
inline oscar_status check_device(const oscar_ctx* ctx) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "current device");
  if (dev != ctx->device)
    return fail(OSCAR_ERR_INVALID, "the context's buffers are on device %d, the current device is %d", ctx->device, dev);
  return OSCAR_OK;
}

// Whether two arrays of so many bytes share one (a null array holds none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

inline oscar_status need_kv8(oscar_ctx* ctx) {
  if (!ctx) return fail(OSCAR_ERR_INVALID, "context is null");
  if (!ctx->kv8_pool) return fail(OSCAR_ERR_INVALID, "no 8-bit cache is bound to the context (oscar_kv8_bind)");
  return check_device(ctx);
}

// Rows of heads x d elements, *stride elements apart (0: adjacent), read in 16-byte vectors.
inline oscar_status check_rows(const char* name, const void* p, int64_t* stride, int heads, int d, int dtype) {
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

inline oscar_status check_batch(int32_t batch, int32_t bt_stride) {
  if (batch < 0 || bt_stride < 1) return fail(OSCAR_ERR_INVALID, "bad batch/bt_stride");
  if (batch > kMaxGrid) return fail(OSCAR_ERR_UNSUPPORTED, "batch %d exceeds %d", batch, kMaxGrid);
  return OSCAR_OK;
}

// What the two attention calls and the selection have in common.
inline oscar_status check_query(oscar_ctx* ctx, int32_t layer, const void* q, int64_t* q_stride, int32_t q_dtype,
                         const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch) {
  oscar_status st = need_kv8(ctx);
  if (st != OSCAR_OK) return st;
  if ((st = check_layer(ctx, layer)) != OSCAR_OK) return st;
  if ((st = check_batch(batch, bt_stride)) != OSCAR_OK) return st;
  if (batch == 0) return OSCAR_OK;
  if (!block_table || !seq_lens) return fail(OSCAR_ERR_INVALID, "null tensor argument");
  return check_rows("q", q, q_stride, ctx->g.Hq, ctx->g.D, q_dtype);
}

}  // namespace oscar
