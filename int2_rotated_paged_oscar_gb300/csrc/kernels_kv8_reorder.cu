// Beams' states after a selection: new beam j of an item continues beam parents[j].
//
// A beam's state is its block-table row, its length, and its BF16 tail rows in its request slot.  The first child of a beam
// keeps the slot, so its tail does not move; each further child takes the slot of a beam without a child, and n mod P rows are
// copied there in every layer.  Slots that are read are never written, so the copies need no order among themselves.
// Bound by memory: layers x kv heads x 2 x (n mod P) rows of 2 d bytes, read and written once per copied child.  A CTA
// takes runs (layer, kv head, K or V) as one range of 16-byte vectors, eight of a thread under way: 36 layers of 16 x 8 beams
// 88 us, 22 us for 4 x 4 (147 and 23 with one run a CTA at a time).
#include "beam_internal.h"
#include "common.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256, kAhead = 8;  // loads of a thread that are under way

__global__ void __launch_bounds__(kThreads) kv8_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int s_par[kMaxBeams];
  __shared__ int s_used[kMaxBeams];
  const Geom& g = a.g;
  const int tid = threadIdx.x, K = a.beams, child = blockIdx.y % K, row0 = blockIdx.y - child, j = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  if (tid < K) {
    int p = a.parents[row0 + tid];
    if (p < -1 || p >= K) {
      if (blockIdx.x == 0 && tid == child) flag_error(a.status, kDevBadSlot);
      p = -1;
    }
    s_par[tid] = p;
    s_used[tid] = 0;
  }
  __syncthreads();
  if (tid < K && s_par[tid] >= 0) s_used[s_par[tid]] = 1;
  __syncthreads();
  const int p = s_par[child];
  // children before this one that are their parents' first, and whether it is one itself
  int firsts = 0;
  bool first = p >= 0;
  for (int t = 0; t < child; ++t) {
    bool f = s_par[t] >= 0;
    for (int u = 0; u < t; ++u) f &= s_par[u] != s_par[t];
    firsts += f;
    first &= s_par[t] != p;
  }
  int from = p;                     // the beam whose slot it takes
  if (!first) {
    int skip = child - firsts;
    for (from = 0; from < K; ++from)
      if (!s_used[from] && skip-- == 0) break;
  }
  const int slot = a.req_slot[row0 + from];
  const int n = p >= 0 ? a.seq_lens[row0 + p] : 0;
  if (blockIdx.x == 0) {
    const int* src = a.block_table + (size_t)(row0 + max(p, 0)) * a.bt_stride;
    int* dst = a.new_block_table + (size_t)j * a.bt_stride;
    for (int i = tid; i < a.bt_stride; i += kThreads) dst[i] = p >= 0 ? src[i] : -1;
    if (tid == 0) {
      a.new_seq_lens[j] = n;
      a.new_req_slot[j] = slot;
      // (a state is checked wherever it goes: a parent's first child hands its length and slot on without a copy)
      const bool bad_slot = slot < 0 || slot >= g.max_req, bad_len = n < 0 || (long long)n > (long long)g.max_pages_per_req * g.P;
      if (bad_slot || bad_len) flag_error(a.status, (bad_slot ? kDevBadSlot : 0) | (bad_len ? kDevBadLen : 0));
    }
  }
  if (first || p < 0) return;
  const int src_slot = a.req_slot[row0 + p];
  if (src_slot < 0 || src_slot >= g.max_req || slot < 0 || slot >= g.max_req) return;
  if (n < 0 || (long long)n > (long long)g.max_pages_per_req * g.P) return;
  const int vecs = (n % g.P) * g.D / 8;                 // 16-byte vectors of the K or V rows of one kv head
  if (vecs == 0) return;
  const size_t half = (size_t)g.P * g.D, region = (size_t)g.Hkv * 2 * half, layer = (size_t)g.max_req * region;
  const int parts = 2 * g.Hkv, total = g.L * parts;
  const uint16_t* src = a.tail + (size_t)src_slot * region;
  uint16_t* dst = a.tail + (size_t)slot * region;
  // this CTA's share of the (layer, kv head, K or V) runs, as one range of vectors
  const int u0 = (int)((long long)total * blockIdx.x / gridDim.x), u1 = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
  const unsigned all = (unsigned)(u1 - u0) * vecs;      // (fits: 2 Hkv L runs of at most 1024 vectors in a grid's share)
  for (unsigned i0 = tid; i0 < all; i0 += kAhead * kThreads) {
    uint4 x[kAhead];
    size_t at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const unsigned i = min(i0 + k * kThreads, all - 1), u = i / vecs;
      at[k] = (size_t)((u0 + u) / parts) * layer + (size_t)((u0 + u) % parts) * half + (size_t)(i - u * vecs) * 8;
      x[k] = __ldcs(reinterpret_cast<const uint4*>(src + at[k]));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kThreads < all) __stcs(reinterpret_cast<uint4*>(dst + at[k]), x[k]);
  }
}

}  // namespace

int launch_kv8_reorder(const ReorderArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rows = a.batch * a.beams, units = a.g.L * 2 * a.g.Hkv;
  // enough CTAs for every SM, and no more: most children keep their slot, and theirs end at once
  int x = (152 * 32 + rows - 1) / rows;
  x = x < units ? x : units;
  return launch_pdl(kv8_reorder_kernel, dim3(x, rows), dim3(kThreads), 0, s, pdl, a);
}

}  // namespace oscar
