// 8-bit cache write and append.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;

struct Item {
  int b, page;           // request, logical page completed by this item (-1: none)
  int tail0, tail1;      // tokens copied into the tail
  int start, row0;       // first new token and its input row
};

// The work of one (item, kv head, K|V) CTA.  A request whose chunk completes c pages has
// max(c, 1) items: item j quantises its j-th page, item 0 also stores the rows of the page
// that stays incomplete, after it has read the rows of the old one from the same tail.
__device__ bool find_item(const Kv8WriteArgs& a, int item, Item* out, bool* bad) {
  const Geom& g = a.g;
  const int lane = threadIdx.x & 31;
  const long long cap = (long long)g.max_pages_per_req * g.P;
  int base = 0;
  *bad = false;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + lane;
    int cnt = 0, start = 0, len = 0, row0 = 0;
    if (b < a.batch) {
      start = a.start_pos[b];
      row0 = a.cu_seqlens ? a.cu_seqlens[b] : b;
      const long long l = a.cu_seqlens ? (long long)a.cu_seqlens[b + 1] - row0 : 1;
      const int slot = a.req_slot[b];
      const bool ok = start >= 0 && row0 >= 0 && l >= 0 && row0 + l <= a.total_tokens && start + l <= cap;
      if (!ok) flag_error(a.status, kDevBadLen);
      if (slot < 0 || slot >= g.max_req) flag_error(a.status, kDevBadSlot);
      if (ok && slot >= 0 && slot < g.max_req && l > 0) {
        len = (int)l;
        cnt = max((start + len) / g.P - start / g.P, 1);
      }
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (item < base + total) {
      const unsigned hit = __ballot_sync(0xffffffffu, base + incl > item);
      const int l = __ffs(hit) - 1;
      start = __shfl_sync(0xffffffffu, start, l);
      len = __shfl_sync(0xffffffffu, len, l);
      row0 = __shfl_sync(0xffffffffu, row0, l);
      const int j = item - base - __shfl_sync(0xffffffffu, incl - cnt, l);
      const int first = start / g.P, last = (start + len) / g.P;
      out->b = b0 + l;
      out->page = first + j < last ? first + j : -1;
      out->start = start;
      out->row0 = row0;
      // an append keeps its row in the tail even when it completes the page
      out->tail0 = j == 0 ? (a.cu_seqlens ? max(last * g.P, start) : start) : 0;
      out->tail1 = j == 0 ? start + len : 0;
      return true;
    }
    base += total;
  }
  return false;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(Kv8WriteArgs a) {
  __shared__ Item s_item;
  __shared__ int s_have;
  __shared__ int s_max;
  __shared__ uint32_t s_lo[D], s_hi[D];
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int tid = threadIdx.x, h = blockIdx.y, kv = blockIdx.z;
  if (tid < 32) {
    Item it;
    bool bad;
    const bool have = find_item(a, blockIdx.x, &it, &bad);
    if (tid == 0) {
      s_item = it;
      s_have = have;
      s_max = 0;
    }
  }
  for (int i = tid; i < D; i += kThreads) {
    s_lo[i] = 255u;
    s_hi[i] = 0u;
  }
  __syncthreads();
  if (!s_have) return;
  const Item it = s_item;
  const void* src = kv ? a.V : a.K;
  const long long stride = kv ? a.v_stride : a.k_stride;
  uint16_t* tail = a.tail + ((size_t)a.layer * g.max_req + a.req_slot[it.b]) * kv8_tail_req_elems(g) +
                   ((size_t)h * 2 + kv) * g.P * D;
  // BF16 bits of channel ch of token t: an input row, or the tail row of an older token
  auto value = [&](int t, int ch) -> uint32_t {
    if (t < it.start) return tail[(size_t)(t % g.P) * D + ch];
    const size_t i = (size_t)(it.row0 + (t - it.start)) * stride + (size_t)h * D + ch;
    if (a.dtype == kDtypeBF16) return static_cast<const uint16_t*>(src)[i];
    return __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<const float*>(src)[i]));
  };
  if (it.page >= 0) {
    const int lp = it.page;
    const int pid = lp < a.bt_stride ? a.block_table[(size_t)it.b * a.bt_stride + lp] : -1;
    const bool ok = pid >= 0 && pid < g.num_pages;
    if (!ok && tid == 0) flag_error(a.status, kDevBadPage);
    int big = 0;
    bool odd = false;
    for (int i = tid; i < g.P * D; i += kThreads) {
      const int m = value(lp * g.P + i / D, i % D) & 0x7fff;
      if (m >= 0x7f80) odd = true;
      else big = max(big, m);
    }
    if (odd) flag_error(a.status, kDevBadValue);
    atomicMax(&s_max, big);
    __syncthreads();
    const float m = __uint_as_float((uint32_t)s_max << 16);
    const bool some = m >= kKv8Smallest;
    uint8_t* block = a.pool + ((size_t)a.layer * g.num_pages + (ok ? pid : 0)) * kg.page_bytes() + (size_t)h * kg.block_bytes();
    for (int i = tid; i < g.P * D; i += kThreads) {
      const int r = i / D, ch = i % D;
      const float x = __uint_as_float(value(lp * g.P + r, ch) << 16);
      const uint32_t code = some ? kv8_encode<FMT>(x, m) : (FMT == kKv8Int8 ? 128u : 0u);
      if (ok) block[(kv ? kg.v_off() : 0) + (kv ? kv8_place<D, true>(r, ch) : kv8_place<D, false>(r, ch))] = (uint8_t)code;
      if (!kv) {
        atomicMin(&s_lo[ch], kv8_key<FMT>(code));
        atomicMax(&s_hi[ch], kv8_key<FMT>(code));
      }
    }
    __syncthreads();
    if (ok && tid == 0)
      reinterpret_cast<float*>(block + kg.scale_off())[kv] = some ? __fdiv_rn(m, FMT == kKv8Int8 ? 127.f : 448.f) : 0.f;
    if (ok && !kv)
      for (int i = tid; i < D; i += kThreads) {
        block[kg.lo_off() + i] = (uint8_t)kv8_unkey<FMT>(s_lo[i]);
        block[kg.hi_off() + i] = (uint8_t)kv8_unkey<FMT>(s_hi[i]);
      }
    __syncthreads();
  }
  for (int i = tid; i < (it.tail1 - it.tail0) * D; i += kThreads) {
    const int t = it.tail0 + i / D;
    tail[(size_t)(t % g.P) * D + i % D] = (uint16_t)value(t, i % D);
  }
}

}  // namespace

int launch_kv8_write(const Kv8WriteArgs& a, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int items = a.cu_seqlens ? a.total_tokens / a.g.P + a.batch : a.batch;
  const dim3 grid(items, a.g.Hkv, 2);
  if (a.g.D == 128) {
    if (a.fmt == kKv8Int8) kv8_write_kernel<128, kKv8Int8><<<grid, kThreads, 0, s>>>(a);
    else kv8_write_kernel<128, kKv8E4m3><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (a.fmt == kKv8Int8) kv8_write_kernel<64, kKv8Int8><<<grid, kThreads, 0, s>>>(a);
    else kv8_write_kernel<64, kKv8E4m3><<<grid, kThreads, 0, s>>>(a);
  }
  return (int)cudaGetLastError();
}

}  // namespace oscar
