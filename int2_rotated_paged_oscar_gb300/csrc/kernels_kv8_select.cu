// Page selection for sparse decode over the 8-bit cache.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kScoreThreads = 256;
constexpr int kSelThreads = 1024;
using Key = unsigned long long;

// One warp per page: U = scale * sum_c (a_c hi_c - b_c lo_c) in float64.
template <int D, int FMT>
__global__ void __launch_bounds__(kScoreThreads) kv8_score_kernel(Kv8SelectArgs a) {
  __shared__ double wa[D], wb[D];
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const int G = g.gq();
  const int n = a.seq_lens[b];
  if (n < 0 || n > a.max_seq) return;
  const int pages = n / g.P;
  if (pages <= a.n_select) return;
  for (int c = tid; c < D; c += kScoreThreads) {
    double x = 0, y = 0;
    for (int hh = 0; hh < G; ++hh) {
      const double q = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)(h * G + hh) * D + c, a.q_dtype);
      x += q > 0 ? q : 0;
      y += q < 0 ? -q : 0;
    }
    wa[c] = x;
    wb[c] = y;
  }
  __syncthreads();
  const int p = blockIdx.x * (kScoreThreads / 32) + (tid >> 5);
  if (p >= pages) return;
  Key key = 0;
  if (p < a.keep_first || p >= pages - a.keep_last) {
    key = ~0ull;
  } else {
    const int pid = p < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + p] : -1;
    if (pid < 0 || pid >= g.num_pages) {
      if (lane == 0) flag_error(a.status, kDevBadPage);
    } else {
      const uint8_t* block = a.pool + ((size_t)a.layer * g.num_pages + pid) * kg.page_bytes() + (size_t)h * kg.block_bytes();
      double u = 0;
      for (int c = lane; c < D; c += 32)
        u += wa[c] * kv8_value<FMT>(block[kg.hi_off() + c]) - wb[c] * kv8_value<FMT>(block[kg.lo_off() + c]);
      for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
      u = u * reinterpret_cast<const float*>(block + kg.scale_off())[0] + 0.0;
      const Key bits = (Key)__double_as_longlong(u);
      key = u != u ? 0 : (bits >> 63) ? ~bits : (bits | 0x8000000000000000ull);
    }
  }
  if (lane == 0) reinterpret_cast<Key*>(a.ws)[((size_t)b * g.Hkv + h) * a.max_pages + p] = key;
}

// The n_select largest keys of a (request, kv head), lowest index first among equal ones, in
// ascending order of the index: the n_select-th largest key digit by digit, then one pass.
__global__ void __launch_bounds__(kSelThreads) kv8_pick_kernel(Kv8SelectArgs a) {
  __shared__ int hist[256], warp_sum[32];
  __shared__ Key s_prefix;
  __shared__ int s_need;
  const Geom& g = a.g;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* out = a.page_idx + ((size_t)b * g.Hkv + h) * a.n_select;
  const int n = a.seq_lens[b];
  const bool ok = n >= 0 && n <= a.max_seq;
  if (!ok && tid == 0) flag_error(a.status, kDevBadLen);
  const int pages = ok ? n / g.P : 0;
  if (pages <= a.n_select) {
    for (int i = tid; i < a.n_select; i += kSelThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const Key* keys = reinterpret_cast<const Key*>(a.ws) + ((size_t)b * g.Hkv + h) * a.max_pages;
  if (tid == 0) {
    s_prefix = 0;
    s_need = a.n_select;
  }
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const Key prefix = s_prefix;
    for (int i = tid; i < pages; i += kSelThreads) {
      const Key k = keys[i];
      if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, d = 255;
      while (d > 0 && hist[d] < need) need -= hist[d--];
      s_need = need;
      s_prefix = prefix | ((Key)d << shift);
    }
    __syncthreads();
  }
  const Key limit = s_prefix;
  const int need = s_need;  // how many of those equal to the limit
  int taken = 0, equal = 0;
  for (int i0 = 0; i0 < pages; i0 += kSelThreads) {
    const int i = i0 + tid;
    const Key k = i < pages ? keys[i] : 0;
    const bool eq = i < pages && k == limit;
    // exclusive counts over the block: equal ones first, then those that are taken
    auto scan = [&](bool f, int* total) {
      const unsigned m = __ballot_sync(0xffffffffu, f);
      __syncthreads();
      if (lane == 0) warp_sum[warp] = __popc(m);
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
      }
      *total = all;
      return before + __popc(m & ((1u << lane) - 1));
    };
    int total;
    const int rank = equal + scan(eq, &total);
    equal += total;
    const bool take = i < pages && (k > limit || (eq && rank < need));
    const int at = taken + scan(take, &total);
    if (take) out[at] = i;
    taken += total;
  }
}

}  // namespace

size_t kv8_select_ws_bytes(const Geom& g, int batch, int max_seq) {
  return (size_t)batch * g.Hkv * (max_seq / g.P) * sizeof(Key);
}

int launch_kv8_select(const Kv8SelectArgs& a, void* stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.max_pages > a.n_select) {
    const dim3 grid((a.max_pages + kScoreThreads / 32 - 1) / (kScoreThreads / 32), a.g.Hkv, a.batch);
    if (a.g.D == 128) {
      if (a.fmt == kKv8Int8) kv8_score_kernel<128, kKv8Int8><<<grid, kScoreThreads, 0, s>>>(a);
      else kv8_score_kernel<128, kKv8E4m3><<<grid, kScoreThreads, 0, s>>>(a);
    } else {
      if (a.fmt == kKv8Int8) kv8_score_kernel<64, kKv8Int8><<<grid, kScoreThreads, 0, s>>>(a);
      else kv8_score_kernel<64, kKv8E4m3><<<grid, kScoreThreads, 0, s>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
  }
  kv8_pick_kernel<<<dim3(a.g.Hkv, a.batch), kSelThreads, 0, s>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace oscar
