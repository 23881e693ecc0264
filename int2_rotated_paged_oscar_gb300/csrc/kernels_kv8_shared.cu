// Decode attention of requests that share a prefix: the shared pages of a group, apart from the requests' own parts.
#include "kv8.cuh"

namespace oscar {
namespace {

// A warp per (split, query head, request): tokens one after another, channels over the lanes.
template <int D, int FMT>
__global__ void __launch_bounds__(32) prefix_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  constexpr int C = D / 32;
  const Geom& g = a.g;
  const int split = blockIdx.x, head = blockIdx.y, b = blockIdx.z, lane = threadIdx.x, ch = lane * C, h = head / g.gq();
  pdl_wait();
  pdl_launch_dependents();
  const int shared = kv8_shared_of(a, b), n = a.seq_lens[b];
  if (n <= 0 || !kv8_own_sound(a, n, shared)) return;
  const int per = a.groups.units_per_split * (kPrefixUnit / g.P);
  const int e0 = split * per, e1 = min(e0 + per, shared);
  if (e0 >= e1) return;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
  float q[C], o[C], m = -INFINITY, l = 0.f;
  for (int i = 0; i < C; ++i) {
    q[i] = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)head * D + ch + i, a.q_dtype);
    o[i] = 0.f;
  }
  const float f = 1.4426950408889634f / sqrtf((float)D);
  for (int e = e0; e < e1; ++e) {
    const int pid = e < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + e] : -1;
    if (pid < 0 || pid >= g.num_pages) {
      if (lane == 0) flag_error(a.status, kDevBadPage);
      continue;
    }
    const uint8_t* block = layer + (size_t)pid * kg.page_bytes();
    const float2 scale = *reinterpret_cast<const float2*>(block + kg.scale_off());
    for (int t = 0; t < g.P; ++t) {
      const uint8_t *k = block + kv8_place<D, false>(t, ch), *v = block + kg.v_off() + kv8_place<D, true>(t, ch);
      float c = 0.f;
      for (int i = 0; i < C; ++i) c = fmaf(kv8_value<FMT>(k[i]), q[i], c);
      for (int x = 16; x; x >>= 1) c += __shfl_xor_sync(0xffffffffu, c, x);
      const float s = c * (scale.x * f), top = fmaxf(m, s), alpha = ex2(m - top), p = ex2(s - top);
      l = fmaf(l, alpha, p);
      for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], alpha, p * (kv8_value<FMT>(v[i]) * scale.y));
      m = top;
    }
  }
  float* pp = a.part + (((size_t)b * g.Hq + head) * a.wl.max_splits + split) * (D + 4);
  if (lane == 0) {
    pp[0] = l == l ? m : INFINITY;
    pp[1] = l;
  }
  for (int i = 0; i < C; ++i) pp[4 + ch + i] = o[i];
}

}  // namespace

Kv8DecodeWs kv8_shared_plan(const Geom& g, int batch, int n_groups, int max_shared, int max_own, Kv8Groups* groups, int* own_splits) {
  Kv8DecodeWs w = kv8_plan(g, batch, max_own / g.P);
  *own_splits = w.max_splits;
  // The split that takes the fewest rounds of (its units + 3, a CTA's start and end).
  const long long tiles = ((long long)max_shared * g.P + kPrefixUnit - 1) / kPrefixUnit;
  const long long rows = (long long)batch * g.gq(), row_tiles = rows / 128 > n_groups ? rows / 128 : n_groups;
  const long long pairs = row_tiles * g.Hkv > 0 ? row_tiles * g.Hkv : 1;
  long long best = 1, cost = -1;
  for (long long per = 1; per <= 256 && per <= (tiles > 0 ? tiles : 1); ++per) {
    const long long ctas = pairs * ((tiles + per - 1) / per), c = ((ctas + 151) / 152) * (per + 3);
    if (cost < 0 || c < cost) best = per, cost = c;
  }
  groups->n = n_groups;
  groups->max_shared = max_shared;
  groups->max_own = max_own;
  groups->units_per_split = (int)best;
  groups->max_tiles = (int)(rows / 128 + n_groups);
  groups->slots = tiles > 0 ? (int)((tiles + best - 1) / best) : 1;
  w.max_splits += groups->slots;
  w.total = (size_t)batch * g.Hq * w.max_splits * (g.D + 4) * sizeof(float);
  return w;
}

int launch_kv8_shared_prefix(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(a.groups.slots, a.g.Hq, a.batch);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(32), 0, s, pdl, a); };
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? go(prefix_kernel<128, kKv8Int8>) : go(prefix_kernel<128, kKv8E4m3>);
  return a.fmt == kKv8Int8 ? go(prefix_kernel<64, kKv8Int8>) : go(prefix_kernel<64, kKv8E4m3>);
}

}  // namespace oscar
