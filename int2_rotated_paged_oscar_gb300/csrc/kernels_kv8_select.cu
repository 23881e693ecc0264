// Page selection for sparse decode over the 8-bit cache.
//
//   U_p = scale_p sum_c (a_c hi_pc - b_c lo_pc),  a = sum_h max(q_h, 0),  b = sum_h max(-q_h, 0)
//
// over the heads h that share a kv head, and of the pages the n_select largest, equal ones by the lower
// index.  It reads 2 d + 4 bytes per page and kv head, 1 / P of what dense attention reads, so latency
// decides: a score kernel over all pages and a pick kernel per (request, kv head).
//
// The order is float64's, the scores are float32's.  A float32 score is off by at most
//   E_p = 2^-18 M scale_p sum_c (a_c + b_c),   M the largest code:
// its terms add up to at most E_p 2^18, and it takes fewer than 64 roundings of half a step (2^-24) each:
// 7 in a sum over 8 heads, one in a product, 3 + 32 in the sum of a lane and of its page, one in the scale.
// With E the largest E_p and t the n-th largest float32 score, the n-th largest exact score lies within E of
// t; so a page above t + 2 E is in, one below t - 2 E is out, and only the ones between, mostly the n-th
// alone, are scored again in float64 and ranked.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kPagesPerCta = 64;   // 8 lanes a page, 16 pages at a time
constexpr int kPickThreads = 512;
constexpr int kSmemKeys = 8192;    // pages whose keys the pick kernel holds in shared memory
constexpr int kSerialBand = 64;    // band of pages scored again that is ranked within shared memory tiles of this size
using Key = unsigned long long;

// Workspace: float32 keys [batch][Hkv][max_pages], float64 keys of the band (same count), its page indexes,
// and the largest E_p of each score CTA [batch][Hkv][chunks].
struct SelectWs {
  size_t keys, band, index, bound, total;
  int chunks;
};
__host__ __device__ inline SelectWs select_ws(int Hkv, int batch, int max_pages) {
  SelectWs w;
  const size_t n = (size_t)batch * Hkv * max_pages;
  w.chunks = (max_pages + kPagesPerCta - 1) / kPagesPerCta;
  w.band = 0;
  w.keys = n * sizeof(Key);
  w.index = w.keys + n * sizeof(uint32_t);
  w.bound = w.index + n * sizeof(int);
  w.total = w.bound + (size_t)batch * Hkv * w.chunks * sizeof(float);
  return w;
}

// Order-preserving unsigned keys of floating-point numbers (NaN first, -0 as +0) and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 0u : (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ double value_of(uint32_t k) {
  return (double)__uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ Key key_of(double x) {
  const Key u = (Key)__double_as_longlong(x + 0.0);
  return x != x ? 0ull : (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ int page_id(const Kv8SelectArgs& a, int b, int p) {
  const int pid = p < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + p] : -1;
  return pid < a.g.num_pages ? pid : -1;
}

__device__ __forceinline__ bool kept(const Kv8SelectArgs& a, int p, int pages) {
  return p < a.keep_first || p >= pages - a.keep_last;
}

// ------------------------------------------------------------------ scores
template <int D, int FMT>
__global__ void __launch_bounds__(kScoreThreads) kv8_score_kernel(const __grid_constant__ Kv8SelectArgs a) {
  constexpr int C = D / 8;                 // channels of a lane
  __shared__ float s_bound[kScoreThreads / 32];
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, sub = lane & 7;
  const int G = g.gq();
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  if (n < 0 || n > a.max_seq) return;
  const int pages = n / g.P, p0 = blockIdx.x * kPagesPerCta;
  if (pages <= a.n_select || p0 >= pages) return;
  float wa[C], wb[C];
#pragma unroll
  for (int c = 0; c < C; ++c) wa[c] = wb[c] = 0.f;
  for (int hh = 0; hh < G; ++hh) {
    const size_t at = (size_t)b * a.q_stride + (size_t)(h * G + hh) * D + sub * C;
#pragma unroll
    for (int c = 0; c < C; c += 8) {
      float x[8];
      if (a.q_dtype == kDtypeBF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at + c);
        x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z), x[5] = bf16_hi(u.z), x[6] = bf16_lo(u.w), x[7] = bf16_hi(u.w);
      } else {
        const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + c);
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + c + 4);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // (not fmaxf: a NaN has to stay one)
        wa[c + i] += x[i] < 0.f ? 0.f : x[i];
        wb[c + i] += x[i] > 0.f ? 0.f : -x[i];
      }
    }
  }
  float mass = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) mass += wa[c] + wb[c];
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  mass *= (FMT == kKv8Int8 ? 127.f : 448.f) * 0x1p-18f;
  uint32_t* keys = reinterpret_cast<uint32_t*>(a.ws + select_ws(g.Hkv, a.batch, a.max_pages).keys) +
                   ((size_t)b * g.Hkv + h) * a.max_pages;
  const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
  float bound = 0.f;
#pragma unroll
  for (int it = 0; it < kPagesPerCta / (kScoreThreads / 8); ++it) {
    const int p = p0 + it * (kScoreThreads / 8) + (tid >> 3);
    int pid = -1;
    bool scored = false;
    if (p < pages && !kept(a, p, pages)) {
      pid = page_id(a, b, p);
      scored = pid >= 0;
      if (!scored && sub == 0) flag_error(a.status, kDevBadPage);
    }
    float u = 0.f, scale = 0.f;
    if (scored) {
      const uint8_t* block = layer + (size_t)pid * kg.page_bytes();
      scale = *reinterpret_cast<const float*>(block + kg.scale_off());
      uint32_t lo[C / 4], hi[C / 4];
      if constexpr (C == 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(block + kg.lo_off() + sub * C);
        const uint4 y = *reinterpret_cast<const uint4*>(block + kg.hi_off() + sub * C);
        lo[0] = x.x, lo[1] = x.y, lo[2] = x.z, lo[3] = x.w;
        hi[0] = y.x, hi[1] = y.y, hi[2] = y.z, hi[3] = y.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(block + kg.lo_off() + sub * C);
        const uint2 y = *reinterpret_cast<const uint2*>(block + kg.hi_off() + sub * C);
        lo[0] = x.x, lo[1] = x.y;
        hi[0] = y.x, hi[1] = y.y;
      }
#pragma unroll
      for (int w = 0; w < C / 4; ++w) {
        const uint32_t l2[2] = {kv8_pair<FMT, 0>(lo[w]), kv8_pair<FMT, 1>(lo[w])};
        const uint32_t h2[2] = {kv8_pair<FMT, 0>(hi[w]), kv8_pair<FMT, 1>(hi[w])};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&l2[i]));
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h2[i]));
          const int c = 4 * w + 2 * i;
          u = fmaf(wa[c], y.x, u);
          u = fmaf(-wb[c], x.x, u);
          u = fmaf(wa[c + 1], y.y, u);
          u = fmaf(-wb[c + 1], x.y, u);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    if (p < pages && sub == 0) keys[p] = scored ? key_of(u * scale) : 0u;
    if (scored) {
      const float e = mass * scale + 0x1p-140f;  // (and the roundings among the subnormal numbers)
      // no finite bound, or a score that overflowed: every page is scored again
      bound = (e <= 3e38f && fabsf(u * scale) <= 3e38f) ? fmaxf(bound, e) : INFINITY;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) bound = warp_max_xor(bound, o);
  if (lane == 0) s_bound[tid >> 5] = bound;
  __syncthreads();
  if (tid == 0) {
    const SelectWs w = select_ws(g.Hkv, a.batch, a.max_pages);
    float m = 0.f;
    for (int i = 0; i < kScoreThreads / 32; ++i) m = fmaxf(m, s_bound[i]);
    reinterpret_cast<float*>(a.ws + w.bound)[((size_t)b * g.Hkv + h) * w.chunks + blockIdx.x] = m;
  }
}

// ------------------------------------------------------------------ pick
// Exclusive count of f over the block's lower threads, and the block's total.  sums: one int per warp.
__device__ __forceinline__ int block_rank(bool f, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned m = __ballot_sync(0xffffffffu, f);
  if (lane == 0) sums[warp] = __popc(m);
  __syncthreads();
  const int v = lane < kPickThreads / 32 ? sums[lane] : 0;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  *total = __shfl_sync(0xffffffffu, incl, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, incl, warp - 1) : 0;
  __syncthreads();
  return before + __popc(m & ((1u << lane) - 1));
}

template <int D, int FMT>
__global__ void __launch_bounds__(kPickThreads) kv8_pick_kernel(const __grid_constant__ Kv8SelectArgs a) {
  __shared__ uint32_t s_keys[kSmemKeys];
  __shared__ int hist[256], sums[kPickThreads / 32];
  __shared__ uint32_t s_lo[kPickThreads / 32], s_hi[kPickThreads / 32], s_prefix;
  __shared__ float s_e[kPickThreads / 32];
  __shared__ int s_need, s_band, s_above;
  __shared__ double wa[D], wb[D];
  __shared__ Key tile[kSerialBand];
  __shared__ int tile_at[kSerialBand];
  const Geom& g = a.g;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t pair = (size_t)b * g.Hkv + h;
  int* out = a.page_idx + pair * a.n_select;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  const bool ok = n >= 0 && n <= a.max_seq;
  if (!ok && tid == 0) flag_error(a.status, kDevBadLen);
  const int pages = ok ? n / g.P : 0;
  if (pages <= a.n_select) {
    for (int i = tid; i < a.n_select; i += kPickThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const SelectWs w = select_ws(g.Hkv, a.batch, a.max_pages);
  uint32_t* keys = reinterpret_cast<uint32_t*>(a.ws + w.keys) + pair * a.max_pages;
  Key* band_key = reinterpret_cast<Key*>(a.ws + w.band) + pair * a.max_pages;
  int* band_at = reinterpret_cast<int*>(a.ws + w.index) + pair * a.max_pages;
  const float* bounds = reinterpret_cast<const float*>(a.ws + w.bound) + pair * w.chunks;
  // the free choice: pages keep_first .. pages - keep_last, `need` of them
  const int first = a.keep_first, last = pages - a.keep_last;
  const int need0 = a.n_select - a.keep_first - a.keep_last;
  if (pages <= kSmemKeys) {
    for (int i = tid; i < pages; i += kPickThreads) s_keys[i] = keys[i];
    keys = s_keys;
  }
  uint32_t lo = ~0u, hi = 0u;
  float e = 0.f;
  __syncthreads();
  for (int i = first + tid; i < last; i += kPickThreads) {
    lo = min(lo, keys[i]);
    hi = max(hi, keys[i]);
  }
  const int used_chunks = (pages + kPagesPerCta - 1) / kPagesPerCta;
  for (int i = tid; i < used_chunks; i += kPickThreads) e = fmaxf(e, bounds[i]);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
#pragma unroll
  for (int o = 16; o; o >>= 1) e = warp_max_xor(e, o);
  if (lane == 0) {
    s_lo[warp] = lo;
    s_hi[warp] = hi;
    s_e[warp] = e;
  }
  if (tid == 0) {
    s_prefix = 0;
    s_need = need0;
    s_band = s_above = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPickThreads / 32; ++i) {
    lo = min(lo, s_lo[i]);
    hi = max(hi, s_hi[i]);
    e = fmaxf(e, s_e[i]);
  }
  double above = INFINITY, below = INFINITY;  // need0 == 0: only the kept ones
  if (need0 > 0) {
    // the need-th largest of keys - lo, eight bits at a time from the highest bit in which they differ
    int shift = max(0, 24 - __clz((hi - lo) | 1)), width = 8;
    bool top = true;
    while (true) {
      for (int i = tid; i < 256; i += kPickThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t prefix = s_prefix;
      for (int i = first + tid; i < last; i += kPickThreads) {
        const uint32_t k = keys[i] - lo;
        if (top || (k >> (shift + width)) == (prefix >> (shift + width)))
          atomicAdd(&hist[(k >> shift) & ((1 << width) - 1)], 1);
      }
      __syncthreads();
      if (warp == 0) {  // bins from the largest down: lane l holds 255 - 8 l .. 248 - 8 l
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const int want = s_need;
        int before = incl - sum;
        __syncwarp();
        if (before < want && want <= incl) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < want && want <= before + c[i]) {
              s_need = want - before;
              s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            }
            before += c[i];
          }
        }
      }
      __syncthreads();
      if (shift == 0) break;
      top = false;
      width = min(8, shift);
      shift -= width;
    }
    const double t = value_of(s_prefix + lo);
    above = t + 2.0 * e;
    below = t - 2.0 * e;
    if (!(e < INFINITY) || !(t > -INFINITY)) above = INFINITY, below = -INFINITY;  // score all again
  }
  // count the ones above, list the ones between
  for (int i = first + tid; need0 > 0 && i < last; i += kPickThreads) {
    const uint32_t k = keys[i];
    const double v = value_of(k);
    if (k && v > above) {
      atomicAdd(&s_above, 1);
    } else if (!(below > -INFINITY) || (k && v >= below)) {
      band_at[atomicAdd(&s_band, 1)] = i;
    }
  }
  __syncthreads();
  const int band = s_band, need = need0 - s_above;
  const bool rank = band > need;  // else the whole band is in
  if (rank) {
    for (int c = tid; c < D; c += kPickThreads) {
      double x = 0, y = 0;
      for (int hh = 0; hh < g.gq(); ++hh) {
        const double q = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)(h * g.gq() + hh) * D + c, a.q_dtype);
        x += q < 0 ? 0 : q;
        y += q > 0 ? 0 : -q;
      }
      wa[c] = x;
      wb[c] = y;
    }
    __syncthreads();
    const Kv8Geom kg{g.P, D, g.Hkv};
    const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
    for (int j = warp; j < band; j += kPickThreads / 32) {
      const int pid = page_id(a, b, band_at[j]);
      Key k = 0;
      if (pid >= 0) {
        const uint8_t* block = layer + (size_t)pid * kg.page_bytes();
        double u = 0;
        for (int c = lane; c < D; c += 32)
          u += wa[c] * kv8_value<FMT>(block[kg.hi_off() + c]) - wb[c] * kv8_value<FMT>(block[kg.lo_off() + c]);
#pragma unroll
        for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        k = key_of(u * (double)*reinterpret_cast<const float*>(block + kg.scale_off()));
      }
      if (lane == 0) band_key[j] = k;
    }
    __syncthreads();
    // rank of each: those with a larger key, or an equal one and a lower index
    for (int j0 = 0; j0 < band; j0 += kPickThreads) {
      const int j = j0 + tid;
      const Key k = j < band ? band_key[j] : 0;
      const int at = j < band ? band_at[j] : 0;
      int r = 0;
      for (int i0 = 0; i0 < band; i0 += kSerialBand) {
        __syncthreads();
        if (tid < kSerialBand && i0 + tid < band) {
          tile[tid] = band_key[i0 + tid];
          tile_at[tid] = band_at[i0 + tid];
        }
        __syncthreads();
        const int m = min(kSerialBand, band - i0);
        for (int i = 0; i < m; ++i) r += tile[i] > k || (tile[i] == k && tile_at[i] < at);
      }
      if (j < band) keys[at] = r < need ? ~0u : 0u;
    }
    __syncthreads();
  }
  // ascending list
  int taken = 0;
  for (int i0 = 0; i0 < pages; i0 += kPickThreads) {
    const int i = i0 + tid;
    bool take = false;
    if (i < pages) {
      take = i < first || i >= last;
      if (!take && need0 > 0) {
        const uint32_t k = keys[i];
        const double v = value_of(k);
        take = rank ? k == ~0u || (k && v > above) : !(below > -INFINITY) || (k && v >= below);
      }
    }
    int total;
    const int at = taken + block_rank(take, sums, &total);
    if (take && at < a.n_select) out[at] = i;
    taken += total;
  }
}

template <int D, int FMT>
int launch_select(const Kv8SelectArgs& a, cudaStream_t s, bool pdl) {
  if (a.max_pages > a.n_select) {
    const dim3 grid((a.max_pages + kPagesPerCta - 1) / kPagesPerCta, a.g.Hkv, a.batch);
    const int e = launch_pdl(kv8_score_kernel<D, FMT>, grid, dim3(kScoreThreads), 0, s, pdl, a);
    if (e) return e;
  }
  return launch_pdl(kv8_pick_kernel<D, FMT>, dim3(a.g.Hkv, a.batch), dim3(kPickThreads), 0, s, pdl, a);
}

}  // namespace

size_t kv8_select_ws_bytes(const Geom& g, int batch, int max_seq) { return select_ws(g.Hkv, batch, max_seq / g.P).total; }

int launch_kv8_select(const Kv8SelectArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? launch_select<128, kKv8Int8>(a, s, pdl) : launch_select<128, kKv8E4m3>(a, s, pdl);
  return a.fmt == kKv8Int8 ? launch_select<64, kKv8Int8>(a, s, pdl) : launch_select<64, kKv8E4m3>(a, s, pdl);
}

}  // namespace oscar
