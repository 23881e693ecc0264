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
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
constexpr int kFew = 64;           // keys that are ranked one by one
constexpr int kTile = 64;          // pages scored again are ranked against tiles of this many
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
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }
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

// sum_h max(q_hc, 0) and sum_h max(-q_hc, 0) over the heads of kv head h (a NaN stays one).
__device__ __forceinline__ float2 query_sums(const Kv8SelectArgs& a, int b, int h, int c, int D) {
  const int G = a.g.gq();
  const size_t at = (size_t)b * a.q_stride + (size_t)h * G * D + c;
  float q[8];
#pragma unroll
  for (int hh = 0; hh < 8; ++hh) q[hh] = hh < G ? kv8_load(a.q, at + (size_t)hh * D, a.q_dtype) : 0.f;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int hh = 0; hh < 8; ++hh) {
    s.x += q[hh] < 0.f ? 0.f : q[hh];
    s.y += q[hh] > 0.f ? 0.f : -q[hh];
  }
  return s;
}

// ------------------------------------------------------------------ scores
template <int D, int FMT>
__global__ void __launch_bounds__(kScoreThreads) kv8_score_kernel(const __grid_constant__ Kv8SelectArgs a) {
  constexpr int C = D / 8;                 // channels of a lane
  constexpr int kRounds = kPagesPerCta / (kScoreThreads / 8);
  __shared__ float s_bound[kScoreThreads / 32];
  __shared__ __align__(16) float s_wa[D], s_wb[D];
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, sub = lane & 7;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  const int p0 = blockIdx.x * kPagesPerCta;
  // the table entries and the query travel together
  int pids[kRounds];
#pragma unroll
  for (int it = 0; it < kRounds; ++it) {
    const int p = p0 + it * (kScoreThreads / 8) + (tid >> 3);
    pids[it] = p < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + p] : -1;
  }
  for (int c = tid; c < D; c += kScoreThreads) {
    // (channels 4 w .. 4 w + 3 of lane `sub` next to those of the other lanes: no bank conflicts)
    const float2 x = query_sums(a, b, h, c, D);
    const int at = ((c % C) / 4 * 8 + c / C) * 4 + c % 4;
    s_wa[at] = x.x;
    s_wb[at] = x.y;
  }
  if (n < 0 || n > a.max_seq) return;
  const int pages = n / g.P;
  if (pages <= a.n_select || p0 >= pages) return;
  __syncthreads();
  // and so do the bounds of all this CTA's pages
  const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
  uint32_t lo[kRounds][C / 4], hi[kRounds][C / 4];
  float scale[kRounds];
#pragma unroll
  for (int it = 0; it < kRounds; ++it) {
    const int p = p0 + it * (kScoreThreads / 8) + (tid >> 3);
    const bool wanted = p < pages && !kept(a, p, pages);
    if (wanted && (pids[it] < 0 || pids[it] >= g.num_pages) && sub == 0) flag_error(a.status, kDevBadPage);
    if (!wanted || pids[it] >= g.num_pages) pids[it] = -1;
  }
#pragma unroll
  for (int it = 0; it < kRounds; ++it) {
    const uint8_t* block = layer + (size_t)max(pids[it], 0) * kg.page_bytes();   // (page 0 in the place of none)
    scale[it] = *reinterpret_cast<const float*>(block + kg.scale_off());
    if constexpr (C == 16) {
      const uint4 x = *reinterpret_cast<const uint4*>(block + kg.lo_off() + sub * C);
      const uint4 y = *reinterpret_cast<const uint4*>(block + kg.hi_off() + sub * C);
      lo[it][0] = x.x, lo[it][1] = x.y, lo[it][2] = x.z, lo[it][3] = x.w;
      hi[it][0] = y.x, hi[it][1] = y.y, hi[it][2] = y.z, hi[it][3] = y.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(block + kg.lo_off() + sub * C);
      const uint2 y = *reinterpret_cast<const uint2*>(block + kg.hi_off() + sub * C);
      lo[it][0] = x.x, lo[it][1] = x.y;
      hi[it][0] = y.x, hi[it][1] = y.y;
    }
  }
  float mass = 0.f, u[kRounds];
#pragma unroll
  for (int it = 0; it < kRounds; ++it) u[it] = 0.f;
#pragma unroll
  for (int w = 0; w < C / 4; ++w) {
    const float4 wa = reinterpret_cast<const float4*>(s_wa)[w * 8 + sub], wb = reinterpret_cast<const float4*>(s_wb)[w * 8 + sub];
    mass += ((wa.x + wb.x) + (wa.y + wb.y)) + ((wa.z + wb.z) + (wa.w + wb.w));
#pragma unroll
    for (int it = 0; it < kRounds; ++it) {
      const uint32_t l0 = kv8_pair<FMT, 0>(lo[it][w]), l1 = kv8_pair<FMT, 1>(lo[it][w]);
      const uint32_t h0 = kv8_pair<FMT, 0>(hi[it][w]), h1 = kv8_pair<FMT, 1>(hi[it][w]);
      const float2 x0 = __half22float2(*reinterpret_cast<const __half2*>(&l0)), x1 = __half22float2(*reinterpret_cast<const __half2*>(&l1));
      const float2 y0 = __half22float2(*reinterpret_cast<const __half2*>(&h0)), y1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
      u[it] = fmaf(wa.x, y0.x, fmaf(-wb.x, x0.x, u[it]));
      u[it] = fmaf(wa.y, y0.y, fmaf(-wb.y, x0.y, u[it]));
      u[it] = fmaf(wa.z, y1.x, fmaf(-wb.z, x1.x, u[it]));
      u[it] = fmaf(wa.w, y1.y, fmaf(-wb.w, x1.y, u[it]));
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
#pragma unroll
    for (int it = 0; it < kRounds; ++it) u[it] += __shfl_xor_sync(0xffffffffu, u[it], o);
  }
  mass *= (FMT == kKv8Int8 ? 127.f : 448.f) * 0x1p-18f;
  uint32_t* keys = reinterpret_cast<uint32_t*>(a.ws + select_ws(g.Hkv, a.batch, a.max_pages).keys) +
                   ((size_t)b * g.Hkv + h) * a.max_pages;
  float bound = 0.f;
#pragma unroll
  for (int it = 0; it < kRounds; ++it) {
    const int p = p0 + it * (kScoreThreads / 8) + (tid >> 3);
    const bool scored = pids[it] >= 0;
    const float score = u[it] * scale[it];
    if (p < pages && sub == 0) keys[p] = scored ? key_of(score) : 0u;
    if (scored) {
      const float e = mass * scale[it] + 0x1p-140f;  // (and the roundings among the subnormal numbers)
      // no finite bound, or a score that overflowed: every page is scored again
      bound = (e <= 3e38f && fabsf(score) <= 3e38f) ? fmaxf(bound, e) : INFINITY;
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
template <int D, int FMT>
__global__ void __launch_bounds__(kPickThreads, 2) kv8_pick_kernel(const __grid_constant__ Kv8SelectArgs a) {
  __shared__ uint32_t s_keys[kSmemKeys];
  __shared__ int hist[kBins];              // then the list's bit words
  __shared__ uint32_t s_few[kFew];
  __shared__ uint32_t u_lo[kPickThreads / 32], u_hi[kPickThreads / 32];
  __shared__ float f_e[kPickThreads / 32];
  __shared__ int sums[kPickThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_count, s_few_n, s_band, s_above;
  __shared__ float s_q[8 * D];
  __shared__ double wa[D], wb[D];
  __shared__ Key tile[kTile];
  __shared__ int tile_at[kTile];
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
  // the free choice: pages keep_first .. pages - keep_last, need0 of them
  const int first = a.keep_first, last = pages - a.keep_last;
  const int need0 = a.n_select - a.keep_first - a.keep_last;
  // keys into shared memory where they fit, their range, and the largest bound
  uint32_t lo = ~0u, hi = 0u;
  const bool fits = pages <= kSmemKeys;
  for (int i = tid; i < pages; i += kPickThreads) {
    const uint32_t k = keys[i];
    if (fits) s_keys[i] = k;
    if (i >= first && i < last) {
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  if (fits) keys = s_keys;
  // the query for a second scoring, should there be one, travels with the keys
  for (int i = tid; i < g.gq() * D; i += kPickThreads)
    s_q[i] = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)h * g.gq() * D + i, a.q_dtype);
  float e = 0.f;
  const int chunks = (pages + kPagesPerCta - 1) / kPagesPerCta;
  for (int i = tid; i < chunks; i += kPickThreads) e = fmaxf(e, bounds[i]);
  for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
  if (tid == 0) {
    s_prefix = 0;
    s_need = need0;
    s_band = s_above = s_few_n = 0;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
#pragma unroll
  for (int o = 16; o; o >>= 1) e = warp_max_xor(e, o);
  if (lane == 0) {
    u_lo[warp] = lo;
    u_hi[warp] = hi;
    f_e[warp] = e;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, u_lo[lane % (kPickThreads / 32)]);
  hi = __reduce_max_sync(0xffffffffu, u_hi[lane % (kPickThreads / 32)]);
  e = f_e[lane % (kPickThreads / 32)];
#pragma unroll
  for (int o = kPickThreads / 64; o; o >>= 1) e = warp_max_xor(e, o);
  // keys over `above` are in, those under `below` out (need0 == 0: only the kept pages are in).  Both come from float32
  // arithmetic rounded outwards: the card's float64 rate is a hundredth of that, too slow for every page.
  uint32_t above = ~0u, below = ~0u;
  if (need0 > 0) {
    // the need-th largest of keys - lo, eleven bits at a time from the highest bit in which they differ, until few
    // enough keys share its digits to be ranked one by one
    int shift = max(0, 32 - kBinBits - __clz((hi - lo) | 1)), width = kBinBits;
    bool top = true;
    uint32_t found;
    while (true) {
      const uint32_t prefix = s_prefix;
      for (int i = first + tid; i < last; i += kPickThreads) {
        const uint32_t k = keys[i] - lo;
        if (top || (k >> (shift + width)) == (prefix >> (shift + width)))
          atomicAdd(&hist[(k >> shift) & ((1 << width) - 1)], 1);
      }
      __syncthreads();
      // bins from the largest down: thread t holds the kBins / kPickThreads below kBins - 1 - t kBins / kPickThreads
      constexpr int kPer = kBins / kPickThreads;
      int c[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += c[i] = hist[kBins - 1 - tid * kPer - i];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sums[warp] = incl;
      const int want = s_need;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPickThreads / 32; ++i) incl += i < warp ? sums[i] : 0;
      int before = incl - sum;
      if (before < want && want <= incl) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (before < want && want <= before + c[i]) {
            s_need = want - before;
            s_count = c[i];
            s_prefix = prefix | ((uint32_t)(kBins - 1 - tid * kPer - i) << shift);
          }
          before += c[i];
        }
      }
      __syncthreads();
      found = s_prefix;
      if (shift == 0) break;
      if (s_count <= kFew) {
        for (int i = first + tid; i < last; i += kPickThreads) {
          const uint32_t k = keys[i] - lo;
          if ((k >> shift) == (found >> shift)) s_few[atomicAdd(&s_few_n, 1)] = k;
        }
        __syncthreads();
        // the need-th largest of them: fewer than need are larger, and it with its equals reaches need
        const int m = s_few_n, left = s_need;
        if (tid < m) {
          const uint32_t k = s_few[tid];
          int more = 0, same = 0;
          for (int i = 0; i < m; ++i) {
            more += s_few[i] > k;
            same += s_few[i] == k;
          }
          if (more < left && left <= more + same) s_prefix = k;
        }
        __syncthreads();
        found = s_prefix;
        break;
      }
      for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
      __syncthreads();
      top = false;
      width = min(kBinBits, shift);
      shift -= width;
    }
    const float t = value_of(found + lo), far = 2.f * e;
    if (e < 3e38f / 2 && t > -INFINITY) {
      above = key_of(__fadd_ru(t, far));
      below = key_of(__fadd_rd(t, -far));
    } else {
      below = 0u;  // score all again
    }
  }
  // count the ones above, list the ones between
  for (int i = first + tid; need0 > 0 && i < last; i += kPickThreads) {
    const uint32_t k = keys[i];
    if (k > above) atomicAdd(&s_above, 1);
    else if (k >= below) band_at[atomicAdd(&s_band, 1)] = i;
  }
  __syncthreads();
  const int band = s_band, need = need0 - s_above;
  const bool rank = band > need;  // else the whole band is in
  if (rank) {
    for (int c = tid; c < D; c += kPickThreads) {
      double x = 0, y = 0;
      for (int i = c; i < g.gq() * D; i += D) {
        const double q = s_q[i];
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
        const double scale = *reinterpret_cast<const float*>(block + kg.scale_off());
        double u = 0;
#pragma unroll
        for (int c = 0; c < D; c += 32)
          u += wa[c + lane] * kv8_value<FMT>(block[kg.hi_off() + c + lane]) - wb[c + lane] * kv8_value<FMT>(block[kg.lo_off() + c + lane]);
#pragma unroll
        for (int o = 16; o; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        k = key_of(u * scale);
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
      for (int i0 = 0; i0 < band; i0 += kTile) {
        __syncthreads();
        if (tid < kTile && i0 + tid < band) {
          tile[tid] = band_key[i0 + tid];
          tile_at[tid] = band_at[i0 + tid];
        }
        __syncthreads();
        const int m = min(kTile, band - i0);
        for (int i = 0; i < m; ++i) r += tile[i] > k || (tile[i] == k && tile_at[i] < at);
      }
      if (j < band) keys[at] = r < need ? ~0u : 0u;
    }
    __syncthreads();
  }
  // ascending list: a bit per page, 32 kWords pages at a time; thread t counts and writes those of word t
  constexpr int kWords = kPickThreads;
  uint32_t* words = reinterpret_cast<uint32_t*>(hist);
  static_assert(kWords <= kBins, "the bit words take the bins' place");
  int taken = 0;
  for (int i0 = 0; i0 < pages; i0 += 32 * kWords) {
    const int m = min(pages - i0, 32 * kWords);
    for (int j = tid; j < (m + 31) / 32 * 32; j += kPickThreads) {
      const int i = i0 + j;
      bool take = false;
      if (i < pages) {
        const uint32_t k = keys[i];
        take = i < first || i >= last || (need0 > 0 && (rank ? k > above || k == ~0u : k >= below));
      }
      const unsigned bits = __ballot_sync(__activemask(), take);
      if (lane == 0) words[j / 32] = bits;
    }
    __syncthreads();
    uint32_t mine = tid < (m + 31) / 32 ? words[tid] : 0;
    int incl = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int at = taken + incl - __popc(mine);
#pragma unroll
    for (int i = 0; i < kPickThreads / 32; ++i) {
      const int s = sums[i];
      at += i < warp ? s : 0;
      taken += s;
    }
    for (; mine; mine &= mine - 1, ++at)
      if (at < a.n_select) out[at] = i0 + 32 * tid + __ffs(mine) - 1;
    __syncthreads();
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
