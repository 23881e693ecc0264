// Page selection for sparse decode over the 8-bit cache.
//
//   U_p = scale_p sum_c (a_c hi_pc - b_c lo_pc),  a = sum_h max(q_h, 0),  b = sum_h max(-q_h, 0)
//
// over the heads h that share a kv head (scoring pages by their channels' smallest and largest keys is the method of Tang et
// al., "Quest: Query-Aware Sparsity for Efficient Long-Context LLM Inference", 2024), and of the pages the n_select largest,
// equal ones by the lower index.  It reads 2 d + 4 bytes per page and kv head, 1 / P of what dense attention reads, so latency
// decides: a score kernel over all pages and a pick kernel per (request, kv head).
//
// A score is a product of a page's 2 d codes (exact f16 numbers) with one vector per (request, kv head), taken on the
// tensor cores: 16 pages a warp, the vector as f16 high and low halves in two columns: 62 instructions a page, where 8
// lanes a page on the CUDA cores took 81.  Measured, both kernels: 7.8 us for 4 requests of 8K tokens (4 kv heads), 11 for
// one of 131K, 22 for 32 of 16K to 32K (8 kv heads), whose bounds lie in 100,000 places 16 KB apart.
//
// The order is that of bounds exact to about 48 bits, the scores are float32's.  One is off by at most
//   E_p = 2^-14 A_p,   A_p = scale_p sum_c (a_c |hi_pc| + b_c |lo_pc|):
// the sums over 8 heads take 7 roundings of half a step (2^-24), the halves leave out 2^-22 of a weight, the scale takes a
// rounding, and each of the 2 d / 16 <= 16 matrix instructions adds 17 numbers and loses less than a step (2^-23) of the
// largest for each: 7 + 4 + 1 + 16 x 17 x 2 = 556 half steps, where 2^-14 is 1024; A_p itself comes from the same
// instructions on the magnitudes, off by as little.  Weights below f16's normal numbers are off by up to 2^-25 (the largest
// being 2^14), which adds 2 d M 2^-25 in these units, M the largest code; a product of sum and scale among float32's subnormal numbers
// is off by 2^-150, for which 2^-140 is added.
// With E the largest E_p and t the n-th largest float32 score, the n-th largest exact score lies within E of
// t; so a page above t + 2 E is in, one below t - 2 E is out, and only the ones between, mostly the n-th
// alone, are scored again to about 48 bits and ranked.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kScoreWarps = 4;
constexpr int kChunk = 16;         // pages that a warp scores
// The pick kernel's threads, its digits' bits, and how many pages' keys it holds in shared memory.  Up to 1024 pages a
// small block takes less time than a large one spends in its barriers and empty bins (4 requests of 8K tokens, both
// kernels: 8.0 us, 8.5 with the large block).
template <bool SMALL>
struct Pick {
  static constexpr int kThreads = SMALL ? 128 : 512;
  static constexpr int kBits = SMALL ? 8 : 11;
  static constexpr int kKeys = SMALL ? 1024 : 8192;
};
constexpr int kFew = 64;           // keys that are ranked one by one
constexpr int kTile = 64;          // pages scored again are ranked against tiles of this many
// Up to this many of them.  More, where equal or nearly equal pages leave all of them open, are chosen digit by digit: a query
// of zeros over 64, 128, 256, 1024 and 8192 pages 15.8, 22, 47, 443 and 7167 us ranked, 17.4, 21, 30, 82 and 211 by digits.
constexpr int kRanked = 128;
using Key = unsigned long long;

// Workspace: float32 keys [batch][Hkv][max_pages], 64-bit keys of the band (same count), its page indexes,
// and the largest E_p of each chunk [batch][Hkv][chunks].
struct SelectWs {
  size_t keys, band, index, bound, total;
  int chunks;
};
__host__ __device__ inline SelectWs select_ws(int Hkv, int batch, int max_pages) {
  SelectWs w;
  const size_t n = (size_t)batch * Hkv * max_pages;
  w.chunks = (max_pages + kChunk - 1) / kChunk;
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

// A sum of float32 numbers kept as hi + lo, about 48 bits: the second scoring.  (The card's float64 rate is a sixtieth of
// float32's.)  The additions are Knuth's exact two-number sum.
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
  }
  // code (8 significant bits) times the weight w + v
  __device__ __forceinline__ void add_product(float code, float w, float v) {
    const float p = __fmul_rn(code, w);
    add(p);
    lo = fmaf(code, v, lo + fmaf(code, w, -p));
  }
};

// ------------------------------------------------------------------ scores
// A warp scores 16 pages of one kv head.  Neighbouring warps take the kv heads of the same pages, whose bounds lie in the
// same few megabytes: fewer address translations than with 64 pages of one head a CTA.
template <int D, int FMT, bool QF32>
__global__ void __launch_bounds__(32 * kScoreWarps) kv8_score_kernel(const __grid_constant__ Kv8SelectArgs a) {
  constexpr int KS = D / 16, NC = D / 64;  // k-steps of a section (hi or lo), 16-byte chunks of it that a lane holds
  __shared__ __align__(16) __half s_w[kScoreWarps][2][2][D];  // [hi, lo section][high, low half][channel]
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int b = blockIdx.y, unit = blockIdx.x * kScoreWarps + warp, h = unit % g.Hkv, chunk = unit / g.Hkv;
  const int G = g.gq();
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  const int p0 = chunk * kChunk;
  // the table entries of this lane's two pages and the query travel together
  int pid[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int p = p0 + gid + 8 * r;
    pid[r] = p < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + p] : -1;
  }
  float4 q[8];                             // channels 4 lane .. 4 lane + 3 (lanes of D = 64: the lower half)
  const int qc = 4 * lane % D;
#pragma unroll
  for (int hh = 0; hh < 8; ++hh)
    if (hh < G) q[hh] = kv8_load4<QF32>(a.q, (size_t)b * a.q_stride + (size_t)(h * G + hh) * D + qc);
  if (n < 0 || n > a.max_seq) return;
  const int pages = n / g.P;
  if (pages <= a.n_select || p0 >= pages) return;
  const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
  uint4 code[2][2][NC];                    // [hi, lo][page][chunk tig + 4 c]
  float scale[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int p = p0 + gid + 8 * r;
    const bool wanted = p < pages && !kept(a, p, pages);
    if (wanted && (pid[r] < 0 || pid[r] >= g.num_pages) && tig == 0) flag_error(a.status, kDevBadPage);
    if (!wanted || pid[r] >= g.num_pages) pid[r] = -1;
    const uint8_t* block = layer + (size_t)max(pid[r], 0) * kg.page_bytes();   // (page 0 in the place of none)
    scale[r] = *reinterpret_cast<const float*>(block + kg.scale_off());
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      code[0][r][c] = *reinterpret_cast<const uint4*>(block + kg.hi_off() + (tig + 4 * c) * 16);
      code[1][r][c] = *reinterpret_cast<const uint4*>(block + kg.lo_off() + (tig + 4 * c) * 16);
    }
  }
  // a = sum_h max(q_h, 0) and -b = -sum_h max(-q_h, 0) as f16 halves, the largest component brought to 2^14
  float4 pos = make_float4(0.f, 0.f, 0.f, 0.f), neg = pos;
#pragma unroll
  for (int hh = 0; hh < 8; ++hh)
    if (hh < G) {
      pos.x += fmaxf(q[hh].x, 0.f), pos.y += fmaxf(q[hh].y, 0.f), pos.z += fmaxf(q[hh].z, 0.f), pos.w += fmaxf(q[hh].w, 0.f);
      neg.x += fminf(q[hh].x, 0.f), neg.y += fminf(q[hh].y, 0.f), neg.z += fminf(q[hh].z, 0.f), neg.w += fminf(q[hh].w, 0.f);
    }
  float big = fmaxf(fmaxf(fmaxf(pos.x, pos.y), fmaxf(pos.z, pos.w)), -fminf(fminf(neg.x, neg.y), fminf(neg.z, neg.w)));
#pragma unroll
  for (int o = 16; o; o >>= 1) big = warp_max_xor(big, o);
  float up, down;
  power_of_two(big, &up, &down);
  if (4 * lane < D) {
#pragma unroll
    for (int sect = 0; sect < 2; ++sect) {
      const float4 x = sect ? neg : pos;
      const uint2 hi = make_uint2(pack_half2(x.x * up, x.y * up), pack_half2(x.z * up, x.w * up));
      const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&hi.x)), h1 = __half22float2(*reinterpret_cast<const __half2*>(&hi.y));
      *reinterpret_cast<uint2*>(&s_w[warp][sect][0][qc]) = hi;
      *reinterpret_cast<uint2*>(&s_w[warp][sect][1][qc]) =
          make_uint2(pack_half2(x.x * up - h0.x, x.y * up - h0.y), pack_half2(x.z * up - h1.x, x.w * up - h1.y));
    }
  }
  __syncwarp();
  // columns 0 and 1: high and low halves; sc: scores, sa: sums of magnitudes
  float sc[4] = {0.f, 0.f, 0.f, 0.f}, sa[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int sect = 0; sect < 2; ++sect)
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int c = kk / 4, w = kk % 4;
      uint2 bw = make_uint2(0u, 0u);
      if (gid < 2) bw = *reinterpret_cast<const uint2*>(&s_w[warp][sect][gid][(tig + 4 * c) * 16 + 4 * w]);
      uint32_t x[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 v = code[sect][r][c];
        x[r] = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
      }
      const uint32_t a0 = kv8_pair<FMT, 0>(x[0]), a1 = kv8_pair<FMT, 0>(x[1]), a2 = kv8_pair<FMT, 1>(x[0]), a3 = kv8_pair<FMT, 1>(x[1]);
      constexpr uint32_t kAbs = 0x7fff7fffu;
      mma_f16(sc, a0, a1, a2, a3, bw.x, bw.y);
      mma_f16(sa, a0 & kAbs, a1 & kAbs, a2 & kAbs, a3 & kAbs, bw.x & kAbs, bw.y & kAbs);
    }
  const SelectWs w = select_ws(g.Hkv, a.batch, a.max_pages);
  const size_t pair = (size_t)b * g.Hkv + h;
  uint32_t* keys = reinterpret_cast<uint32_t*>(a.ws + w.keys) + pair * a.max_pages;
  float bound = 0.f;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int p = p0 + gid + 8 * r;
    // (without the query's power of two, which is the same for every page: with it, scale and all could leave the normal numbers)
    const float score = (sc[2 * r] + sc[2 * r + 1]) * scale[r];
    constexpr float kFloor = 2 * D * (FMT == kKv8Int8 ? 127.f : 448.f) * 0x1p-25f;
    const float e = fmaf(sa[2 * r] + sa[2 * r + 1], 0x1p-14f, kFloor) * scale[r] + 0x1p-140f;   // (and float32's own subnormal numbers)
    if (tig == 0 && p < pages) keys[p] = pid[r] >= 0 ? key_of(score) : 0u;
    // no finite bound, or a score that overflowed: every page is scored again
    if (tig == 0 && pid[r] >= 0) bound = (e <= 3e38f && fabsf(score) <= 3e38f) ? fmaxf(bound, e) : INFINITY;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) bound = warp_max_xor(bound, o);
  if (lane == 0) reinterpret_cast<float*>(a.ws + w.bound)[pair * w.chunks + chunk] = bound;
}

// ------------------------------------------------------------------ pick
template <int D, int FMT, bool SMALL>
__global__ void __launch_bounds__(Pick<SMALL>::kThreads, 2) kv8_pick_kernel(const __grid_constant__ Kv8SelectArgs a) {
  constexpr int kPickThreads = Pick<SMALL>::kThreads, kSmemKeys = Pick<SMALL>::kKeys;
  constexpr int kBinBits = Pick<SMALL>::kBits, kBins = 1 << kBinBits;
  __shared__ uint32_t s_keys[kSmemKeys];
  __shared__ int hist[kBins];              // then the list's bit words
  __shared__ uint32_t s_few[kFew];
  __shared__ uint32_t u_lo[kPickThreads / 32], u_hi[kPickThreads / 32];
  __shared__ float f_e[kPickThreads / 32];
  __shared__ int sums[kPickThreads / 32];
  __shared__ uint32_t s_nth;
  __shared__ int s_bin, s_need, s_count, s_few_n, s_band, s_above;
  __shared__ float s_q[8 * D];
  __shared__ __align__(16) float w_hi[2][D], w_lo[2][D];   // [a, b]: the weights of a second scoring as two numbers
  __shared__ float s_big[kPickThreads / 32];
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
  const int chunks = (pages + kChunk - 1) / kChunk;
  for (int i = tid; i < chunks; i += kPickThreads) e = fmaxf(e, bounds[i]);
  for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
  if (tid == 0) {
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
  // arithmetic rounded outwards: float64 comparisons of every page took 8 us of 21 at 131K tokens.
  uint32_t above = ~0u, below = ~0u;
  // s_bin: the bin of hist, counted from the largest, with the s_need-th; s_need: which of that bin's s_count it is
  auto find_bin = [&] {
    // thread t holds the kBins / kPickThreads below kBins - 1 - t kBins / kPickThreads
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
          s_bin = kBins - 1 - tid * kPer - i;
        }
        before += c[i];
      }
    }
    __syncthreads();
  };
  if (need0 > 0) {
    // the need-th largest of keys - lo, a digit at a time from the highest bit in which they differ, until few
    // enough keys share its digits to be ranked one by one
    int shift = max(0, 32 - kBinBits - __clz((hi - lo) | 1)), width = kBinBits;
    bool top = true;
    uint32_t found = 0;
    while (true) {
      for (int i = first + tid; i < last; i += kPickThreads) {
        const uint32_t k = keys[i] - lo;
        if (top || (k >> (shift + width)) == (found >> (shift + width)))
          atomicAdd(&hist[(k >> shift) & ((1 << width) - 1)], 1);
      }
      __syncthreads();
      find_bin();
      found |= (uint32_t)s_bin << shift;
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
          if (more < left && left <= more + same) s_nth = k;
        }
        __syncthreads();
        found = s_nth;
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
    float big = 0.f;
    for (int i = tid; i < g.gq() * D; i += kPickThreads) big = fmaxf(big, fabsf(s_q[i]));
#pragma unroll
    for (int o = 16; o; o >>= 1) big = warp_max_xor(big, o);
    if (lane == 0) s_big[warp] = big;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPickThreads / 32; ++i) big = fmaxf(big, s_big[i]);
    float up, down;
    power_of_two(big, &up, &down);
    for (int c = tid; c < D; c += kPickThreads) {
      Sum2 x{0.f, 0.f}, y{0.f, 0.f};
      for (int i = c; i < g.gq() * D; i += D) {
        const float q = s_q[i] * up;
        x.add(fmaxf(q, 0.f));
        y.add(fmaxf(-q, 0.f));
      }
      w_hi[0][c] = x.hi, w_lo[0][c] = x.lo;
      w_hi[1][c] = y.hi, w_lo[1][c] = y.lo;
    }
    __syncthreads();
    // eight lanes a page
    constexpr int C = D / 8;
    const Kv8Geom kg{g.P, D, g.Hkv};
    const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
    for (int j0 = 0; j0 < band; j0 += kPickThreads / 8) {
      const int j = j0 + (tid >> 3), sub = tid & 7;
      const int pid = j < band ? page_id(a, b, band_at[j]) : -1;
      const uint8_t* block = layer + (size_t)max(pid, 0) * kg.page_bytes();
      const float scale = *reinterpret_cast<const float*>(block + kg.scale_off());
      Sum2 u{0.f, 0.f};
#pragma unroll
      for (int i = 0; i < C / 4; ++i) {
        const uint32_t hw = *reinterpret_cast<const uint32_t*>(block + kg.hi_off() + sub * C + 4 * i);
        const uint32_t lw = *reinterpret_cast<const uint32_t*>(block + kg.lo_off() + sub * C + 4 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = sub * C + 4 * i + k;
          u.add_product(kv8_value<FMT>((hw >> (8 * k)) & 255u), w_hi[0][c], w_lo[0][c]);
          u.add_product(-kv8_value<FMT>((lw >> (8 * k)) & 255u), w_hi[1][c], w_lo[1][c]);
        }
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, u.hi, o), y = __shfl_xor_sync(0xffffffffu, u.lo, o);
        u.add(x);
        u.lo += y;
      }
      // (the power of two is the same for every page)
      if (sub == 0 && j < band) band_key[j] = pid >= 0 ? key_of(((double)u.hi + (double)u.lo) * scale) : 0ull;
    }
    __syncthreads();
    if (band <= kRanked) {
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
    } else {
      // the need-th in that order, a digit at a time, first of the keys, then of the indexes of the ones equal to its key
      auto nth = [&](int bits, auto value, auto among) {
        Key prefix = 0;
        for (int shift = bits; shift > 0;) {
          const int top_bits = shift, width = min(kBinBits, shift);
          shift -= width;
          for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
          __syncthreads();
          for (int j = tid; j < band; j += kPickThreads) {
            const Key v = value(j);
            if (among(j) && (top_bits == bits || (v >> top_bits) == (prefix >> top_bits)))
              atomicAdd(&hist[(int)(v >> shift) & ((1 << width) - 1)], 1);
          }
          __syncthreads();
          find_bin();
          prefix |= (Key)s_bin << shift;
          if (s_need == s_count) break;                 // every one with these digits is in
        }
        return prefix;
      };
      if (tid == 0) s_need = need;
      const Key key = nth(64, [&](int j) { return band_key[j]; }, [](int) { return true; });
      const bool ties = s_need < s_count;
      __syncthreads();
      Key low = 0;
      if (ties) low = nth(32, [&](int j) { return (Key)~(uint32_t)band_at[j]; }, [&](int j) { return band_key[j] == key; });
      for (int j = tid; j < band; j += kPickThreads)
        keys[band_at[j]] = band_key[j] > key || (band_key[j] == key && (Key)~(uint32_t)band_at[j] >= low) ? ~0u : 0u;
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
    const long long units = (long long)((a.max_pages + kChunk - 1) / kChunk) * a.g.Hkv;
    const dim3 grid((unsigned)((units + kScoreWarps - 1) / kScoreWarps), a.batch);
    const int e = a.q_dtype == kDtypeF32 ? launch_pdl(kv8_score_kernel<D, FMT, true>, grid, dim3(32 * kScoreWarps), 0, s, pdl, a)
                                         : launch_pdl(kv8_score_kernel<D, FMT, false>, grid, dim3(32 * kScoreWarps), 0, s, pdl, a);
    if (e) return e;
  }
  const dim3 grid(a.g.Hkv, a.batch);
  if (a.max_pages <= Pick<true>::kKeys)
    return launch_pdl(kv8_pick_kernel<D, FMT, true>, grid, dim3(Pick<true>::kThreads), 0, s, pdl, a);
  return launch_pdl(kv8_pick_kernel<D, FMT, false>, grid, dim3(Pick<false>::kThreads), 0, s, pdl, a);
}

}  // namespace

size_t kv8_select_ws_bytes(const Geom& g, int batch, int max_seq) { return select_ws(g.Hkv, batch, max_seq / g.P).total; }

int launch_kv8_select(const Kv8SelectArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? launch_select<128, kKv8Int8>(a, s, pdl) : launch_select<128, kKv8E4m3>(a, s, pdl);
  return a.fmt == kKv8Int8 ? launch_select<64, kKv8Int8>(a, s, pdl) : launch_select<64, kKv8E4m3>(a, s, pdl);
}

}  // namespace oscar
