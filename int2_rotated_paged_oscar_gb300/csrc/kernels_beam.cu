// The next beams of a beam search: of an item's beams x vocabulary candidates
//
//     key(i, v) = score_i + ((x_iv - m_i) - log sum_u e^{x_iu - m_i}),  m_i = max_u x_iu,
//
// the n_out largest, the lowest i V + v first among equal ones.
//
// The logits are read once: a first kernel, a warp per unit of 1024 logits, leaves the unit's maximum and sum of exponentials.  It is
// bound by memory and by the latency of a warp's one chain (32 x 8 rows of 131,072 BF16 logits: 14.6 us, 4.6 of 6.7 TB/s;
// fewer CTAs whose warps take one unit after another, the next one's loads ahead: 19 us).  A second one, a CTA per item, forms
// the rows' normalisers and looks through the best few units once more, 128 logits a warp with a common floor; then through those
// others whose largest candidate comes before the last of the n_out at hand.  That is one chain of barriers, 5 to 13 us
// (both kernels: 11 us for 8 x 4 beams of 32,768 and 25 for 32 x 8 of 131,072; 33 and 107 in the simplest form).
#include "beam_internal.h"
#include "common.cuh"

namespace oscar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Logits [i, i + N) of a row, N adjacent ones that make 16 bytes; -infinity from the vocabulary's end on.  Which logits a thread
// takes does not depend on the row's alignment, so equal rows have equal sums.
template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* row, int i, int vocab, bool aligned) {
    if (aligned && i + N <= vocab) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)i * (BF16 ? 2 : 4));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16) {
        const uint32_t lo = i + 2 * k < vocab ? static_cast<const uint16_t*>(row)[i + 2 * k] : 0xFF80u;
        const uint32_t hi = i + 2 * k + 1 < vocab ? static_cast<const uint16_t*>(row)[i + 2 * k + 1] : 0xFF80u;
        w[k] = hi << 16 | lo;
      } else {
        w[k] = i + k < vocab ? static_cast<const uint32_t*>(row)[i + k] : 0xFF800000u;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (BF16) return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
    return __uint_as_float(w[j]);
  }
};

__device__ __forceinline__ const void* row_of(const BeamArgs& a, long long row) {
  return static_cast<const uint8_t*>(a.logits) + row * a.stride * (a.dtype == kDtypeBF16 ? 2 : 4);
}

// ------------------------------------------------------------------ units
constexpr int kUnitThreads = 256;
constexpr float kNear = 4096.f;                            // c and its last place are below 2^13 and 2^-11

template <bool BF16>
__global__ void __launch_bounds__(kUnitThreads) beam_unit_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<BF16>;
  constexpr int kVecs = kBeamUnit / (32 * V::N);
  const int lane = threadIdx.x & 31, units = beam_units(a.vocab);
  const long long at = (long long)blockIdx.x * (kUnitThreads / 32) + (threadIdx.x >> 5);
  const long long row = at >> 32 ? at / units : (uint32_t)at / (uint32_t)units;  // (a division of 64 bits takes five times as long)
  pdl_wait();
  pdl_launch_dependents();
  if (row >= (long long)a.batch * a.beams) return;
  const uint8_t done = a.finished ? a.finished[row] : 0;
  const void* x = row_of(a, row);
  const bool aligned = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  const int i0 = (int)(at - row * units) * kBeamUnit + lane * V::N;
  if (done) return;
  V v[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) v[k].load(x, i0 + k * 32 * V::N, a.vocab, aligned);
  float m = -INFINITY;
  if constexpr (BF16) {
    __nv_bfloat162 t = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) t = __hmax2(t, *reinterpret_cast<const __nv_bfloat162*>(&v[k].w[j]));
    m = fmaxf(__low2float(t), __high2float(t));
  } else {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) m = max3(max3(m, v[k].get(0), v[k].get(1)), v[k].get(2), v[k].get(3));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) m = warp_max_xor(m, d);
  const float ref = m == -INFINITY ? 0.f : m;
  // 2^(x log2 e - c) with c = ref log2 e rounded, and what that leaves out once, for the sum; beyond kNear it is no small number
  const bool near = fabsf(ref) < kNear;
  const float c = ref * kLog2e;
  const uint64_t up = pair(kLog2e, kLog2e), off = pair(-c, -c);
  uint64_t s[2] = {0, 0};                                 // (a NaN or +infinity makes a NaN of it)
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int j = 0; j < V::N; j += 2) {
      const float lo = v[k].get(j), hi = v[k].get(j + 1);
      const uint64_t y = near ? fma2(pair(lo, hi), up, off) : pair((lo - ref) * kLog2e, (hi - ref) * kLog2e);
      s[(j >> 1) & 1] = add2(s[(j >> 1) & 1], pair(ex2(first(y)), ex2(second(y))));
    }
  s[0] = add2(s[0], s[1]);
  float sum = first(s[0]) + second(s[0]);
  if (near) sum = fmaf(sum, fmaf(-ref, kLog2e, c) * 0.6931471805599453f, sum);  // (2^r of |r| <= 2^-12, half a last place of c)
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) reinterpret_cast<float2*>(a.part)[at] = make_float2(m, sum);
}

// ------------------------------------------------------------------ candidates
constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32;
constexpr int kSlice = 128;                                // logits of a unit that a warp looks through, four a lane
constexpr int kRound = kPickWarps * kSlice / kBeamUnit;    // units looked through at a time
constexpr int kRoom = kMaxCandidates + kPickWarps * kSlice;  // candidates at hand: those kept and the warps' most

// A double as an unsigned number of the same order; 0 stands for no candidate (-infinity).
__device__ __forceinline__ unsigned long long ordered(double k) {
  if (k == -INFINITY) return 0;
  const unsigned long long u = (unsigned long long)__double_as_longlong(k + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double from_ordered(unsigned long long u) {
  return __longlong_as_double((long long)(u >> 63 ? u & ~(1ull << 63) : ~u));
}

// What decides between equal keys, the larger first: the lower beam, the larger logit (within a beam the keys differ as the
// logits do, however little of it a double keeps), the lower token (or chunk).
__device__ __forceinline__ unsigned long long order_of(int beam, float x, int v) {
  const uint32_t u = __float_as_uint(x + 0.f), up = u >> 31 ? ~u : u | 0x80000000u;
  return (unsigned long long)(kMaxBeams - 1 - beam) << 56 | (unsigned long long)up << 24 | (uint32_t)(kMaxVocab - 1 - v);
}
__device__ __forceinline__ int beam_of(unsigned long long order) { return kMaxBeams - 1 - (int)(order >> 56); }
__device__ __forceinline__ float logit_of(unsigned long long order) {
  const uint32_t up = (uint32_t)(order >> 24);
  return __uint_as_float(up >> 31 ? up & 0x7FFFFFFFu : ~up);
}
__device__ __forceinline__ int token_of(unsigned long long order) { return kMaxVocab - 1 - (int)(order & (kMaxVocab - 1)); }

struct Entry {
  unsigned long long key, order;
  __device__ __forceinline__ bool before(const Entry& o) const { return key > o.key || (key == o.key && order > o.order); }
};

struct PickSmem {
  Entry pool[kRoom], kept[kMaxCandidates];
  float group[kPickThreads / 8];
  int group_unit[kPickThreads / 8], first[kRound];
  float mark[kPickWarps];
  float norm[kMaxBeams], norm_lo[kMaxBeams];  // log of the sum of exponentials, as two numbers
  float top[kMaxBeams];       // m_i
  float score[kMaxBeams];
  int kind[kMaxBeams];        // 0: open, 1: finished, 2: no candidates
  int unit[kPickThreads];     // units to look through
  Entry floor;                // what a candidate has to come before, or be
  int n_unit, n_first, count, n_kept;
};

__device__ __forceinline__ double key_of(const PickSmem& s, int i, float x) {
  return (double)s.score[i] + (((double)x - (double)s.top[i]) - ((double)s.norm[i] + (double)s.norm_lo[i]));
}

// Places of n entries among themselves, eight threads an entry; the first `most` of them are handed to put(place, entry).
template <typename Put>
__device__ __forceinline__ void rank_entries(int n, int most, const Entry* list, Put put) {
  const int part = threadIdx.x & 7;
  for (int e = threadIdx.x >> 3; e < ((n + 3) & ~3); e += kPickThreads / 8) {
    const Entry mine = e < n ? list[e] : Entry{0, 0};
    int before = 0;
    for (int o = part; o < n; o += 8) before += list[o].before(mine);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
    if (part == 0 && mine.key != 0 && before < most) put(before, e);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickSmem& s = *reinterpret_cast<PickSmem*>(smem_raw);
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.beams, units = beam_units(a.vocab), N = a.n_out, total = K * units;
  const float2* part = reinterpret_cast<const float2*>(a.part) + (long long)b * K * units;
  pdl_wait();
  pdl_launch_dependents();
  // (what the first steps need, all under way at once)
  const float own_top = tid < total ? part[tid].x : 0.f;
  // the rows' normalisers
  for (int i = warp; i < K; i += kPickWarps) {
    const long long row = (long long)b * K + i;
    const float2* mine = part + (long long)i * units;
    constexpr int kHold = 4;
    float2 p[kHold];
#pragma unroll
    for (int k = 0; k < kHold; ++k) p[k] = lane + 32 * k < units ? mine[lane + 32 * k] : make_float2(-INFINITY, 0.f);
    const float score = a.scores[row];
    int kind = a.finished && a.finished[row] ? 1 : 0;
    bool sound = score < INFINITY;                       // (false for a NaN)
    float m = -INFINITY;
    float sum = 0.f, rest = 0.f;                          // rest: what the additions lose
    auto add = [&](float y) {
      const float t = sum + y, z = t - sum;
      rest += (sum - (t - z)) + (y - z);
      sum = t;
    };
    if (kind == 0) {                                      // (else nothing was written there)
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        m = fmaxf(m, p[k].x);
        sound &= p[k].y == p[k].y;
      }
      for (int c = lane + 32 * kHold; c < units; c += 32) {
        const float2 q = mine[c];
        m = fmaxf(m, q.x);
        sound &= q.y == q.y;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) m = warp_max_xor(m, d);
      if (m > -INFINITY) {
#pragma unroll
        for (int k = 0; k < kHold; ++k) add(p[k].y * expf(p[k].x - m));
        for (int c = lane + 32 * kHold; c < units; c += 32) add(mine[c].y * expf(mine[c].x - m));
      }
#pragma unroll 1
      for (int d = 16; d; d >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, sum, d), its = __shfl_xor_sync(0xffffffffu, rest, d);
        add(other);
        rest += its;
      }
      if (m == -INFINITY) kind = 2;
    }
    sound = __all_sync(0xffffffffu, sound);
    if (!sound || score == -INFINITY) kind = 2;
    if (lane == 0) {
      if (!sound) flag_error(a.status, kDevBadValue);
      // log of the sum: float32's, and a Newton step for what it leaves out
      const float y = logf(sum);
      s.score[i] = score;
      s.top[i] = m;
      s.norm[i] = kind == 0 ? y : 0.f;
      s.norm_lo[i] = kind == 0 ? fmaf(sum, expf(-y), -1.f) + rest / sum : 0.f;
      s.kind[i] = kind;
    }
  }
  if (tid == 0) {
    s.floor = Entry{0, 0};
    s.count = s.n_kept = s.n_first = 0;
  }
  __syncthreads();
  // What `n` units (at most kRound) have of candidates that can be among the first N, to the pool.  A slice has N logits that are no
  // less than the N-th largest of its lanes' largest (half as many lanes with a second one for more than 32): the best of those
  // marks is a floor.  Of logits that equal a slice's own mark N are enough.
  auto look_through = [&](const int* list, int n) {
    constexpr int kShare = kPickWarps / kRound;           // warps of a unit
    const int which = warp / kShare;
    const int u = which < n ? list[which] : 0, i = u / units, at = (u - i * units) * kBeamUnit + (warp % kShare) * kSlice + lane * 4;
    const bool open = which < n && s.kind[i] == 0;
    float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mark = -INFINITY, shift = 0.f;
    if (which < n && !open && warp % kShare == 0 && lane == 0) s.pool[atomicAdd(&s.count, 1)].order = order_of(i, 0.f, a.pad_token);
    if (open) {
      const uint8_t* row = static_cast<const uint8_t*>(row_of(a, (long long)b * K + i)) + (size_t)at * (BF16 ? 2 : 4);
      if (at + 4 <= a.vocab && (reinterpret_cast<uintptr_t>(row) & (BF16 ? 7 : 15)) == 0) {
        if constexpr (BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(row);
          x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(row);
          x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (at + j < a.vocab)
            x[j] = BF16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[j] << 16) : reinterpret_cast<const float*>(row)[j];
      }
      const float hi0 = fmaxf(x[0], x[1]), lo0 = fminf(x[0], x[1]), hi1 = fmaxf(x[2], x[3]), lo1 = fminf(x[2], x[3]);
      float y = N <= 32 ? fmaxf(hi0, hi1) : fmaxf(fminf(hi0, hi1), hi0 > hi1 ? lo0 : lo1);
      // the lanes' values in ascending order
#pragma unroll
      for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int d = k >> 1; d; d >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, y, d);
          y = ((lane & d) == 0) == ((lane & k) == 0) ? fminf(y, o) : fmaxf(y, o);
        }
      mark = __shfl_sync(0xffffffffu, y, 32 - (N <= 32 ? N : (N + 1) / 2));
      shift = s.score[i] - s.norm[i] - s.top[i];
    }
    // (float32 keys, with room for what they lose: the keys proper come later)
    const float slack = open ? 1e-6f * (fabsf(s.score[i]) + s.norm[i] + 2.f * fabsf(s.top[i]) + 1.f) : 0.f;
    if (lane == 0) s.mark[warp] = mark > -INFINITY ? mark + shift - slack - 1e-6f * fabsf(mark) : -INFINITY;
    __syncthreads();
    float floor = s.mark[lane];
#pragma unroll
    for (int d = 16; d; d >>= 1) floor = warp_max_xor(floor, d);
    if (s.floor.key) floor = fmaxf(floor, (float)from_ordered(s.floor.key));
    if (!open) return;
    const float least = floor == -INFINITY ? -3.402823466e38f : floor - shift - slack - 1e-6f * fabsf(floor);
    unsigned ties = 0, takes = 0;                         // of this lane's logits (a floor beyond float32's range, a NaN, stops none)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ties |= (unsigned)(x[j] == mark && x[j] > -INFINITY) << j;
      takes |= (unsigned)(!(x[j] < least) && x[j] > -INFINITY) << j;
    }
    ties &= takes;
    int scan = __popc(ties);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += o;
    }
    int before = scan - __popc(ties);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ties >> j & 1)
        if (before++ >= N) takes &= ~(1u << j);
    int mine = __popc(takes), sum = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    int to = 0;
    if (lane == 31 && sum > 0) to = atomicAdd(&s.count, sum);
    to = __shfl_sync(0xffffffffu, to, 31) + sum - mine;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (takes >> j & 1) s.pool[to++].order = order_of(i, x[j], at + j);
  };
  // The first N of the pool stay, in order; N of them are a floor.
  auto keep_first = [&]() {
    __syncthreads();
    const int count = s.count;
    for (int e = s.n_kept + tid; e < count; e += kPickThreads) {   // the new ones' keys
      const int i = beam_of(s.pool[e].order);
      s.pool[e].key = ordered(s.kind[i] == 1 ? (double)s.score[i] : key_of(s, i, logit_of(s.pool[e].order)));
    }
    __syncthreads();
    rank_entries(count, N, s.pool, [&](int place, int e) {
      s.kept[place] = s.pool[e];
      atomicMax(&s.n_kept, place + 1);
    });
    __syncthreads();
    const int kept = s.n_kept;
    if (tid < kept) s.pool[tid] = s.kept[tid];
    if (tid == 0) {
      s.count = kept;
      if (kept == N) s.floor = s.kept[N - 1];
    }
    __syncthreads();
  };
  for (int u0 = 0; u0 < total; u0 += kPickThreads) {
    // a thread's unit: its largest candidate's key, and how far float32 may be off
    const int u = u0 + tid, i = u < total ? u / units : 0, c = u - i * units;
    float top = 0.f, key = -INFINITY, off = 0.f;
    bool there = false;
    if (u < total && s.kind[i] == 0) {
      top = u0 == 0 ? own_top : part[u].x;
      there = top > -INFINITY;
      const float low = top - s.top[i];
      key = s.score[i] + (low - s.norm[i]);
      off = 1e-6f * (fabsf(s.score[i]) + fabsf(low) + s.norm[i] + fabsf(key) + 1.f);
    } else if (u < total && s.kind[i] == 1 && c == 0) {
      there = true;
      key = s.score[i];
    }
    if (u0 == 0) {  // the best units of the best groups of eight
      float best = there ? key : -INFINITY;
      int unit = u;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, best, d);
        const int other = __shfl_xor_sync(0xffffffffu, unit, d);
        if (o > best || (o == best && other < unit)) best = o, unit = other;
      }
      if ((tid & 7) == 0) {
        s.group[tid >> 3] = best;
        s.group_unit[tid >> 3] = unit;
      }
      __syncthreads();
      {
        const int e = tid >> 3;
        const float own = s.group[e];
        int before = 0;
#pragma unroll
        for (int o = tid & 7; o < kPickThreads / 8; o += 8) before += s.group[o] > own || (s.group[o] == own && o < e);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
        if ((tid & 7) == 0 && own > -INFINITY && before < kRound) {
          s.first[before] = s.group_unit[e];
          atomicMax(&s.n_first, before + 1);
        }
      }
      __syncthreads();
      look_through(s.first, s.n_first);
      keep_first();
      for (int k = 0; k < s.n_first; ++k) there &= s.first[k] != u;  // (done)
    }
    if (tid == 0) s.n_unit = 0;
    __syncthreads();
    const Entry floor = s.floor;
    bool look = there;
    if (there && floor.key) {
      const float f = (float)from_ordered(floor.key);
      off += 1e-6f * fabsf(f);
      look = key >= f - off;
      if (look && key <= f + off)
        look = !floor.before(Entry{ordered(s.kind[i] == 1 ? (double)s.score[i] : key_of(s, i, top)), order_of(i, top, c * kBeamUnit)});
    }
    const unsigned some = __ballot_sync(0xffffffffu, look);
    if (some) {
      int to = 0;
      if (lane == 0) to = atomicAdd(&s.n_unit, __popc(some));
      to = __shfl_sync(0xffffffffu, to, 0) + __popc(some & ((1u << lane) - 1));
      if (look) s.unit[to] = u;
    }
    __syncthreads();
    const int n_unit = s.n_unit;
    for (int r = 0; r < n_unit; r += kRound) {
      look_through(s.unit + r, min(n_unit - r, kRound));
      keep_first();
    }
  }
  if (tid < N) {
    const bool some = tid < s.n_kept;
    const long long at = (long long)b * N + tid;
    const Entry e = some ? s.kept[tid] : Entry{0, 0};
    a.out_scores[at] = some ? (float)from_ordered(e.key) : -INFINITY;
    a.out_tokens[at] = some ? token_of(e.order) : -1;
    a.out_parents[at] = some ? beam_of(e.order) : -1;
  }
}

}  // namespace

int launch_beam_units(const BeamArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long all = (long long)a.batch * a.beams * beam_units(a.vocab), per = kUnitThreads / 32;
  const dim3 grid((unsigned)((all + per - 1) / per));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kUnitThreads), 0, s, pdl, a); };
  return a.dtype == kDtypeBF16 ? go(beam_unit_kernel<true>) : go(beam_unit_kernel<false>);
}

int launch_beam_pick(const BeamArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kern) {
    const cudaError_t e = ensure_smem_limit(kern, sizeof(PickSmem));
    if (e != cudaSuccess) return (int)e;
    return launch_pdl(kern, dim3(a.batch), dim3(kPickThreads), sizeof(PickSmem), s, pdl, a);
  };
  return a.dtype == kDtypeBF16 ? go(beam_pick_kernel<true>) : go(beam_pick_kernel<false>);
}

}  // namespace oscar
