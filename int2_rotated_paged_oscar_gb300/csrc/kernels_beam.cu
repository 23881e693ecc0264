// The next beams of a beam search: of an item's beams x vocabulary candidates
//
//     key(i, v) = score_i + ((x_iv - m_i) - log sum_u e^{x_iu - m_i}),  m_i = max_u x_iu,
//
// the n_out largest, the lowest i V + v first among equal ones.
//
// The logits are read once.  A first kernel, a warp per unit of 1024 logits, leaves the unit's maximum and sum of exponentials; it is
// bound by memory (2 or 4 bytes and some five instructions a logit).  A second one, a CTA per item, forms the rows' normalisers and
// looks through the best few units once more; then through those others whose largest candidate comes before the last of the
// n_out at hand.
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

template <bool BF16>
__global__ void __launch_bounds__(kUnitThreads) beam_unit_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<BF16>;
  constexpr int kVecs = kBeamUnit / (32 * V::N);
  const int lane = threadIdx.x & 31, units = beam_units(a.vocab);
  const long long at = (long long)blockIdx.x * (kUnitThreads / 32) + (threadIdx.x >> 5), row = at / units;
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
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int j = 0; j < V::N; ++j) m = fmaxf(m, v[k].get(j));
#pragma unroll
  for (int d = 16; d; d >>= 1) m = warp_max_xor(m, d);
  const float ref = m == -INFINITY ? 0.f : m;
  float s[4] = {0.f, 0.f, 0.f, 0.f};                      // (a NaN or +infinity makes a NaN of it)
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int j = 0; j < V::N; ++j) s[j & 3] += ex2((v[k].get(j) - ref) * kLog2e);
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) reinterpret_cast<float2*>(a.part)[at] = make_float2(m, sum);
}

// ------------------------------------------------------------------ candidates
constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32;
constexpr int kMostPushed = 128;                           // candidates that a warp hands in of a unit
constexpr int kRoom = kMaxCandidates + kPickWarps * kMostPushed;   // candidates at hand: those kept and the warps' most
constexpr int kFirst = 4;                                  // units that are looked through first

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
  Entry group[kPickThreads / 8];
  int group_unit[kPickThreads / 8], first[kFirst];
  double norm[kMaxBeams];     // log of the sum of exponentials
  float top[kMaxBeams];       // m_i
  float score[kMaxBeams];
  int kind[kMaxBeams];        // 0: open, 1: finished, 2: no candidates
  int unit[kPickThreads];     // units to look through
  Entry floor;                // what a candidate has to come before, or be
  int n_unit, n_first, count, n_kept;
};

__device__ __forceinline__ double key_of(const PickSmem& s, int i, float x) {
  return (double)s.score[i] + (((double)x - (double)s.top[i]) - s.norm[i]);
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
  using V = Vec<BF16>;
  constexpr int kVecs = kBeamUnit / (32 * V::N);
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
    double sum = 0.0;
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
        for (int k = 0; k < kHold; ++k) sum += (double)(p[k].y * expf(p[k].x - m));
        for (int c = lane + 32 * kHold; c < units; c += 32) sum += (double)(mine[c].y * expf(mine[c].x - m));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (m == -INFINITY) kind = 2;
    }
    sound = __all_sync(0xffffffffu, sound);
    if (!sound || score == -INFINITY) kind = 2;
    if (lane == 0) {
      if (!sound) flag_error(a.status, kDevBadValue);
      // log of the sum: float32's, and a Newton step for what it leaves out
      const float total = (float)sum, y = logf(total), rest = fmaf(total, expf(-y), -1.f);
      s.score[i] = score;
      s.top[i] = m;
      s.norm[i] = kind == 0 ? (double)y + (double)rest : 0.0;
      s.kind[i] = kind;
    }
  }
  if (tid == 0) {
    s.floor = Entry{0, 0};
    s.count = s.n_kept = s.n_first = 0;
  }
  __syncthreads();
  // What a unit has of candidates that can be among the first N, to the pool.  At least N of its logits are no less than the N-th
  // largest of its lanes' largest (or half as many lanes have a second one of at least that): those before the floor among
  // them, unless equal ones make them too many.
  auto look_through = [&](int u) {
    const Entry floor = s.floor;
    const int i = u / units, at = (u - i * units) * kBeamUnit;
    if (s.kind[i] == 1) {
      if (lane == 0) s.pool[atomicAdd(&s.count, 1)].order = order_of(i, 0.f, a.pad_token);
      return;
    }
    const void* row = row_of(a, (long long)b * K + i);
    const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    V v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k].load(row, at + (k * 32 + lane) * V::N, a.vocab, aligned);
    float one = -INFINITY, two = -INFINITY;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        const float x = v[k].get(j);
        two = fmaxf(two, fminf(one, x));
        one = fmaxf(one, x);
      }
    const float mark = N <= 32 ? one : two;
    const int need = N <= 32 ? N : (N + 1) / 2;
    int before = 0;
#pragma unroll
    for (int d = 1; d < 32; ++d) {
      const int from = (lane + d) & 31;
      const float o = __shfl_sync(0xffffffffu, mark, from);
      before += o > mark || (o == mark && from < lane);
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, before == need - 1)) - 1;
    // the least logit whose key can reach the floor, a little below it
    float least = fmaxf(-3.402823466e38f, __shfl_sync(0xffffffffu, mark, src));
    if (floor.key) {
      const double t = ((from_ordered(floor.key) - (double)s.score[i]) + s.norm[i]) + (double)s.top[i];
      least = fmaxf(least, __double2float_rd(t - fabs(t) * 1e-14 - 1e-12));
    }
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
#pragma unroll
      for (int j = 0; j < V::N; ++j) mine += v[k].get(j) >= least;
    const int all = __reduce_add_sync(0xffffffffu, mine);
    if (all == 0) return;
    if (all <= kMostPushed) {
      int to = 0;
      if (lane == 0) to = atomicAdd(&s.count, all);
      to = __shfl_sync(0xffffffffu, to, 0);
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      to += sum - mine;
      if (mine > 0)
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
          for (int j = 0; j < V::N; ++j)
            if (v[k].get(j) >= least)
              s.pool[to++].order = order_of(i, v[k].get(j), at + (k * 32 + lane) * V::N + j);
      return;
    }
    float last = INFINITY;                                // the unit's N first, one after another
    int after = -1;
    for (int n = 0; n < N; ++n) {
      float top = -INFINITY;
      int where = 0x7fffffff;
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          const float x = v[k].get(j);
          const int p = at + (k * 32 + lane) * V::N + j;
          if (x > top && (x < last || (x == last && p > after))) top = x, where = p;
        }
      float best = top;
#pragma unroll
      for (int d = 16; d; d >>= 1) best = warp_max_xor(best, d);
      const int first = __reduce_min_sync(0xffffffffu, top == best ? where : 0x7fffffff);
      if (!(best >= least)) break;
      if (lane == 0) s.pool[atomicAdd(&s.count, 1)].order = order_of(i, best, first);
      last = best, after = first;
    }
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
    // a thread's unit: its largest candidate
    const int u = u0 + tid, i = u < total ? u / units : 0, c = u - i * units;
    Entry mine{0, 0};
    if (u < total && s.kind[i] == 0) {
      const float top = u0 == 0 ? own_top : part[u].x;
      mine = Entry{ordered(key_of(s, i, top)), order_of(i, top, c * kBeamUnit)};
    } else if (u < total && s.kind[i] == 1 && c == 0) {
      mine = Entry{ordered((double)s.score[i]), order_of(i, 0.f, 0)};
    }
    if (u0 == 0) {  // the best units of the best groups of eight
      Entry best = mine;
      int unit = u;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        const Entry o{__shfl_xor_sync(0xffffffffu, best.key, d), __shfl_xor_sync(0xffffffffu, best.order, d)};
        const int other = __shfl_xor_sync(0xffffffffu, unit, d);
        if (o.before(best)) best = o, unit = other;
      }
      if ((tid & 7) == 0) {
        s.group[tid >> 3] = best;
        s.group_unit[tid >> 3] = unit;
      }
      __syncthreads();
      const int groups = (min(total, kPickThreads) + 7) / 8;
      rank_entries(groups, kFirst, s.group, [&](int place, int e) {
        s.first[place] = s.group_unit[e];
        atomicMax(&s.n_first, place + 1);
      });
      __syncthreads();
      if (warp < s.n_first) look_through(s.first[warp]);
      keep_first();
      for (int k = 0; k < s.n_first; ++k)
        if (s.first[k] == u) mine.key = 0;                // (done)
    }
    if (tid == 0) s.n_unit = 0;
    __syncthreads();
    const bool look = mine.key != 0 && !s.floor.before(mine);
    const unsigned some = __ballot_sync(0xffffffffu, look);
    if (some) {
      int to = 0;
      if (lane == 0) to = atomicAdd(&s.n_unit, __popc(some));
      to = __shfl_sync(0xffffffffu, to, 0) + __popc(some & ((1u << lane) - 1));
      if (look) s.unit[to] = u;
    }
    __syncthreads();
    const int n_unit = s.n_unit;
    for (int r = 0; r < n_unit; r += kPickWarps) {
      if (r + warp < n_unit) look_through(s.unit[r + warp]);
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
