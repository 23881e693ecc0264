// The next beams of a beam search: of an item's beams x vocabulary candidates
//
//     key(i, v) = score_i + ((x_iv - m_i) - log sum_u e^{x_iu - m_i}),  m_i = max_u x_iu,
//
// the n_out largest, the lowest i V + v first among equal ones.
//
// The logits are read once.  A first kernel leaves the maximum and the sum of exponentials of every chunk of a row; it is bound
// by memory (2 or 4 bytes and some six instructions a logit).  A second one, a CTA per item, forms the rows' normalisers and
// ranks the (beam, chunk) pairs by the key of their largest logit.  The n_out best candidates lie in the n_out first pairs: if
// a candidate's pair came later, n_out pairs before it each had a candidate, their largest, that comes before it too (its key is
// larger, or equal with a larger logit of the same beam or a lower index, chunks being ranges of ascending index).  So only n_out chunks are looked through again.
#include "beam_internal.h"
#include "common.cuh"

namespace oscar {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Logits [i, i + N) of a row as float32, N adjacent ones that make 16 bytes; -infinity from the vocabulary's end on.  Which
// logits a thread takes does not depend on the row's alignment, so equal rows have equal sums.
template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;
  float v[N];
  __device__ __forceinline__ void load(const void* row, int i, int vocab, bool aligned) {
    if (aligned && i + N <= vocab) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (size_t)i * (BF16 ? 2 : 4));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
          v[2 * k] = bf16_lo(w[k]);
          v[2 * k + 1] = bf16_hi(w[k]);
        } else {
          v[k] = __uint_as_float(w[k]);
        }
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = -INFINITY;
      if (i + k < vocab)
        v[k] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(row)[i + k] << 16) : static_cast<const float*>(row)[i + k];
    }
  }
};

__device__ __forceinline__ const void* row_of(const BeamArgs& a, long long row) {
  return static_cast<const uint8_t*>(a.logits) + row * a.stride * (a.dtype == kDtypeBF16 ? 2 : 4);
}

// (m, s) and (m2, s2) as one: sums of 2^((x - m) log2 e).  A NaN stays one.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2), ref = top == -INFINITY ? 0.f : top;
  s = s * ex2((m - ref) * kLog2e) + s2 * ex2((m2 - ref) * kLog2e);
  m = top;
}

// ------------------------------------------------------------------ chunks
constexpr int kChunkThreads = 128;

template <bool BF16>
__global__ void __launch_bounds__(kChunkThreads) beam_chunk_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<BF16>;
  __shared__ float2 s_part[kChunkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long row = blockIdx.x / a.plan.chunks;
  const int c = blockIdx.x % a.plan.chunks;
  pdl_wait();
  pdl_launch_dependents();
  if (a.finished && a.finished[row]) return;
  const void* x = row_of(a, row);
  const bool aligned = (reinterpret_cast<uintptr_t>(x) & 15) == 0;
  const int end = (int)min((long long)(c + 1) * a.plan.chunk, (long long)a.vocab);
  float m = -INFINITY, s = 0.f;
  constexpr int kAhead = 4, kStep = kChunkThreads * V::N;
  for (int i0 = c * a.plan.chunk + tid * V::N; i0 < end; i0 += kAhead * kStep) {
    V v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k].load(x, i0 + k * kStep, end, aligned);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float top = m;
#pragma unroll
      for (int j = 0; j < V::N; ++j) top = fmaxf(top, v[k].v[j]);
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V::N; ++j) sum += ex2((v[k].v[j] - ref) * kLog2e);   // (a NaN or +infinity makes a NaN of it)
      s = fmaf(s, ex2((m - ref) * kLog2e), sum);
      m = top;
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) join(m, s, __shfl_xor_sync(0xffffffffu, m, d), __shfl_xor_sync(0xffffffffu, s, d));
  if (lane == 0) s_part[tid >> 5] = make_float2(m, s);
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kChunkThreads / 32; ++w) join(m, s, s_part[w].x, s_part[w].y);
    reinterpret_cast<float2*>(a.part)[row * a.plan.chunks + c] = make_float2(m, s);
  }
}

// ------------------------------------------------------------------ candidates
constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32;
constexpr int kRoom = kMaxCandidates * (kPickWarps + 1);   // candidates at hand: those kept and a warp's most

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
__device__ __forceinline__ int token_of(unsigned long long order) { return kMaxVocab - 1 - (int)(order & (kMaxVocab - 1)); }

struct PickSmem {
  unsigned long long pair_key[kMaxPairs], pair_order[kMaxPairs];
  unsigned long long key[kRoom], kept_key[kMaxCandidates];
  unsigned long long order[kRoom], kept_order[kMaxCandidates];
  int sel[kMaxCandidates];
  double norm[kMaxBeams];     // log of the sum of exponentials
  float top[kMaxBeams];       // m_i
  float score[kMaxBeams];
  int kind[kMaxBeams];        // 0: open, 1: finished, 2: no candidates
  int n_sel, count, kept;
};

__device__ __forceinline__ double key_of(const PickSmem& s, int i, float x) {
  return (double)s.score[i] + (((double)x - (double)s.top[i]) - s.norm[i]);
}

// Places of n entries among themselves, the largest (key, order) first; the first `most` of them are handed to put(place, entry).
template <typename Put>
__device__ __forceinline__ void rank_entries(int n, int most, const unsigned long long* key, const unsigned long long* order, Put put) {
  for (int e = threadIdx.x; e < n; e += kPickThreads) {
    const unsigned long long k = key[e];
    if (k == 0) continue;
    const unsigned long long at = order[e];
    int before = 0;
    for (int o = 0; o < n && before < most; ++o) {
      const unsigned long long ko = key[o];
      before += ko > k || (ko == k && order[o] > at);
    }
    if (before < most) put(before, e);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const __grid_constant__ BeamArgs a) {
  using V = Vec<BF16>;
  constexpr int kVecs = kBeamUnit / (32 * V::N);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PickSmem& s = *reinterpret_cast<PickSmem*>(smem_raw);
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int K = a.beams, chunks = a.plan.chunks, N = a.n_out;
  pdl_wait();
  pdl_launch_dependents();
  // the rows' normalisers
  for (int i = warp; i < K; i += kPickWarps) {
    const long long row = (long long)b * K + i;
    const float score = a.scores[row];
    int kind = a.finished && a.finished[row] ? 1 : 0;
    bool sound = score < INFINITY;                       // (false for a NaN)
    float m = -INFINITY;
    double sum = 0.0;
    if (kind == 0) {
      const float2* part = reinterpret_cast<const float2*>(a.part) + row * chunks;
      for (int c = lane; c < chunks; c += 32) {
        const float2 p = part[c];
        m = fmaxf(m, p.x);
        sound &= p.y == p.y;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) m = warp_max_xor(m, d);
      if (m > -INFINITY)
        for (int c = lane; c < chunks; c += 32) sum += (double)part[c].y * (double)expf(part[c].x - m);
#pragma unroll
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (m == -INFINITY) kind = 2;
    }
    sound = __all_sync(0xffffffffu, sound);
    if (!sound || score == -INFINITY) kind = 2;
    if (lane == 0) {
      if (!sound) flag_error(a.status, kDevBadValue);
      s.score[i] = score;
      s.top[i] = m;
      s.norm[i] = kind == 0 ? log(sum) : 0.0;
      s.kind[i] = kind;
    }
  }
  if (tid == 0) s.n_sel = s.count = s.kept = 0;
  __syncthreads();
  // the best pairs
  const int pairs = K * chunks;
  for (int p = tid; p < pairs; p += kPickThreads) {
    const int i = p / chunks, c = p % chunks;
    unsigned long long k = 0;
    float top = 0.f;
    if (s.kind[i] == 0) {
      top = a.part[2 * (((long long)b * K + i) * chunks + c)];
      k = ordered(key_of(s, i, top));
    }
    if (s.kind[i] == 1 && c == 0) k = ordered((double)s.score[i]);
    s.pair_key[p] = k;
    s.pair_order[p] = order_of(i, top, c);
  }
  __syncthreads();
  rank_entries(pairs, N, s.pair_key, s.pair_order, [&](int place, int e) {
    s.sel[place] = e;
    atomicMax(&s.n_sel, place + 1);
  });
  __syncthreads();
  const int n_sel = s.n_sel;
  // the candidates in them, a unit a warp and round; `floor`: what a candidate needs to be among the first N
  unsigned long long floor = n_sel == N ? s.pair_key[s.sel[N - 1]] : 0;
  const int per = a.plan.chunk / kBeamUnit, units = n_sel * per;
  for (int u0 = 0; u0 < units; u0 += kPickWarps) {
    const int u = u0 + warp;
    if (u < units) {
      const int p = s.sel[u / per], i = p / chunks, at = (p % chunks) * a.plan.chunk + (u % per) * kBeamUnit;
      if (s.kind[i] == 1) {
        if (u % per == 0 && lane == 0) {
          const int to = atomicAdd(&s.count, 1);
          s.key[to] = s.pair_key[p];
          s.order[to] = order_of(i, 0.f, a.pad_token);
        }
      } else if (at < a.vocab) {
        const void* row = row_of(a, (long long)b * K + i);
        const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
        V v[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k) v[k].load(row, at + (k * 32 + lane) * V::N, a.vocab, aligned);
        // the least logit whose key can reach the floor, a little below it
        float least = -3.402823466e38f;
        if (floor) {
          const double t = ((from_ordered(floor) - (double)s.score[i]) + s.norm[i]) + (double)s.top[i];
          least = fmaxf(least, __double2float_rd(t - fabs(t) * 1e-14 - 1e-12));
        }
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
          for (int j = 0; j < V::N; ++j) mine += v[k].v[j] >= least;
        const int all = __reduce_add_sync(0xffffffffu, mine);
        if (all > 0 && all <= kMaxCandidates) {
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
#pragma unroll
          for (int k = 0; k < kVecs; ++k)
#pragma unroll
            for (int j = 0; j < V::N; ++j)
              if (v[k].v[j] >= least) {
                s.key[to] = ordered(key_of(s, i, v[k].v[j]));
                s.order[to++] = order_of(i, v[k].v[j], at + (k * 32 + lane) * V::N + j);
              }
        } else if (all > 0) {  // more than can be among the first: the unit's N first, one after another
          for (int r = 0; r < N; ++r) {
            float top = -INFINITY;
            int where = 0x7fffffff;
#pragma unroll
            for (int k = 0; k < kVecs; ++k)
#pragma unroll
              for (int j = 0; j < V::N; ++j)
                if (v[k].v[j] > top) top = v[k].v[j], where = at + (k * 32 + lane) * V::N + j;
            float best = top;
#pragma unroll
            for (int d = 16; d; d >>= 1) best = warp_max_xor(best, d);
            const int first = __reduce_min_sync(0xffffffffu, top == best ? where : 0x7fffffff);
            if (!(best >= least)) break;
            if (top == best && where == first) {
#pragma unroll
              for (int k = 0; k < kVecs; ++k)
#pragma unroll
                for (int j = 0; j < V::N; ++j)
                  if (at + (k * 32 + lane) * V::N + j == first) v[k].v[j] = -INFINITY;
              const int to = atomicAdd(&s.count, 1);
              s.key[to] = ordered(key_of(s, i, best));
              s.order[to] = order_of(i, best, first);
            }
            __syncwarp();
          }
        }
      }
    }
    __syncthreads();
    const int count = s.count;
    rank_entries(count, N, s.key, s.order, [&](int place, int e) {
      s.kept_key[place] = s.key[e];
      s.kept_order[place] = s.order[e];
      atomicMax(&s.kept, place + 1);
    });
    __syncthreads();
    const int kept = s.kept;
    if (tid < kept) {
      s.key[tid] = s.kept_key[tid];
      s.order[tid] = s.kept_order[tid];
    }
    if (tid == 0) s.count = kept;
    if (kept == N) floor = s.kept_key[N - 1];
    __syncthreads();
  }
  if (tid < N) {
    const bool some = tid < s.kept;
    const long long at = (long long)b * N + tid;
    const unsigned long long order = some ? s.kept_order[tid] : 0;
    a.out_scores[at] = some ? (float)from_ordered(s.kept_key[tid]) : -INFINITY;
    a.out_tokens[at] = some ? token_of(order) : -1;
    a.out_parents[at] = some ? beam_of(order) : -1;
  }
}

}  // namespace

BeamPlan beam_plan(int batch, int beams, int vocab, int n_out) {
  // Ranking p pairs takes p p / 26 clocks or so, looking through n chunks of c logits n c / 32: the chunk that makes the sum
  // smallest.
  BeamPlan best{};
  double least = -1.0;
  for (long long c = kBeamUnit; c <= 2LL * kMaxVocab; c *= 2) {
    const long long chunks = (vocab + c - 1) / c, p = beams * chunks;
    if (p > kMaxPairs) continue;
    const double cost = (double)p * p / 26.0 + (double)(n_out < p ? n_out : p) * c / 32.0;
    if (least < 0.0 || cost < least) {
      least = cost;
      best.chunk = (int)c;
      best.chunks = (int)chunks;
    }
  }
  best.total = (size_t)batch * beams * best.chunks * 2 * sizeof(float);
  return best;
}

int launch_beam_chunks(const BeamArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)((long long)a.batch * a.beams * a.plan.chunks));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kChunkThreads), 0, s, pdl, a); };
  return a.dtype == kDtypeBF16 ? go(beam_chunk_kernel<true>) : go(beam_chunk_kernel<false>);
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
