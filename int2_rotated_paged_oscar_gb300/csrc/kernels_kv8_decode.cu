// Decode attention over the 8-bit cache: every complete page of a request, or a selected list of them
// per kv head, and the BF16 tail rows of the page that is not complete.
//
// o = softmax(q K^T / sqrt d) V is split along the tokens: CTA (split, kv head, request) reads its pages
// once for all query heads of the kv head and leaves (m, l, acc) with weights 2^(s - m); a second kernel
// merges the partials.  What it must read is 2 d bytes per token and kv head, so it is bound by memory;
// 4 d flops per token and query head run on the tensor cores.
//
// A CTA has one producer warp and four consumer warps around a ring of stages of 64 tokens (128 at
// d = 64 and P >= 32; each page one bulk copy of codes and scales).  A consumer warp takes a quarter of a stage,
// one block of 16 tokens or two of one page:
//   scores: A = 16 tokens x 16 channels of codes, B = the query as f16 (a power of two brings its largest
//           component to 2^14; BF16 queries are exact in one f16 down to 2^-28 of it, float32 ones take two);
//           channels are taken in the order in which a lane's 16-byte loads hold them.
//   values: A = 16 channels x 16 tokens of codes, B = the weights as f16 high and low halves (24 bits
//           relative to the blocks' largest).
// Codes are exact f16 numbers, so the only roundings are float32's, but for a query's components far below its largest one; where
// those decide, the split is taken again in plain float32 (plain_split).  The block's scales multiply scores
// and sums in float32, and the weights are relative to the maximum of a warp's own blocks, all of one page, so a quiet page
// next to a loud one keeps its digits.  A token's distance from that maximum is formed from the raw sums, before any scale:
// it is 0 at the maximum and below 0 elsewhere whatever the scores' size, so no weight leaves [0, 1].  The tail rows go the same way with BF16 operands, 16 rows a warp, in the CTA of the
// request's last pages while its first pages are on their way.
//
// Measured (8 kv heads of 128 channels, pages of 64, layers larger than L2): batch 1 at 32K, INT8, 4 heads a kv head 16.9 us
// (67 MB, 0.59 of the measured copy bandwidth: the start, the end and the merge take 7 us); 64 requests of 8K to 32K, E4M3,
// 8 heads a kv head 434 us (2.7 GB, 0.91).  32 requests of 8K to 16K at d = 64: 0.75 to 0.81 with up to four heads a kv head,
// 0.66 to 0.71 with eight; with pages of 16, half again as many instructions a byte, 0.62 to 0.68 and 0.55 to 0.59.  Not kept, at the 64 requests: CTAs that stay and take one split after another through the same
// ring, the next split's pages ahead (468 us: the warps wait at every split's end); four CTAs an SM with three stages
// (531); two with six (451); a rescaling of the sums only where a maximum moved (434).
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
// log2(e) / sqrt(d) as two floats: a score is far larger than its distance from the largest one, which is what counts, so
// scale and distance are formed without a rounding of the score itself; what the rounding of the largest one's logarithm
// leaves out goes into its block's weight.
template <int D>
struct Scale {
  static constexpr double kValue = 1.4426950408889634 / (D == 128 ? 11.313708498984761 : 8.0);
  static constexpr float hi = (float)kValue, lo = (float)(kValue - (double)(float)kValue);
};

// CTAs an SM: four where their stages are small or, with fewer heads' sums, their registers few.  (d = 64, P = 64, 32 requests
// of 8K to 16K tokens: up to four heads 72 us with four CTAs of three stages, 75 with three of four; eight heads 87 and 85,
// in float32 98 and 86.)
OSCAR_HD constexpr int resident(int D, int stage_tokens, bool g8) { return D == 64 && !(stage_tokens == 128 && g8) ? 4 : 3; }

// NB: blocks of 16 tokens that a warp takes of a stage.
template <int D, int NB, bool G8>
struct Layout {
  static constexpr int kTokens = 64 * NB;
  static constexpr int kResident = resident(D, kTokens, G8);
  static constexpr int kStages = NB == 2 && kResident == 4 ? 3 : 4;
  static constexpr int kPad = 128;  // scales, and the 128-byte alignment of the next page
  OSCAR_HD static int page_stride(int P) { return 2 * P * D + kPad; }
  OSCAR_HD static int stage_bytes(int P) { return (kTokens / P) * page_stride(P); }
  static size_t smem(int P) {
    const size_t ring = (size_t)kStages * stage_bytes(P);
    const size_t merge = kConsumers * 8 * (D + 2) * sizeof(float);
    return (ring > merge ? ring : merge) + 128;
  }
};

// A block's largest raw sum cm times f = fh + fl, the scale of a score: m is the product rounded down, over(r) the product
// less r to float32's digits, with r the larger of m and another block's.  A weight 2^over(r) is that of the exact product.
// Where scores are so large, 2^28 and more, that a last place of one is many units, it stays a finite number (64 at most), and
// where r is m it is no less than 1 but for roundings of the difference itself.
struct Top {
  float cm, fh, fl, m;
  __device__ __forceinline__ Top(float c, float h, float l) : cm(c), fh(h), fl(l) { m = __fmaf_rd(c, h, c * l); }
  __device__ __forceinline__ float over(float r) const { return fminf(fmaf(cm, fl, fmaf(cm, fh, -r)), 64.f); }
};

__device__ __forceinline__ bool length_ok(const Kv8DecodeArgs& a, int n) {
  return n >= 0 && n <= (a.page_idx ? (long long)a.g.max_pages_per_req * a.g.P : (long long)a.max_seq);
}

// Partial of a split (m, l, -, -, acc[D]).
__device__ __forceinline__ float* partial(const Kv8DecodeArgs& a, int b, int head, int split, int D) {
  return a.part + (((size_t)b * a.g.Hq + head) * a.wl.max_splits + split) * (D + 4);
}

__device__ __forceinline__ void store_out(const Kv8DecodeArgs& a, size_t i, float y) {
  if (a.out_dtype == kDtypeBF16) static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(y);
  else static_cast<float*>(a.out)[i] = y;
}

// Splits of a request with `have` page entries: one at least, for its tail.
__device__ __forceinline__ int split_count(const Kv8DecodeArgs& a, int have) {
  const int per = a.wl.stages_per_split * (kv8_stage_tokens(a.g.D, a.g.P) / a.g.P);
  return max((have + per - 1) / per, 1);
}

// The tail's K rows of request b and kv head h (the V rows follow P rows on); null for a bad slot.
__device__ __forceinline__ const uint16_t* tail_of(const Kv8DecodeArgs& a, int b, int h) {
  const Geom& g = a.g;
  const int slot = a.req_slot[b];
  if (slot < 0 || slot >= g.max_req) return nullptr;
  return a.tail + ((size_t)a.layer * g.max_req + slot) * kv8_tail_req_elems(g) + (size_t)h * 2 * g.P * g.D;
}

// x, y as three BF16 pairs whose sum has float32's digits.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = pack_bf162(x, y);
    x -= bf16_lo(t[i]);
    y -= bf16_hi(t[i]);
  }
}

// ------------------------------------------------------------------ tail rows
// 16 BF16 rows of the tail (cnt of them there) as a warp's first block: m, l, acc as the page loop goes on with them.
// Keys and values are BF16 operands as they are, queries and weights sums of up to three.
template <int D, bool G8, bool QF32, int NH>
__device__ __forceinline__ void tail_block(const Kv8DecodeArgs& a, int b, int h, const uint16_t* krows, const uint16_t* vrows, int cnt,
                                           float (&m_run)[NH], float (&l_run)[NH], float (&acc)[D / 16][2 * NH]) {
  constexpr int KS = D / 16;
  const int G = a.g.gq(), lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int head = G8 ? gid : gid >> 1;
  const bool odd = !G8 && (gid & 1), live = head < G;
  const size_t qat = (size_t)b * a.q_stride + (size_t)(h * G + (live ? head : 0)) * D;
  const uint4 none = make_uint4(0, 0, 0, 0);
  float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {   // 32 channels: two k-steps from 16 bytes a lane
    const int ch = c * 32 + tig * 8;
    const uint4 k0 = gid < cnt ? *reinterpret_cast<const uint4*>(krows + (size_t)gid * D + ch) : none;
    const uint4 k1 = gid + 8 < cnt ? *reinterpret_cast<const uint4*>(krows + (size_t)(gid + 8) * D + ch) : none;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float4 q = kv8_load4<QF32>(a.q, qat + ch + 4 * u);
      if (!live) q = make_float4(0.f, 0.f, 0.f, 0.f);
      const uint32_t a0 = u ? k0.z : k0.x, a2 = u ? k0.w : k0.y, a1 = u ? k1.z : k1.x, a3 = u ? k1.w : k1.y;
      if constexpr (QF32) {
        uint32_t x[3], y[3];
        split3(q.x, q.y, x);
        split3(q.z, q.w, y);
        if constexpr (G8) {
#pragma unroll
          for (int i = 0; i < 3; ++i) mma_bf16(sc, a0, a1, a2, a3, x[i], y[i]);
        } else {
          mma_bf16(sc, a0, a1, a2, a3, odd ? x[1] : x[0], odd ? y[1] : y[0]);
          mma_bf16(sc, a0, a1, a2, a3, odd ? 0u : x[2], odd ? 0u : y[2]);
        }
      } else {
        const uint32_t x = odd ? 0u : pack_bf162(q.x, q.y), y = odd ? 0u : pack_bf162(q.z, q.w);
        mma_bf16(sc, a0, a1, a2, a3, x, y);
      }
    }
  }
  uint32_t pb[3][2];
  float pr[NH][2];
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    // (BF16 queries leave their odd columns empty: an infinite key times their 0 would be NaN)
    const float ca = G8 ? sc[i] : QF32 ? sc[0] + sc[1] : sc[0], cb = G8 ? sc[2 + i] : QF32 ? sc[2] + sc[3] : sc[2];
    float cm = fmaxf(gid < cnt ? ca : -INFINITY, gid + 8 < cnt ? cb : -INFINITY);
    cm = warp_max_xor(cm, 4);
    cm = warp_max_xor(cm, 8);
    cm = warp_max_xor(cm, 16);
    const Top top(cm, Scale<D>::hi, Scale<D>::lo);
    const float r = top.over(top.m);
    const float da = ca - cm, db = cb - cm;
    pr[i][0] = gid < cnt ? ex2(fmaf(da, Scale<D>::hi, fmaf(da, Scale<D>::lo, r))) : 0.f;
    pr[i][1] = gid + 8 < cnt ? ex2(fmaf(db, Scale<D>::hi, fmaf(db, Scale<D>::lo, r))) : 0.f;
    m_run[i] = top.m;
    l_run[i] = pr[i][0] + pr[i][1];
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    uint32_t t[3];
    if constexpr (G8) {
      split3(pr[0][r], pr[1][r], t);
    } else {  // columns 2 h, 2 h + 1: the first and second part of head h's weight; then the third
      split3(pr[0][r], 0.f, t);
      t[0] = (t[0] & 0xffffu) | (t[1] << 16);
      t[1] = t[2] & 0xffffu;
    }
#pragma unroll
    for (int i = 0; i < (G8 ? 3 : 2); ++i) pb[i][r] = transpose_8x8(t[i]);
  }
  // values: rows 2 tig (+ 1, + 8, + 9), channels gid D / 8 and on
  uint32_t vw[4][KS];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = 2 * tig + (j & 1) + 8 * (j >> 1);
#pragma unroll
    for (int c = 0; c < KS / 4; ++c) {
      const uint4 v = t < cnt ? *reinterpret_cast<const uint4*>(vrows + (size_t)t * D + gid * (D / 8) + 8 * c) : none;
      vw[j][4 * c] = v.x, vw[j][4 * c + 1] = v.y, vw[j][4 * c + 2] = v.z, vw[j][4 * c + 3] = v.w;
    }
  }
#pragma unroll
  for (int mt = 0; mt < KS; ++mt) {
    const uint32_t a0 = prmt(vw[0][mt], vw[1][mt], 0x5410u), a1 = prmt(vw[0][mt], vw[1][mt], 0x7632u);
    const uint32_t a2 = prmt(vw[2][mt], vw[3][mt], 0x5410u), a3 = prmt(vw[2][mt], vw[3][mt], 0x7632u);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < (G8 ? 3 : 2); ++i) mma_bf16(o, a0, a1, a2, a3, pb[i][0], pb[i][1]);
    if constexpr (G8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][i] = o[i];
    } else {
      acc[mt][0] = o[0] + o[1];
      acc[mt][1] = o[2] + o[3];
    }
  }
}

// ------------------------------------------------------------------ a split in plain float32
// A query component is held to 2^-25 (its head's largest being 2^14 to 2^15), so a raw sum to L = D M 2^-25, M the largest
// code, and a score of scale f to L f.  That is no more than 2^-20 while f <= 32 / (D M); and it is below 2^-18 of the sum's own
// terms, a float32 sum's error, where the sums whose weights count, those down to 30 / f below the largest one cm, are not
// near 0: |cm| >= 2 D M > D M / 128 + 30 / f.  A block that meets neither has keys of 0 under the loudest components of a query
// whose quiet ones still decide its weights.
template <int D, int FMT>
__device__ __forceinline__ bool digits_lost(float f, float cm) {
  constexpr float kSum = D * (FMT == kKv8Int8 ? 127.f : 448.f);
  return f > 32.f / kSum && fabsf(cm) < 2.f * kSum;
}

// What the warps leave for the merge ([warp][head][m, l, acc]) of a split in which such a block was met: all of it again, a
// token at a time from global memory, channels over the lanes, one head after another.  (Where every split needs it: batch 1 at
// 32K 260 us, 64 ragged requests 37 ms.  Its test costs the other calls 1 %, up to 6 % at d = 64 with eight heads.)
template <int D, int FMT, bool QF32, typename Page>
__device__ void plain_split(const Kv8DecodeArgs& a, int b, int h, int e0, int e1, Page page_of, const uint16_t* tail, int rows, float* mg) {
  constexpr int C = D / 32;                             // channels of a lane
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int G = g.gq(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = lane * C;
  const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
  for (int hh = 0; hh < G; ++hh) {
    float q[C], o[C], big = 0.f, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      q[i] = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)(h * G + hh) * D + ch + i, QF32 ? kDtypeF32 : kDtypeBF16);
      o[i] = 0.f;
      big = fmaxf(big, fabsf(q[i]));
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) big = warp_max_xor(big, x);
    float up, down;
    power_of_two(big, &up, &down);
    // a token of score c f and values v
    auto token = [&](float c, float f, const float (&v)[C]) {
#pragma unroll
      for (int x = 16; x; x >>= 1) c += __shfl_xor_sync(0xffffffffu, c, x);
      const float s = c * f, m_new = fmaxf(m, s), alpha = ex2(m - m_new), p = ex2(s - m_new);
      l = fmaf(l, alpha, p);
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] = fmaf(o[i], alpha, p * v[i]);
      m = m_new;
    };
    for (int r = warp; r < rows; r += kConsumers) {
      const uint16_t* k = tail + (size_t)r * D + ch;
      float c = 0.f, v[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        c = fmaf(__uint_as_float((uint32_t)k[i] << 16), q[i], c);
        v[i] = __uint_as_float((uint32_t)k[(size_t)g.P * D + i] << 16);
      }
      token(c, Scale<D>::hi, v);
    }
    for (int e = e0 + warp; e < e1; e += kConsumers) {
      const int pid = page_of(e);
      if (pid < 0) continue;
      const uint8_t* block = layer + (size_t)pid * kg.page_bytes();
      const float2 scale = *reinterpret_cast<const float2*>(block + kg.scale_off());
      for (int t = 0; t < g.P; ++t) {
        const uint8_t *k = block + kv8_place<D, false>(t, ch), *w = block + kg.v_off() + kv8_place<D, true>(t, ch);
        float c = 0.f, v[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
          c = fmaf(kv8_value<FMT>(k[i]), q[i] * up, c);
          v[i] = kv8_value<FMT>(w[i]) * scale.y;
        }
        token(c, scale.x * (down * Scale<D>::hi), v);
      }
    }
    float* row = mg + (warp * 8 + hh) * (D + 2);
    if (lane == 0) row[0] = m, row[1] = l;
#pragma unroll
    for (int i = 0; i < C; ++i) row[2 + ch + i] = o[i];
  }
}

// ------------------------------------------------------------------ pages
// G8: eight query heads per kv head (an MMA column is a head, low halves go through a second MMA); otherwise
// up to four (columns 2 h and 2 h + 1 are the high and the low half of head h).
template <int D, int FMT, bool G8, bool QF32, int NB>
__global__ void __launch_bounds__(kThreads, (Layout<D, NB, G8>::kResident)) kv8_decode_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  using L = Layout<D, NB, G8>;
  constexpr int kStages = L::kStages;
  constexpr int KS = D / 16;               // k-steps of a score, and channel tiles of a sum
  constexpr int NH = G8 ? 2 : 1;           // heads whose weights a lane holds
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ uint32_t mapped[kStages];     // bit i: page i of the stage is there
  __shared__ int abort_flag, issued;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const Geom& g = a.g;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = g.gq(), P = g.P;
  const int per_stage = L::kTokens / P;
  int e0 = split * a.wl.stages_per_split * per_stage;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  // (The prefix kernel's CTAs, which take an SM each, start when these have ended: 8 requests behind 130,048 shared tokens 94 us a
  // call, 111 where they took the SMs one by one from the start on, 103 without a dependent launch.)
  if (a.groups.n == 0 || a.groups.max_shared == 0) pdl_launch_dependents();
  const int n = a.seq_lens[b];
  int first = 0;                                        // pages of the request that the prefix kernel reads
  if (a.groups.n) {
    first = kv8_shared_of(a, b);
    e0 += max(first, 0);
  }
  // the producer's first table entries travel with the length
  const int* bt = a.block_table + (size_t)b * a.bt_stride;
  const int* list = a.page_idx ? a.page_idx + ((size_t)b * g.Hkv + h) * a.n_select : nullptr;
  int early = -1, early_before = -1;
  if (warp == kConsumers) {
    const int e = e0 + lane;
    if (list) {
      early = e < a.n_select ? list[e] : -1;
      early_before = e > 0 && e <= a.n_select ? list[e - 1] : -1;
    } else {
      early = e < a.bt_stride ? bt[e] : -1;
    }
  }
  const bool sound = a.groups.n ? n == 0 || kv8_own_sound(a, n, first) : length_ok(a, n);
  if (!sound && tid == 0 && split == 0) flag_error(a.status, kDevBadLen);
  if (!sound || n == 0) {
    if (a.wl.max_splits == 1)  // (else the merge writes the zeros)
      for (int i = tid; i < G * D; i += kThreads) store_out(a, ((size_t)b * g.Hq + (size_t)h * G) * D + i, 0.f);
    return;
  }
  const int pages = n / P;
  const int have = a.page_idx ? a.n_select : pages;
  const int splits = split_count(a, have - first);
  if (split >= splits) return;
  const int e1 = min(e0 + a.wl.stages_per_split * per_stage, have);
  const int stages = (e1 - e0 + per_stage - 1) / per_stage;
  const int tail_rows = split == splits - 1 ? n % P : 0;
  const int page_stride = L::page_stride(P), stage_bytes = L::stage_bytes(P);
  __syncthreads();
  const int gid = lane >> 2, tig = lane & 3;
  float m_run[NH], l_run[NH], acc[KS][2 * NH];
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
  }
#pragma unroll
  for (int mt = 0; mt < KS; ++mt)
#pragma unroll
    for (int i = 0; i < 2 * NH; ++i) acc[mt][i] = 0.f;

  // page of entry e (value: the list's or the table's word for it, before: the list's word before it); -1: nothing to copy
  auto lookup = [&](int e, int value, int before) {
    if (e >= e1) return -1;
    int pid = value;
    if (list) {
      if (value < 0) return -1;
      if (value >= pages || before >= value || (e > 0 && before < 0)) {
        flag_error(a.status, kDevBadPage);
        return -1;
      }
      pid = value < a.bt_stride ? bt[value] : -1;
    }
    if (pid < 0 || pid >= g.num_pages) {
      flag_error(a.status, kDevBadPage);
      return -1;
    }
    return pid;
  };
  bool lost = false;                                    // a block's scores need more digits of the query
  if (warp == kConsumers) {
    // ---------------------------------------------------------------- producer
    const Kv8Geom kg{P, D, g.Hkv};
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t bytes = 2 * P * D + 16;
    const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
    auto later = [&](int e) {  // the same for entries after the first 32
      if (e >= e1) return -1;
      return list ? lookup(e, list[e], list[e - 1]) : lookup(e, e < a.bt_stride ? bt[e] : -1, -1);
    };
    int pid_now = lookup(e0 + lane, early, early_before), pid_next = later(e0 + 32 + lane);
    int it = 0;
    bool good = true;
    for (; it < stages; ++it) {
      const int s = it % kStages;
      if (it >= kStages) {
        good = mbar_wait_sleep_bounded(&empty[s], ((it / kStages) - 1) & 1, a.status);
        good = __all_sync(0xffffffffu, good && !*(volatile int*)&abort_flag);
        if (!good) break;
      }
      const int at = it * per_stage;                    // first entry of the stage, relative to e0
      if (at > 0 && at % 32 == 0) {
        pid_now = pid_next;
        pid_next = later(e0 + at + 32 + lane);
      }
      const int pid = __shfl_sync(0xffffffffu, pid_now, (at & 31) + (lane % per_stage));
      const unsigned there = __ballot_sync(0xffffffffu, lane < per_stage && pid >= 0);
      if (lane == 0) {
        mapped[s] = there;
        mbar_arrive_expect_tx(&full[s], __popc(there) * bytes);
      }
      __syncwarp();
      if (lane < per_stage && pid >= 0)
        bulk_g2s_hint(smem + s * stage_bytes + lane * page_stride, layer + (size_t)pid * kg.page_bytes(), bytes, &full[s], policy);
    }
    if (lane == 0) {
      issued = it;
      if (!good) *(volatile int*)&abort_flag = 1;
    }
  } else {
    // ---------------------------------------------------------------- consumers
    uint32_t qf[KS][2], ql[G8 && QF32 ? KS : 1][2];
    float qs[NH];                                       // per head of this lane's columns: 2^-e log2(e) / sqrt(d)
    {
      // lane (column gid, tig): the channels whose codes its 16-byte K loads hold
      const int head = G8 ? gid : gid >> 1;
      const bool low = !G8 && (gid & 1);
      const bool live = head < G;
      const size_t at = (size_t)b * a.q_stride + (size_t)(h * G + (live ? head : 0)) * D;
      float x[KS][4];
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < KS / 4; ++c)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const size_t i = at + (tig + 4 * c) * 16 + 4 * w;
          const float4 v = kv8_load4<QF32>(a.q, i);
          float* y = x[4 * c + w];
          y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
#pragma unroll
          for (int k = 0; k < 4; ++k) big = fmaxf(big, fabsf(y[k]));
        }
      big = warp_max_xor(big, 1);
      big = warp_max_xor(big, 2);
      float up, down;
      power_of_two(big, &up, &down);
      if (!live) down = 0.f;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float y0 = live ? x[kk][2 * p] * up : 0.f, y1 = live ? x[kk][2 * p + 1] * up : 0.f;
          const uint32_t hi = pack_half2(y0, y1);
          if constexpr (QF32) {
            const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
            const uint32_t lo = pack_half2(y0 - __low2float(hh), y1 - __high2float(hh));
            qf[kk][p] = low ? lo : hi;
            if constexpr (G8) ql[kk][p] = lo;
          } else {
            qf[kk][p] = low ? 0u : hi;
          }
        }
#pragma unroll
      for (int i = 0; i < NH; ++i)  // columns 2 tig (+ 1) of this lane: head 2 tig + i (G8) or head tig
        qs[i] = __shfl_sync(0xffffffffu, down, (G8 ? 2 * tig + i : 2 * tig) * 4) * Scale<D>::hi;
    }
    const int pi = warp * 16 * NB / P;                  // page of the stage, and the first block's first token in it
    const int t0 = warp * 16 * NB % P;
    // byte offsets inside a page: K row gid (+ 8), chunk tig (+ 4); V rows 2 tig (+ 1, + 8, + 9), chunk of channels gid D / 8
    const uint32_t k_off = D == 128 ? (t0 + gid) * 128 + ((tig ^ (4 * (gid & 1))) << 4) : (t0 + gid) * 64 + tig * 16;
    const uint32_t v_off = P * D + (D == 128 ? (t0 + 2 * tig) * 128 + ((gid ^ (2 * tig)) << 4)
                                             : (t0 / 2 + tig) * 128 + (((gid >> 1) ^ (2 * tig)) << 4) + (gid & 1) * 8);
    if (warp * 16 < tail_rows) {
      if (const uint16_t* rows = tail_of(a, b, h)) {
        rows += (size_t)warp * 16 * D;
        tail_block<D, G8, QF32>(a, b, h, rows, rows + (size_t)P * D, tail_rows - warp * 16, m_run, l_run, acc);
      } else if (lane == 0) {
        flag_error(a.status, kDevBadSlot);
      }
    }
    for (int it = 0; it < stages; ++it) {
      const int s = it % kStages;
      bool good = mbar_wait_sleep_bounded(&full[s], (it / kStages) & 1, a.status);
      good = __all_sync(0xffffffffu, good);
      if (!good) {
        *(volatile int*)&abort_flag = 1;
        break;
      }
      if ((mapped[s] >> pi) & 1) {
        const uint8_t* page = smem + s * stage_bytes + pi * page_stride;
        const float2 sc2 = *reinterpret_cast<const float2*>(page + 2 * P * D);
        // scores
        float sc[NB][4];
        float cm[NH];                                   // the blocks' largest raw sum
#pragma unroll
        for (int i = 0; i < NH; ++i) cm[i] = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t kw[2][KS];
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < KS / 4; ++c) {
              const uint32_t at = D == 128 ? (k_off ^ (64 * c)) + (2 * nb + r) * 8 * D : k_off + (2 * nb + r) * 8 * D;
              const uint4 v = *reinterpret_cast<const uint4*>(page + at);
              kw[r][4 * c] = v.x, kw[r][4 * c + 1] = v.y, kw[r][4 * c + 2] = v.z, kw[r][4 * c + 3] = v.w;
            }
          // (in two chains: the tensor cores' sums lose a last place or so a step, and the scores' errors count in full)
          float sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nb][i] = 0.f;
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) {
            const uint32_t a0 = kv8_pair<FMT, 0>(kw[0][kk]), a1 = kv8_pair<FMT, 0>(kw[1][kk]);
            const uint32_t a2 = kv8_pair<FMT, 1>(kw[0][kk]), a3 = kv8_pair<FMT, 1>(kw[1][kk]);
            mma_f16(kk & 1 ? sd : sc[nb], a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
            if constexpr (G8 && QF32) mma_f16(kk & 1 ? sd : sc[nb], a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[nb][i] += sd[i];
          if constexpr (!G8 && QF32) {                  // the low halves' columns
            sc[nb][0] += sc[nb][1];
            sc[nb][2] += sc[nb][3];
          }
#pragma unroll
          for (int i = 0; i < NH; ++i) cm[i] = fmaxf(cm[i], fmaxf(G8 ? sc[nb][i] : sc[nb][0], G8 ? sc[nb][2 + i] : sc[nb][2]));
        }
        // weights relative to the blocks' maximum
        float beta[NH], alpha[NH], fh[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          cm[i] = warp_max_xor(cm[i], 4);
          cm[i] = warp_max_xor(cm[i], 8);
          cm[i] = warp_max_xor(cm[i], 16);
          fh[i] = sc2.x * qs[i];
          const float fl = fmaf(fh[i], Scale<D>::lo / Scale<D>::hi, fmaf(sc2.x, qs[i], -fh[i]));
          lost |= digits_lost<D, FMT>(fh[i], cm[i]);
          const Top top(cm[i], fh[i], fl);
          const float m_new = fmaxf(m_run[i], top.m);
          alpha[i] = ex2(m_run[i] - m_new);
          beta[i] = ex2(top.over(m_new));
          m_run[i] = m_new;
          l_run[i] *= alpha[i];
        }
        uint32_t pb[NB][G8 ? 4 : 2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float pr[NH][2];
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const float da = (G8 ? sc[nb][i] : sc[nb][0]) - cm[i], db = (G8 ? sc[nb][2 + i] : sc[nb][2]) - cm[i];
            pr[i][0] = ex2(da * fh[i]);                 // (w log2 w is small: here f's rounding does not count)
            pr[i][1] = ex2(db * fh[i]);
            l_run[i] = fmaf(beta[i], pr[i][0] + pr[i][1], l_run[i]);
          }
          if constexpr (G8) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t hi = pack_half2(pr[0][r], pr[1][r]);
              const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
              pb[nb][r] = transpose_8x8(hi);
              pb[nb][2 + r] = transpose_8x8(pack_half2(pr[0][r] - __low2float(hh), pr[1][r] - __high2float(hh)));
            }
          } else {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float hi = __half2float(__float2half_rn(pr[0][r]));
              pb[nb][r] = transpose_8x8(pack_half2(hi, pr[0][r] - hi));
            }
          }
        }
        // sums: acc = acc alpha + o beta scale, o over the blocks
#pragma unroll
        for (int i = 0; i < NH; ++i) beta[i] *= sc2.y;
        float o[KS][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t vw[4][KS / 2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(page + v_off + (16 * nb + (j & 1) + 8 * (j >> 1)) * 128);
              vw[j][0] = v.x, vw[j][1] = v.y, vw[j][2] = v.z, vw[j][3] = v.w;
            } else {
              // row 2 tig + 1 is the other half of the 128-byte line: four chunks on
              const uint2 v = *reinterpret_cast<const uint2*>(page + ((v_off - P * D) ^ (64 * (j & 1))) + P * D + (2 * nb + (j >> 1)) * 512);
              vw[j][0] = v.x, vw[j][1] = v.y;
            }
          }
#pragma unroll
          for (int w = 0; w < KS / 2; ++w)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int mt = 2 * w + u;
              const uint32_t x01 = prmt(vw[0][w], vw[1][w], u ? 0x7362u : 0x5140u);
              const uint32_t x23 = prmt(vw[2][w], vw[3][w], u ? 0x7362u : 0x5140u);
              const uint32_t a0 = kv8_pair<FMT, 0>(x01), a1 = kv8_pair<FMT, 1>(x01);
              const uint32_t a2 = kv8_pair<FMT, 0>(x23), a3 = kv8_pair<FMT, 1>(x23);
              if (nb == 0) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
              mma_f16(o[mt], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
              if constexpr (G8) mma_f16(o[mt], a0, a1, a2, a3, pb[nb][2], pb[nb][3]);
              if (nb == NB - 1) {
                if constexpr (G8) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) acc[mt][i] = fmaf(acc[mt][i], alpha[i & 1], o[mt][i] * beta[i & 1]);
                } else {
                  acc[mt][0] = fmaf(acc[mt][0], alpha[0], (o[mt][0] + o[mt][1]) * beta[0]);
                  acc[mt][1] = fmaf(acc[mt][1], alpha[0], (o[mt][2] + o[mt][3]) * beta[0]);
                }
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[s])) : "memory");
      }
    }
  }
  const bool again = __syncthreads_or(lost);
  if (abort_flag) {  // a wait ran out: let the copies in flight land before the CTA ends
    if (tid == 0)
      for (int k = max(issued - kStages, 0); k < issued; ++k)
        (void)mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, nullptr);
    __syncthreads();
    return;
  }
  // merge the four warps' partials: [warp][head][D + 2] in the ring's memory
  float* mg = reinterpret_cast<float*>(smem);
  if (again) {
    if (warp < kConsumers) {
      const uint16_t* rows = tail_rows > 0 ? tail_of(a, b, h) : nullptr;
      auto page_of = [&](int e) {
        return list ? lookup(e, list[e], e > 0 ? list[e - 1] : -1) : lookup(e, e < a.bt_stride ? bt[e] : -1, -1);
      };
      plain_split<D, FMT, QF32>(a, b, h, e0, e1, page_of, rows, rows ? tail_rows : 0, mg);
    }
  } else if (warp < kConsumers) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 4);
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 8);
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 16);
      const int hh = G8 ? 2 * tig + i : tig;
      float* row = mg + (warp * 8 + hh) * (D + 2);
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {  // rows gid and gid + 8 of tile mt: channels gid D / 8 + 2 mt and the next
        row[2 + gid * (D / 8) + 2 * mt] = acc[mt][i];
        row[2 + gid * (D / 8) + 2 * mt + 1] = acc[mt][NH + i];
      }
      if (gid == 0) {
        row[0] = m_run[i];
        row[1] = l_run[i];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kThreads) {
    const int hh = i / D, ch = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, mg[(w * 8 + hh) * (D + 2)]);
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      const float* row = mg + (w * 8 + hh) * (D + 2);
      const float f = row[0] == -INFINITY ? 0.f : ex2(row[0] - M);
      l = fmaf(f, row[1], l);
      o = fmaf(f, row[2 + ch], o);
    }
    if (a.wl.max_splits == 1) {  // nothing to merge with
      store_out(a, ((size_t)b * g.Hq + h * G + hh) * D + ch, l == 0.f ? 0.f : o / l);
      continue;
    }
    float* pp = partial(a, b, h * G + hh, a.groups.slots + split, D);
    pp[4 + ch] = o;
    if (ch == 0) {
      pp[0] = l == l ? M : INFINITY;  // the merge takes no partial at -infinity: a NaN must not look like one
      pp[1] = l;
    }
  }
}

// ------------------------------------------------------------------ merge of the splits
// One CTA per (query head, request): warp w takes every W-th partial, N of them on their way at once and weighted relative
// to the warp's own maximum; a lane has D / 32 channels.  (With a first pass for the maximum of all, batch 1 at 32K took
// 18.4 us instead of 16.8.)  What the splits' count needs is read before the wait: no kernel since the decode kernel's own
// wait writes it.
template <int D, int W, int N>
__global__ void __launch_bounds__(32 * W) kv8_combine_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  constexpr int C = D / 32;
  __shared__ float s_o[W][D];
  __shared__ float2 s_ml[W];
  const Geom& g = a.g;
  const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = a.seq_lens[b];
  int count = 0, gap_at = 0x7fffffff, gap = 0;          // partials from gap_at on lie gap places further on
  if (a.groups.n) {
    const int first = kv8_shared_of(a, b);
    if (n > 0 && kv8_own_sound(a, n, first)) {
      gap_at = kv8_prefix_splits(a, first);
      gap = a.groups.slots - gap_at;
      count = gap_at + split_count(a, n / g.P - first);
    }
  } else if (length_ok(a, n) && n > 0) {
    count = split_count(a, a.page_idx ? a.n_select : n / g.P);
  }
  const float* base = partial(a, b, head, 0, D);
  pdl_wait();
  pdl_launch_dependents();
  float M = -INFINITY, l = 0.f, r[C];
#pragma unroll
  for (int c = 0; c < C; ++c) r[c] = 0.f;
  for (int i0 = warp; i0 < count; i0 += N * W) {
    float2 ml[N];
    float v[N][C];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int at = min(i0 + k * W, count - 1);
      const float* p = base + (size_t)(at >= gap_at ? at + gap : at) * (D + 4);
      ml[k] = *reinterpret_cast<const float2*>(p);
      if constexpr (C == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + 4 + lane * 4);
        v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p + 4 + lane * 2);
        v[k][0] = x.x, v[k][1] = x.y;
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (i0 + k * W >= count) ml[k].x = -INFINITY;
      m = fmaxf(m, ml[k].x);
    }
    if (m == -INFINITY) continue;
    const float f = ex2(M - m);
    l *= f;
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] *= f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float w = ex2(ml[k].x - m);
      l = fmaf(w, ml[k].y, l);
#pragma unroll
      for (int c = 0; c < C; ++c) r[c] = w == 0.f ? r[c] : fmaf(w, v[k][c], r[c]);
    }
    M = m;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_o[warp][lane * C + c] = r[c];
  if (lane == 0) s_ml[warp] = make_float2(M, l);
  __syncthreads();
  if (tid >= D) return;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w].x);
  float sum = 0.f, o = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const float f = s_ml[w].x == -INFINITY ? 0.f : ex2(s_ml[w].x - M);
    sum = fmaf(f, s_ml[w].y, sum);
    o = fmaf(f, s_o[w][tid], o);
  }
  store_out(a, ((size_t)b * g.Hq + head) * D + tid, sum == 0.f ? 0.f : o / sum);
}

template <int D, int FMT, int NB>
int launch_pages(const Kv8DecodeArgs& a, cudaStream_t s, bool pdl) {
  const dim3 grid(a.splits, a.g.Hkv, a.batch);
  const size_t smem = a.g.gq() == 8 ? Layout<D, NB, true>::smem(a.g.P) : Layout<D, NB, false>::smem(a.g.P);
  auto go = [&](auto kern) {
    const cudaError_t e = ensure_smem_limit(kern, smem, true);
    if (e != cudaSuccess) return (int)e;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, pdl, a);
  };
  const bool f32 = a.q_dtype == kDtypeF32;
  if (a.g.gq() == 8) return f32 ? go(kv8_decode_kernel<D, FMT, true, true, NB>) : go(kv8_decode_kernel<D, FMT, true, false, NB>);
  return f32 ? go(kv8_decode_kernel<D, FMT, false, true, NB>) : go(kv8_decode_kernel<D, FMT, false, false, NB>);
}

template <int D, int NB>
int launch_format(const Kv8DecodeArgs& a, cudaStream_t s, bool pdl) {
  return a.fmt == kKv8Int8 ? launch_pages<D, kKv8Int8, NB>(a, s, pdl) : launch_pages<D, kKv8E4m3, NB>(a, s, pdl);
}

}  // namespace

Kv8DecodeWs kv8_plan(const Geom& g, int batch, long long max_pages) {
  Kv8DecodeWs w{};
  const int per_stage = kv8_stage_tokens(g.D, g.P) / g.P;
  const long long stages = (max_pages + per_stage - 1) / per_stage;
  // Up to 8 stages one CTA takes them all and writes the output itself.  On the device the merge pays from 5 stages on
  // (batch 1, 8 stages: 6.4 us in one launch, 4.9 in two), but its launch costs the host 2 us, which is what a caller
  // without a graph waits for (8.9 us a call against 10.7).
  long long best = stages > 0 ? stages : 1;
  if (stages > 8) {
    const long long pairs = (long long)batch * g.Hkv > 0 ? (long long)batch * g.Hkv : 1;
    const long long wave = 152LL * resident(g.D, kv8_stage_tokens(g.D, g.P), g.gq() == 8);
    // The split that takes the fewest rounds of (its stages + 6, a CTA's start and end in stages): it fills one wave of CTAs
    // where it can (batch 1 at 32K: 9 stages 18.3 us, 8 23.1, 11 18.3) and keeps CTAs long in large batches (64 ragged
    // requests: 16 stages 472 us, 32 434, 64 423).
    long long cost = -1;
    for (long long per = 1; per <= 64 && per <= stages; ++per) {
      const long long ctas = pairs * ((stages + per - 1) / per);
      const long long c = ((ctas + wave - 1) / wave) * (per + 6);
      if (cost < 0 || c < cost) best = per, cost = c;
    }
  }
  w.stages_per_split = (int)best;
  w.max_splits = stages > 0 ? (int)((stages + best - 1) / best) : 1;
  w.total = (size_t)batch * g.Hq * w.max_splits * (g.D + 4) * sizeof(float);
  return w;
}

int launch_kv8_decode(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return launch_format<128, 1>(a, s, pdl);
  return kv8_stage_tokens(a.g.D, a.g.P) == 128 ? launch_format<64, 2>(a, s, pdl) : launch_format<64, 1>(a, s, pdl);
}

int launch_kv8_combine(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(a.g.Hq, a.batch);
  auto go = [&](auto kern, int warps) { return launch_pdl(kern, grid, dim3(32 * warps), 0, s, pdl, a); };
  // warps and loads enough for every partial to be on its way at once, and no more: a large batch has few partials a row
  const int n = a.wl.max_splits;
  if (a.g.D == 128) {
    if (n > 16) return go(kv8_combine_kernel<128, 8, 8>, 8);
    return n > 4 ? go(kv8_combine_kernel<128, 4, 4>, 4) : go(kv8_combine_kernel<128, 4, 1>, 4);
  }
  if (n > 16) return go(kv8_combine_kernel<64, 8, 8>, 8);
  return n > 4 ? go(kv8_combine_kernel<64, 4, 4>, 4) : go(kv8_combine_kernel<64, 4, 1>, 4);
}

}  // namespace oscar
