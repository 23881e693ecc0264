// Decode attention of requests that share a prefix: the shared pages of a group, read once for all of its requests.
//
// Row r of a group is a query head of one of its requests.  Over a split of the shared pages a CTA forms, for up to 128 rows
// of a kv head at once,
//     S = Q K^T,   p = 2^(s - m),   l = sum p,   O = P V,
// and leaves (m, l, O) for the merge with the partials of the requests' own pages and tail rows, which the decode kernel forms.
// The codes of a page are read once per 128 rows instead of once per 8, and 4 d flops a token and row are on the tensor cores
// (tcgen05): at d = 128 memory bounds up to 147 rows of a kv head, the tensor cores more of them.  Short of either, what
// counts is that a CTA's parts (codes to operands, S, weights, O) run at the same time:
//
// Roles in a CTA, around two buffers of a tile of 128 tokens (64 for float32 queries, whose three terms take the room):
//   2 x 4     warps, keys and values: codes from global memory through registers, two tiles ahead, to operands in shared memory,
//             exactly.  Rows are tokens: for S the channels of a row are the contracted dimension, for O the tokens are.
//   2 warps   issue S = Q K^T and O += P V.
//   1 warp    has the scales of a tile's groups of 16 tokens, a lane each, two tiles ahead (in the warp that issues S they held
//             its next product back: 47 us instead of 43 for 12 ragged groups of head dim 64).
//   2 x 4     warps, one half of a tile's tokens each, a thread per row: S from tensor memory, the running maximum and sum, P to
//             tensor memory in the place of S, which holds two or three tiles.
// Prefix of 130,048 tokens, 8 requests of 4 heads a kv head, INT8: 81 us (3.3 of 6.7 TB/s), of which some 7 are a CTA's start
// and end.  Prefix of 32,768 tokens, 64 requests of 8 heads, E4M3: 89 us, 770 TFLOP/s.  A tile of 128 tokens takes some 2600 clocks
// (1040 on the tensor cores fed without a pause, 1400 in issue slots, 1280 in shared memory's ports); without the softmax and the
// conversion it would take 1530: the handing over from role to role.  On the CUDA cores the same took 3.9 and 12.3 ms.
//
// BF16 queries, brought near 2^14 by a power of two, are f16 numbers but for components below 2^-31 of the largest: keys and
// queries are f16 operands, or BF16 ones where a query has such components; float32 queries are sums of three BF16 operands.
// A score is scaled in the exponent's multiplication by its page's scale.  Weights times their page's V scale are f16: one
// number (11 bits, the V scale in the exponent) for BF16 outputs, which are rounded to 8 bits at the end, and two (22 bits, the
// V scale a factor) for float32 ones: 138 us instead of 89 for the 64 requests, 134 instead of 81 for the 8.
#include <cuda.h>

#include "kv8.cuh"

namespace oscar {
namespace {

#include "tc_common.cuh"

constexpr int kSoft = 8, kConv = 8;                       // warps
constexpr int kThreads = 32 * (kSoft + kConv + 3);
constexpr int kRows = 128;
constexpr int kMostPages = 2048;                          // pages of a split
// Tensor memory, all of it (so that it begins at 0): scores, then weights, of NS tiles; sums.  The tensor cores' additions
// round towards zero: over thousands of tokens that would be 10^-6 of a sum and more, so for float32 outputs the sums are added up
// in float32 proper every kFlush tokens (0.9 10^-6 of bias at 2000 tokens a split without, 0.3 with).
constexpr uint32_t kColTotal = 256, kColO = 384, kCols = 512;
constexpr int kFlush = 512, kMostSlots = 3;
// A row has two reference exponents, whole numbers: m of its scores s, for l, and m + d of s + log2(V scale), for O, so that what
// counts is a page's part in the sum and a loud page that a row does not look at costs nothing.  They follow their maxima when
// these are kLag ahead; a weight at the second one is 2^kBase, none is above 2^(kLag + kBase) = 2^15.
constexpr float kLag = 12.f, kBase = 3.f;
constexpr float kFar = 4194304.f;                         // scores (log2) whose last place counts
constexpr float kLoud = 96.f;                             // log2 of a V scale by the second reference, beyond which float32 ends

template <int D, bool QF32, int TERMS>
struct Lay {
  static constexpr int QT = QF32 ? 3 : 1;                 // terms of a query
  static constexpr int NT = QF32 ? 64 : 128;              // tokens of a tile
  static constexpr int HC = NT / 2;                       // tokens of a half
  static constexpr int NS = TERMS == 2 && !QF32 ? 2 : 3;  // tiles of scores in tensor memory
  static constexpr int kQ = kRows * D * 2, kKV = NT * D * 2;
  static constexpr int oQ = 0, oK = oQ + QT * kQ, oV = oK + 2 * kKV, oPages = oV + 2 * kKV;
  static constexpr int kSmem = oPages + kMostPages * 4 + 1024;
  static constexpr int kTasks = NT * D / 16 / (16 * kConv);  // 16-byte chunks of keys (or of values) a thread takes of a tile
};

// Per group of 16 tokens (of one page): K scale, V scale and its logarithm.
struct Scales {
  float ks[8], vs[8], lg[8];
};

struct Shared {
  // K(i) written and S's place free; S(i) there and scales written; P(i) there and V(i) written; K read; V read and P V done
  uint64_t qk_ready[kMostSlots], s_full[kMostSlots], pv_ready[kMostSlots], k_empty[2], v_empty[2], end;
  Scales sc[kMostSlots];
  int mask[kMostSlots], plain[kMostSlots];  // groups that are there; all are, with V scales
  float2 top[2][2][kRows];       // a half's largest s and s + log2(V scale), of even and odd tiles
  float far[2][kRows];           // a half's largest s - m + log2(V scale), where scores are far from 0
  float l[2][kRows];             // a half's sum, at the end
  float down[kRows];             // what the power of two of a row's query leaves to multiply by
  int row_req[kRows];            // a row's request, -1 for none
  uint32_t there[kMostPages / 32];  // pages that are mapped
  uint32_t tmem;
  int lo, size, shared, tile, holder, holes;
};

// 2^e of a whole number e, within float32's normal numbers; 0 below them.
__device__ __forceinline__ float pow2(float e) { return e < -126.f ? 0.f : __uint_as_float((uint32_t)(127 + (int)fminf(e, 127.f)) << 23); }

// Two neighbouring code bytes of a word as a BF16 pair, both exact: bytes 0, 1 (HALF = 0) or 2, 3.  INT8: the low seven bits
// under the exponent of 128 are 128 + them; the top bit chooses what is taken off, 128 or 256.  E4M3: sign, exponent and mantissa
// in their places are the number times 2^-120.
template <int FMT, int HALF>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t w) {
  __nv_bfloat162 r;
  if constexpr (FMT == kKv8Int8) {
    const uint32_t x = prmt(w, 0, HALF ? 0x4342u : 0x4140u);
    const uint32_t low = (x & 0x007F007Fu) | 0x43004300u, off = (x & 0x00800080u) ^ 0x43804380u;
    r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&low), *reinterpret_cast<const __nv_bfloat162*>(&off));
  } else {
    const uint32_t x = prmt(w, 0, HALF ? 0x3424u : 0x1404u);
    const uint32_t y = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u), up = 0x7B807B80u;
    r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&up));
  }
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Descriptor of an operand whose contracted dimension runs along the rows: 8-row atoms of 128 swizzled bytes, 1024 bytes from
// atom to atom along the rows, `across` bytes from one 64-element block of the other dimension to the next.
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr, uint32_t across) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)(across >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}

// Weights of a row's scores in a half tile, 2^(s - m - d + kBase) by the page's V scale, as TERMS f16 numbers; sum 2^(s - m) is
// returned.  One number: the V scale is in the exponent, and out of the sum again.  Two numbers, of 22 bits: it is
// a factor, with what the rounding of a score's scale f = K scale x query scale leaves out at the group's largest score.
// ONE: all of the half tile's tokens are of one page.
template <int HC, int TERMS, bool ONE>
__device__ __forceinline__ float weigh(const uint32_t (&x)[HC], const float (&cm)[HC / 16], const float (&f)[HC / 16], uint32_t at,
                                       const float* ks, float qs, float qs_lo, float m, float d) {
  const float *vs = ks + 8, *lg = ks + 16;                // (of Scales)
  const float diff = d - kBase, to_o = pow2(-diff);
  float total = 0.f;
#pragma unroll
  for (int c = 0; c < HC / 32; ++c) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = 2 * c + u, s = ONE ? 0 : k;
      float g = 1.f, back, bias;
      if constexpr (TERMS == 2) {
        back = ex2(fminf(cm[k] * fmaf(ks[s], qs_lo, fmaf(ks[s], qs, -f[s])), 1.f));
        g = vs[s] * to_o * back;
        bias = -m;
      } else {
        bias = lg[s] - (m + diff);
        back = ex2(diff - lg[s]);
      }
      const uint64_t ff = pair(f[s], f[s]), bb = pair(bias, bias), gg = pair(g, g);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t e = fma2(pair(x[32 * c + 16 * u + 2 * j], x[32 * c + 16 * u + 2 * j + 1]), ff, bb);
        uint64_t w = pair(ex2(first(e)), ex2(second(e)));
        sum[j & 1] = add2(sum[j & 1], w);
        if constexpr (TERMS == 2) w = mul2(w, gg);
        hi[8 * u + j] = pack_half2(first(w), second(w));
        if constexpr (TERMS == 2) {
          const __half2 h = *reinterpret_cast<const __half2*>(&hi[8 * u + j]);
          lo[8 * u + j] = pack_half2(first(w) - __low2float(h), second(w) - __high2float(h));
        }
      }
      const uint64_t both = add2(sum[0], sum[1]);
      total = fmaf(first(both) + second(both), back, total);
    }
    tmem_st16(at + 16 * c, hi);
    if constexpr (TERMS == 2) tmem_st16(at + HC / 2 + 16 * c, lo);
  }
  return total;
}

// The same where some groups are not there or have no V scale (all of a page's values 0) or one too far from the others, or some
// row's scores are so large (kFar) that a last place of one counts: there distances are formed from the raw sums, 0 at a group's
// largest.  A V scale 2^kLoud above the second reference (on a page whose weights vanish next to it) is taken by 2^kLoud less, its
// weights by as much more.  Other rows come out as from weigh, bit for bit.  A group at a time: few registers, which the caller's
// scores need (all 64 scores at once cost 2 us of 94 at 64 samples of 32K).
template <int HC, int TERMS>
__device__ __noinline__ float weigh_with_care(uint32_t at, const float* ks, float qs, float qs_lo, float m, float d, int mask) {
  constexpr int NG = HC / 16;
  const float *vs = ks + 8, *lg = ks + 16;
  if (m == -INFINITY) m = 0.f;
  const bool far = fabsf(m) >= kFar;
  float v[16];
  auto load = [&](int k) {                                // returns the largest
    tmem_ld16(at + 16 * k, *reinterpret_cast<uint32_t(*)[16]>(&v));
    float cm = v[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) cm = fmaxf(cm, v[j]);
    return cm;
  };
  const bool any = d > -INFINITY;                         // (else no page so far has values)
  const float diff = any ? d - kBase : 0.f;
  float total = 0.f;
  uint32_t lo[TERMS == 2 ? NG : 1][8];
#pragma unroll
  for (int k = 0; k < NG; ++k) {                          // (a group's scores are read before its weights or others' take their place)
    const float f = ks[k] * qs, cm = load(k);
    const bool there = mask >> k & 1, some = there && any && vs[k] > 0.f;
    const bool apart = far && cm > -INFINITY;
    const float off = apart ? cm : 0.f;
    float bias = apart ? fminf(fmaf(cm, f, -m), kLag) : -m, back = 1.f, g = some ? 1.f : 0.f;
    if (TERMS == 1 && some && diff - lg[k] <= 60.f) {
      bias = apart ? bias + (lg[k] - diff) : lg[k] - (m + diff);
      back = ex2(diff - lg[k]);
    } else if (TERMS == 1) {                              // (2^(s + log2(V scale) - m - d) vanishes)
      if (some) g = vs[k] * pow2(-diff);
    } else {
      if (!apart && there) back = ex2(fminf(cm * fmaf(ks[k], qs_lo, fmaf(ks[k], qs, -f)), 1.f));
      const bool loud = some && lg[k] - diff > kLoud;
      const float e = -diff - (loud ? kLoud : 0.f);
      if (some) g = fminf(vs[k] * pow2(fminf(e, 126.f)) * pow2(fmaxf(e - 126.f, 0.f)), 1e36f) * back;
      if (loud) bias += kLoud, back = 0.f;                // (such a weight is below 2^-80 of the row's largest)
    }
    uint32_t hi[8];
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[e] = there ? ex2(fmaf(v[2 * j + e] - off, f, bias)) : 0.f;
        sum[2 * (j & 1) + e] += w[e];
        w[e] = some ? w[e] * g : 0.f;
      }
      hi[j] = pack_half2(w[0], w[1]);
      if constexpr (TERMS == 2) {
        const __half2 h = *reinterpret_cast<const __half2*>(&hi[j]);
        lo[k][j] = pack_half2(w[0] - __low2float(h), w[1] - __high2float(h));
      }
    }
    total = fmaf((sum[0] + sum[2]) + (sum[1] + sum[3]), back, total);
    tmem_st8(at + 8 * k, hi);
  }
  if constexpr (TERMS == 2)
#pragma unroll
    for (int k = 0; k < NG; ++k) tmem_st8(at + HC / 2 + 8 * k, lo[k]);
  return total;
}

// A row's sums times scale.
template <int D>
__device__ __forceinline__ void scale_sums(uint32_t at, float scale) {
  uint32_t w[2][32];
  tmem_ld32_nowait(at, w[0]);
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    tmem_wait_ld();
    if (c + 1 < D / 32) tmem_ld32_nowait(at + 32 * (c + 1), w[(c + 1) & 1]);
#pragma unroll
    for (int j = 0; j < 32; ++j) w[c & 1][j] = __float_as_uint(__uint_as_float(w[c & 1][j]) * scale);
    tmem_st32(at + 32 * c, w[c & 1]);
  }
}

// total = (total + sums) scale, without a total yet sums scale.
template <int D>
__device__ __forceinline__ void add_sums(uint32_t total, uint32_t at, float scale, bool some) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t x[32], y[32];
    tmem_ld32_nowait(at + c, x);
    tmem_ld32_nowait(total + c, y);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __float_as_uint((__uint_as_float(x[j]) + (some ? __uint_as_float(y[j]) : 0.f)) * scale);
    tmem_st32(total + c, x);
  }
}

// 16 bytes that no one writes while the kernel runs, read once by each SM; in the order of the code (the compiler would move a
// plain load down to its use).
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

template <int D, int FMT, bool QF32, int TERMS>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefix_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  using L = Lay<D, QF32, TERMS>;
  constexpr int QT = L::QT, NT = L::NT, HC = L::HC, NG = HC / 16, NS = L::NS, kPeriod = kFlush / NT;
  constexpr bool kTwo = TERMS == 2;                       // sums in two parts
  auto col_s = [](int s) -> uint32_t { return NT * s; };
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t* page_at = reinterpret_cast<uint32_t*>(smem + L::oPages);  // of the split's pages, in units of 128 bytes
  const Geom& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // A page's heads lie together, so CTAs of the same pages follow one another, kv heads first (64 samples of 32K 134 us a call with
  // a head's splits one after another, 131 so; 4 prompts of 8K 41.2, 39.4).
  const int h = blockIdx.x % a.g.Hkv, at_x = blockIdx.x / a.g.Hkv, tile = at_x % a.groups.max_tiles, split = at_x / a.groups.max_tiles;
  const int G = g.gq(), P = g.P;
  // The grid before this one is the decode kernel of the same call: all that this one reads was there before it.  What it leaves
  // (for the merge, which follows this grid) is waited for at the end.
  pdl_launch_dependents();
  if (tid == 0) {
    for (int b = 0; b < NS; ++b) {
      mbar_init(&sh.qk_ready[b], kConv / 2 + 1);
      mbar_init(&sh.s_full[b], 2);
      mbar_init(&sh.pv_ready[b], kSoft + kConv / 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.k_empty[b], 1);
      mbar_init(&sh.v_empty[b], 1);
    }
    mbar_init(&sh.end, 2);
    sh.holes = 0;
    fence_barrier_init();
    for (int b = 0; b < NS; ++b) mbar_arrive(&sh.qk_ready[b]);  // the first S of a place waits for no product
  }
  if (warp == 0) {
    // the group of this row tile, and its first request that is not empty
    int at = -1, before = 0, lo = 0, size = 0, shared = 0;
    for (int i0 = 0; i0 < a.groups.n && at < 0; i0 += 32) {
      const int i = i0 + lane;
      int t = 0, b0 = 0, b1 = 0, s = 0;
      if (i < a.groups.n) {
        b0 = a.groups.starts[i], b1 = a.groups.starts[i + 1], s = a.groups.shared[i];
        if (b0 >= 0 && b0 <= b1 && b1 <= a.batch && s > 0 && s <= a.groups.max_shared) t = ((b1 - b0) * G + kRows - 1) / kRows;
      }
      int sum = t;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + sum > tile);
      if (hit) {
        const int src = __ffs(hit) - 1;
        at = i0 + src;
        lo = __shfl_sync(0xffffffffu, b0, src);
        size = __shfl_sync(0xffffffffu, b1, src) - lo;
        shared = __shfl_sync(0xffffffffu, s, src);
        before += __shfl_sync(0xffffffffu, sum - t, src);
      } else {
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    int holder = -1;
    if (at >= 0)
      for (int r0 = 0; r0 < size && holder < 0; r0 += 32) {
        const int n = r0 + lane < size ? a.seq_lens[lo + r0 + lane] : 0;
        const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && kv8_own_sound(a, n, shared));
        if (hit) holder = lo + r0 + __ffs(hit) - 1;
      }
    if (lane == 0) {
      sh.lo = lo;
      sh.size = size;
      sh.shared = shared;
      sh.tile = tile - before;
      sh.holder = holder;
    }
  }
  __syncthreads();
  const int per = a.groups.units_per_split * (kPrefixUnit / P), e0 = split * per;
  const int pages = sh.holder < 0 ? 0 : min(per, sh.shared - e0);
  // the row of a softmax thread
  bool valid = false;
  int req = 0;
  const int row = tid & (kRows - 1), half = warp >> 2;     // two softmax threads a row
  if (pages > 0 && warp < kSoft) {
    const int r = sh.tile * kRows + row;
    req = sh.lo + r / G;
    if (r < sh.size * G) {
      const int n = a.seq_lens[req];
      valid = n > 0 && kv8_own_sound(a, n, sh.shared);
    }
  }
  if (warp < kSoft / 2) sh.row_req[row] = valid ? req : -1;
  if (!__syncthreads_or(valid)) {                         // no rows, or no pages for them
    pdl_wait();
    return;
  }
  if (warp == 0) tmem_alloc(&sh.tmem, kCols);
  {
    const int* bt = a.block_table + (size_t)sh.holder * a.bt_stride;
    const uint32_t unit = (uint32_t)(Kv8Geom{P, D, g.Hkv}.page_bytes() / 128);
    for (int i0 = 32 * warp; i0 < pages; i0 += kThreads) {
      const int i = i0 + lane, e = e0 + i, pid = i < pages && e < a.bt_stride ? bt[e] : -1;
      const bool some = pid >= 0 && pid < g.num_pages;
      if (i < pages) {
        if (!some) {
          flag_error(a.status, kDevBadPage);
          sh.holes = 1;
        }
        page_at[i] = some ? pid * unit : 0;
      }
      const unsigned all = __ballot_sync(0xffffffffu, some);
      if (lane == 0) sh.there[i0 >> 5] = all;
    }
  }
  const bool live = __any_sync(0xffffffffu, valid);
  // The queries as operands, eight channels a thread and D / 8 threads a row, brought near 2^14 by a power of two
  bool exact = !QF32;                                     // keys and queries are f16 operands
  {
    constexpr int kLanes = D / 8, kStep = 32 * (kSoft + kConv) / kLanes, kPasses = kRows / kStep;
    const int r0 = tid / kLanes, c = tid % kLanes * 8;
    float4 x[kPasses][2];
    if (warp < kSoft + kConv) {
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        const int r = r0 + k * kStep, its = sh.row_req[r];
        x[k][0] = x[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (its >= 0) {
          const size_t at = (size_t)its * a.q_stride + (size_t)(h * G + (sh.tile * kRows + r) % G) * D + c;
          x[k][0] = kv8_load4<QF32>(a.q, at);
          x[k][1] = kv8_load4<QF32>(a.q, at + 4);
        }
      }
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        float4 &u = x[k][0], &w = x[k][1];
        float big = fmaxf(fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))),
                          fmaxf(fmaxf(fabsf(w.x), fabsf(w.y)), fmaxf(fabsf(w.z), fabsf(w.w))));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) big = warp_max_xor(big, d);
        float up, down;
        power_of_two(big, &up, &down);
        if (c == 0) sh.down[r0 + k * kStep] = down;
        u = make_float4(u.x * up, u.y * up, u.z * up, u.w * up);
        w = make_float4(w.x * up, w.y * up, w.z * up, w.w * up);
      }
    }
    auto put = [&](bool f16) {
      bool all = true;
#pragma unroll
      for (int k = 0; k < kPasses; ++k) {
        float y[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (f16) {
              w[j] = pack_half2(y[2 * j], y[2 * j + 1]);
              const __half2 v = *reinterpret_cast<const __half2*>(&w[j]);
              all &= __low2float(v) == y[2 * j] && __high2float(v) == y[2 * j + 1];
            } else {
              w[j] = pack_bf162(y[2 * j], y[2 * j + 1]);
              y[2 * j] -= bf16_lo(w[j]);
              y[2 * j + 1] -= bf16_hi(w[j]);
            }
          }
          *reinterpret_cast<uint4*>(smem + L::oQ + t * L::kQ + sw128_offset(r0 + k * kStep, c, kRows)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      return all;
    };
    if constexpr (!QF32) exact = !__syncthreads_or(warp < kSoft + kConv && !put(true));
    if (!exact && warp < kSoft + kConv) put(false);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr double kScale = 1.4426950408889634 / (D == 128 ? 11.313708498984761 : 8.0);
  const float down = sh.down[row], qs = down * (float)kScale;  // what a score's raw sum is multiplied by, but for the page's scale
  const float qs_lo = down * (float)(kScale - (double)(float)kScale);
  const int tiles = (pages * P + NT - 1) / NT;
  bool good = true;
  float m = -INFINITY, d = -INFINITY, l = 0.f;            // l in units of 2^m, the sums of 2^(m + d - kBase)
  const uint32_t base = (uint32_t)(warp & 3) << 21;  // a softmax warp's 32 lanes

  if (warp < kSoft) {
    // ---------------------------------------------------------------- softmax
    for (int i = 0, b = 0, ph = 0; i < tiles; ++i) {
      if (good) {
        good = mbar_wait_sleep_bounded(&sh.s_full[b], ph, a.status);
        good = __all_sync(0xffffffffu, good);
        tc_fence_after();
      }
      if (live) {
        const uint32_t at = base + col_s(b) + HC * half;
        uint32_t x[HC];
#pragma unroll
        for (int c = 0; c < HC; c += 32) tmem_ld32_nowait(at + c, *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
        const float* ks = sh.sc[b].ks + NG * half;
        const int mask = sh.mask[b] >> (NG * half) & ((1 << NG) - 1), plain = sh.plain[b];
        float f[NG], cm[NG], top = -INFINITY, top_o = -INFINITY;
#pragma unroll
        for (int k = 0; k < NG; ++k) f[k] = ks[k] * qs;
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < NG; ++k) {
          auto v = [&](int j) { return __uint_as_float(x[16 * k + j]); };
          cm[k] = max3(max3(max3(v(0), v(1), v(2)), v(3), v(4)), max3(max3(v(5), v(6), v(7)), v(8), v(9)),
                       max3(max3(v(10), v(11), v(12)), max3(v(13), v(14), v(15)), v(0)));
          const float y = mask >> k & 1 ? __fmul_rd(cm[k], f[k]) : -INFINITY;
          top = fmaxf(top, y);
          top_o = fmaxf(top_o, y + ks[16 + k]);           // (+ the logarithm of the V scale)
        }
        // the largest of both halves: a pair of warps meets once a tile, after a wait that ran out too (a NaN: both go on without)
        sh.top[i & 1][half][row] = make_float2(good ? top : NAN, top_o);
        asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
        const float2 other = sh.top[i & 1][half ^ 1][row];
        good &= other.x == other.x;
        top = fmaxf(top, other.x);
        top_o = fmaxf(top_o, other.y);
        if (good) {
          // as a rule the references stay, and no score is so large that a last place of it counts
          float scale = 1.f;
          bool care = !plain, rescale = false, flush = false;
          if (__any_sync(0xffffffffu, top > m + kLag || top_o > m + d + kLag || !(fabsf(m) < kFar)) || (kTwo && i % kPeriod == 0)) {
            if (top > m + kLag || (m == -INFINITY && top > m)) {
              const float to = ceilf(top);
              l = m == -INFINITY ? l : l * pow2(m - to);
              d += m - to;                                // (m + d stays)
              m = to;
            }
            float d_new = ceilf(top_o - m);
            const bool far = !(fabsf(m) < kFar);
            if (__any_sync(0xffffffffu, far)) {
              // Such a score plus log2(V scale) has lost the V scale: the distances by which the weights go, of both halves (the same
              // rows, so both are here)
              care = true;
              float its = -INFINITY;
#pragma unroll
              for (int k = 0; k < NG; ++k) {
                float most = kTwo && QF32 ? cm[k] : -INFINITY;
                if constexpr (!kTwo || !QF32)             // (again: cm would take registers that the other forms lack)
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    float y = __uint_as_float(x[16 * k + j]);
                    asm volatile("" : "+f"(y));
                    most = fmaxf(most, y);
                  }
                const float t = m == -INFINITY ? 0.f : fminf(fmaf(most, ks[k] * qs, -m), kLag);
                if (mask >> k & 1) its = fmaxf(its, t + ks[16 + k]);
              }
              sh.far[half][row] = its;
              asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
              its = fmaxf(its, sh.far[half ^ 1][row]);
              if (far) d_new = ceilf(its);
            }
            if (d == -INFINITY ? d_new > d : d_new > d + (far ? 0.f : kLag)) {
              scale = d == -INFINITY ? 1.f : pow2(d - d_new);  // (1: there is nothing in the sums)
              d = d_new;
            }
            flush = kTwo && i > 0 && i % kPeriod == 0;
            rescale = __any_sync(0xffffffffu, scale != 1.f) || flush;
          }
          if (care)
            l += weigh_with_care<HC, TERMS>(at, ks, qs, qs_lo, m, d, mask);
          else if (P >= HC)
            l += weigh<HC, TERMS, true>(x, cm, f, at, ks, qs, qs_lo, m, d);
          else
            l += weigh<HC, TERMS, false>(x, cm, f, at, ks, qs, qs_lo, m, d);
          if (rescale) {                                  // (the weights first: by now the sums so far are done)
            good = mbar_wait_sleep_bounded(&sh.v_empty[(i - 1) & 1], ((i - 1) >> 1) & 1, a.status);
            good = __all_sync(0xffffffffu, good);
            tc_fence_after();
            const uint32_t o_at = base + kColO + half * (D / 2), total_at = base + kColTotal + half * (D / 2);
            if (good) {
              if (flush) {
                add_sums<D / 2>(total_at, o_at, scale, i > kPeriod);
              } else {
                scale_sums<D / 2>(o_at, scale);
                if (kTwo && i > kPeriod) scale_sums<D / 2>(total_at, scale);
              }
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0 && good) mbar_arrive(&sh.pv_ready[b]);
      if (++b == NS) b = 0, ph ^= 1;
    }
    sh.l[half][row] = l;
  } else if (warp < kSoft + kConv) {
    // ---------------------------------------------------------------- codes to operands
    constexpr int T = L::kTasks, kStep = D == 128 ? 16 : 32;
    const bool is_v = warp >= kSoft + kConv / 2;
    const int ct = (tid - 32 * kSoft) & (16 * kConv - 1), log_p = 31 - __clz(P);
    const Kv8Geom kg{P, D, g.Hkv};
    // Chunk j of token t0 (+ kStep a task: the turns stay).  Eight neighbouring lanes take the four chunks of 64 channels of two
    // neighbouring tokens: their halves' first (or second) 16 bytes lie in different banks.
    const int t0 = D == 128 ? 4 * (ct >> 5) + 2 * (lane >> 4) + ((lane >> 2) & 1) : ct >> 2;
    const int j = D == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : ct & 3;
    const int turn = is_v ? 2 * ((t0 >> 1) & 3) : D == 128 ? 4 * (t0 & 1) : 0;
    const int place = D == 128 ? j ^ turn : (4 * (t0 & 1) + j) ^ turn;  // of the chunk in its tokens' 128-byte line
    const uint8_t* src = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes() +
                         (is_v ? kg.v_off() : 0) + place * 16;
    uint8_t* dst = smem + (is_v ? L::oV : L::oK) + (j >> 2) * NT * 128 + t0 * 128 + (((2 * (j & 3)) ^ (t0 & 7)) << 4);
    const ptrdiff_t next = (t0 & 1) ? -16 : 16;           // to the chunk's other 16 bytes
    const uint32_t nothing = FMT == kKv8Int8 ? 0x80808080u : 0u;
    const bool holes = sh.holes, f16 = is_v || exact;
    uint64_t *empty = is_v ? sh.v_empty : sh.k_empty, *ready = is_v ? sh.pv_ready : sh.qk_ready;
    uint4 x[2][T];
    auto load = [&](int i, uint4 (&x)[T]) {
#pragma unroll
      for (int k = 0; k < T; ++k) {
        const int t = i * NT + t0 + kStep * k, e = min(t >> log_p, pages - 1);
        x[k] = load_codes(src + (size_t)page_at[e] * 128 + (t & (P - 1) & (D == 64 ? ~1 : ~0)) * D);
      }
    };
    auto store = [&](int i, uint8_t* to, const uint4 (&x)[T], bool f16) {
#pragma unroll
      for (int k = 0; k < T; ++k) {
        uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        if (holes) {  // what was read for a page that is not there may be any bytes: it has no weight, but a NaN times 0 is one
          const int e = min((i * NT + t0 + kStep * k) >> log_p, pages - 1);
          if (!(sh.there[e >> 5] >> (e & 31) & 1)) w[0] = w[1] = w[2] = w[3] = nothing;
        }
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = f16 ? kv8_pair<FMT, 0>(w[i]) : bf16_pair<FMT, 0>(w[i]);
          y[2 * i + 1] = f16 ? kv8_pair<FMT, 1>(w[i]) : bf16_pair<FMT, 1>(w[i]);
        }
        *reinterpret_cast<uint4*>(to + k * kStep * 128) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(to + k * kStep * 128 + next) = make_uint4(y[4], y[5], y[6], y[7]);
      }
    };
    load(0, x[0]);
    load(1, x[1]);
    for (int i0 = 0, s = 0; i0 < tiles && good; i0 += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b, s = s == NS - 1 ? 0 : s + 1) {
        const int i = i0 + b;
        if (i >= tiles) break;
        if (i >= 2) good = mbar_wait_sleep_bounded(&empty[b], ((i >> 1) & 1) ^ 1, a.status);
        good = __all_sync(0xffffffffu, good);
        if (!good) break;
        if (f16) store(i, dst + b * L::kKV, x[b], true);
        else store(i, dst + b * L::kKV, x[b], false);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[s]);
        load(i + 2, x[b]);
      }
    }
  } else if (warp == kSoft + kConv) {
    // ---------------------------------------------------------------- S = Q K^T
    const uint32_t idesc = exact ? idesc_f16_f32(kRows, NT) : idesc_bf16_f32(kRows, NT);
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::oQ)), k_desc = smem_desc_sw128(smem_u32(smem + L::oK));
    for (int i = 0, s = 0, ph = 0; i < tiles; ++i) {
      const int b = i & 1;
      good = mbar_wait_sleep_bounded(&sh.qk_ready[s], ph, a.status);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      fence_proxy_async_smem();                           // (what the other warps wrote, for the tensor cores)
      tc_fence_after();
      if (lane == 0) {
        const uint64_t kd = k_desc + b * (L::kKV >> 4);
#pragma unroll
        for (int t = QT - 1; t >= 0; --t)                 // (the small terms first: a sum loses less of them)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma(col_s(s), q_desc + ((t * L::kQ + (kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4),
                   kd + (((kk >> 2) * (NT * 128) + (kk & 3) * 32) >> 4), idesc, t < QT - 1 || kk);
        tc_commit(&sh.s_full[s]);
        tc_commit(&sh.k_empty[b]);
      }
      __syncwarp();
      if (++s == NS) s = 0, ph ^= 1;
    }
    if (lane == 0) tc_commit(&sh.end);
  } else if (warp == kSoft + kConv + 1) {
    // ---------------------------------------------------------------- scales
    const Kv8Geom kg{P, D, g.Hkv};
    const uint8_t* scales = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes() + kg.scale_off();
    float most = 0.f, least = INFINITY;                   // V scales so far, but for those of pages of zeros
    bool zeros = false;                                   // there were such
    uint2 sc[2];
    auto page_of = [&](int i) { return (i * NT + (lane & (2 * NG - 1)) * 16) >> (31 - __clz(P)); };
    auto load_scales = [&](int i, uint2& s) {
      asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(s.x), "=r"(s.y) : "l"(scales + (size_t)page_at[min(page_of(i), pages - 1)] * 128));
    };
    load_scales(0, sc[0]);
    load_scales(1, sc[1]);
    for (int i = 0, s = 0, ph = 0; i < tiles; ++i) {
      const int b = i & 1;
      const uint2 now = b ? sc[1] : sc[0];
      const int e_page = page_of(i);
      const bool some = e_page < pages && (sh.there[e_page >> 5] >> (e_page & 31) & 1);
      const unsigned mask = __ballot_sync(0xffffffffu, some && lane < 2 * NG);
      const float v_scale = some ? __uint_as_float(now.y) : 0.f, log_v = log2f(v_scale);
      // The careful way is for V scales 2^60 from others so far or so small that 2^-d is beyond float32; and, with two numbers a
      // weight, for whatever comes after a page of zeros: where that one leads, d is as far below as the other scores are.  (Else
      // a row's d is at least the smallest V scale so far, but for kLag.)
      const uint32_t bits = __float_as_uint(v_scale);
      const float high = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < 2 * NG ? bits : 0u));
      const float low = __uint_as_float(__reduce_min_sync(0xffffffffu, lane < 2 * NG && bits ? bits : 0x7F800000u));
      most = fmaxf(most, high);
      least = fminf(least, low);
      const bool all = __all_sync(0xffffffffu, lane >= 2 * NG || bits);
      zeros |= __any_sync(0xffffffffu, lane < 2 * NG && some && !bits);
      const bool plain = all && !(kTwo && zeros) && low > most * 8.673617379884035e-19f && high * 8.673617379884035e-19f < least && least > 7.888609052210118e-31f;
      good = mbar_wait_sleep_bounded(&sh.qk_ready[s], ph, a.status);  // (the place of S and of these is free)
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      if (lane < 2 * NG) {
        sh.sc[s].ks[lane] = some ? __uint_as_float(now.x) : 1.f;
        sh.sc[s].vs[lane] = v_scale;
        sh.sc[s].lg[lane] = log_v;
      }
      if (lane == 0) {
        sh.mask[s] = (int)mask;
        sh.plain[s] = plain;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.s_full[s]);
      if (b) load_scales(i + 2, sc[1]);
      else load_scales(i + 2, sc[0]);
      if (++s == NS) s = 0, ph ^= 1;
    }
  } else {
    // ---------------------------------------------------------------- O += P V
    constexpr uint32_t kIdesc = idesc_f16_f32(kRows, D) | (1u << 16);  // the second operand's contracted dimension along its rows
    const uint64_t v_desc = desc_rows(smem_u32(smem + L::oV), NT * 128);
    for (int i = 0, s = 0, ph = 0; i < tiles; ++i) {
      const int b = i & 1;
      good = mbar_wait_sleep_bounded(&sh.pv_ready[s], ph, a.status);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      fence_proxy_async_smem();
      tc_fence_after();
      if (lane == 0) {
        const uint64_t vd = v_desc + b * (L::kKV >> 4);
#pragma unroll
        for (int u = TERMS - 1; u >= 0; --u)
#pragma unroll
          for (int kk = 0; kk < NT / 16; ++kk)            // (a half's weights: its first terms, then its second ones)
            tc_mma_ts(kColO, col_s(s) + HC * (kk / NG) + u * (HC / 2) + 8 * (kk % NG), vd + ((kk * 2048) >> 4), kIdesc,
                      (kTwo ? i % kPeriod : i) > 0 || u < TERMS - 1 || kk);
        tc_commit(&sh.qk_ready[s]);
        tc_commit(&sh.v_empty[b]);
      }
      __syncwarp();
      if (++s == NS) s = 0, ph ^= 1;
    }
    if (lane == 0) tc_commit(&sh.end);
  }
  // Nothing is under way when the tensor memory is freed, a wait that ran out or not.
  good = mbar_wait_sleep_bounded(&sh.end, 0, a.status) && good;
  tc_fence_before();
  good = !__syncthreads_or(!good);
  tc_fence_after();
  // ------------------------------------------------------------------ the split's partial
  float* o_rows = reinterpret_cast<float*>(smem);         // [row][m, l, -, -, O]; the operands are done with
  if (good && warp < kSoft && live) {
    // m may lag by 2^kLag, and a sum so much larger end float32: the sum of weights is brought to [1, 2) (not where m has no place
    // for it), O with it, by two powers of two
    const float sum = sh.l[0][row] + sh.l[1][row];
    const float up = fabsf(m) < kFar && sum > 0.f && sum < INFINITY ? (float)((int)(__float_as_uint(sum) >> 23) - 127) : 0.f;
    const float to = d - kBase - up, scale = d == -INFINITY ? 0.f : pow2(fmaxf(to, -120.f)), less = pow2(fminf(to + 120.f, 0.f));
#pragma unroll 1
    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {  // (each half of the threads has half of the channels)
      float v[32];
      tmem_ld32(base + kColO + c, v);
      if (kTwo && tiles > kPeriod) {
        float more[32];
        tmem_ld32(base + kColTotal + c, more);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += more[j];
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<float4*>(o_rows + row * (D + 4) + 4 + c + j) =
            make_float4(v[j] * scale * less, v[j + 1] * scale * less, v[j + 2] * scale * less, v[j + 3] * scale * less);
    }
    if (half == 0)                                        // (a NaN must not look like no partial)
      *reinterpret_cast<float2*>(o_rows + row * (D + 4)) = make_float2(sum == sum ? m + up : INFINITY, sum * pow2(-up));
  }
  good = !__syncthreads_or(!good);
  if (good)
    for (int i = tid; i < kRows * (D / 4 + 1); i += kThreads) {  // 16 bytes a thread, a row's next to one another
      const int r = i / (D / 4 + 1), c = i % (D / 4 + 1) * 4, its = sh.row_req[r];
      if (its < 0) continue;
      const size_t to = ((size_t)its * g.Hq + h * G + ((sh.tile * kRows + r) & (G - 1))) * a.wl.max_splits + split;
      *reinterpret_cast<float4*>(a.part + to * (D + 4) + c) = *reinterpret_cast<const float4*>(o_rows + r * (D + 4) + c);
    }
  __syncthreads();
  if (warp == 0) tmem_dealloc(sh.tmem, kCols);
  pdl_wait();
}

}  // namespace

// Units of a split of prefixes of `all` units behind so many row tiles: the split that takes the fewest rounds of (its units + 8, a
// CTA's start and end: 64 samples of 32K 128 us a call in one round of 128 CTAs, 132 in two of 288, which 5 would choose).
static long long prefix_units(const Geom& g, long long row_tiles, long long all) {
  const long long pairs = row_tiles * g.Hkv > 0 ? row_tiles * g.Hkv : 1;
  const long long most = (long long)kMostPages * g.P / kPrefixUnit;
  long long best = most < all ? most : all, cost = -1;
  for (long long rounds = 1; rounds <= 16; ++rounds) {    // as many splits as fill that many rounds
    const long long fit = 152 * rounds / pairs, splits = fit < all ? fit : all;
    if (splits == 0) continue;
    const long long per = (all + splits - 1) / splits;
    const long long c = ((pairs * ((all + per - 1) / per) + 151) / 152) * (per + 8);
    if (per <= most && (cost < 0 || c < cost)) best = per, cost = c;
  }
  return best;
}

static long long prefix_all(const Geom& g, int max_shared) {
  const long long units = ((long long)max_shared * g.P + kPrefixUnit - 1) / kPrefixUnit;
  return units > 0 ? units : 1;
}

Kv8DecodeWs kv8_shared_plan(const Geom& g, int batch, int n_groups, int max_shared, int max_own, Kv8Groups* groups, int* own_splits) {
  Kv8DecodeWs w = kv8_plan(g, batch, max_own / g.P);
  *own_splits = w.max_splits;
  const long long rows = (long long)batch * g.gq(), all = prefix_all(g, max_shared);
  const long long best = prefix_units(g, rows / kRows > n_groups ? rows / kRows : n_groups, all);
  groups->n = n_groups;
  groups->max_shared = max_shared;
  groups->max_own = max_own;
  groups->units_per_split = (int)best;
  // (a group's last tile has a request's rows or more; no more tiles than requests, so a grid of 2^31 would have partials of a TB)
  groups->max_tiles = (int)((rows + (long long)(n_groups < batch ? n_groups : batch) * (kRows - g.gq())) / kRows);
  groups->slots = (int)((all + best - 1) / best);
  w.max_splits += groups->slots;
  w.total = (size_t)batch * g.Hq * w.max_splits * (g.D + 4) * sizeof(float);
  return w;
}

// The most that a plan of up to so many requests and groups takes: fewer rows are split into more parts, so the largest batch is not
// the one with the most partials.  For b requests the row tiles are max(b G / kRows, groups), any count from `lo` to n_groups.
size_t kv8_shared_ws_bytes(const Geom& g, int batch, int n_groups, int max_shared, int max_own) {
  const long long all = prefix_all(g, max_shared);
  auto slots = [&](long long row_tiles) {
    const long long per = prefix_units(g, row_tiles, all);
    return (all + per - 1) / per;
  };
  long long places = 0, next = n_groups, among = 0;       // among: the most slots of row tiles next + 1 .. n_groups
  for (long long b = batch; b > 0; --b) {
    const long long tiles = b * g.gq() / kRows, lo = tiles > 1 ? tiles : 1;
    for (; next >= lo; --next) among = among > slots(next) ? among : slots(next);
    const long long its = b * (kv8_plan(g, (int)b, max_own / g.P).max_splits + (lo <= n_groups ? among : slots(lo)));
    places = its > places ? its : places;
  }
  return (size_t)places * g.Hq * (g.D + 4) * sizeof(float);
}

template <int D, int FMT>
static int launch_prefix(const Kv8DecodeArgs& a, cudaStream_t s, bool pdl) {
  const dim3 grid(a.groups.slots * a.groups.max_tiles * a.g.Hkv);
  auto go = [&](auto kern, size_t smem) {
    const cudaError_t e = ensure_smem_limit(kern, smem);
    if (e != cudaSuccess) return (int)e;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, pdl, a);
  };
  if (a.out_dtype == kDtypeF32)
    return a.q_dtype == kDtypeF32 ? go(kv8_prefix_kernel<D, FMT, true, 2>, Lay<D, true, 2>::kSmem)
                                  : go(kv8_prefix_kernel<D, FMT, false, 2>, Lay<D, false, 2>::kSmem);
  return a.q_dtype == kDtypeF32 ? go(kv8_prefix_kernel<D, FMT, true, 1>, Lay<D, true, 1>::kSmem)
                                : go(kv8_prefix_kernel<D, FMT, false, 1>, Lay<D, false, 1>::kSmem);
}

int launch_kv8_shared_prefix(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? launch_prefix<128, kKv8Int8>(a, s, pdl) : launch_prefix<128, kKv8E4m3>(a, s, pdl);
  return a.fmt == kKv8Int8 ? launch_prefix<64, kKv8Int8>(a, s, pdl) : launch_prefix<64, kKv8E4m3>(a, s, pdl);
}

}  // namespace oscar
