// Decode attention of requests that share a prefix: the shared pages of a group, read once for all of its requests.
//
// Row r of a group is a query head of one of its requests.  Over a split of the shared pages a CTA forms, for up to 128 rows
// of a kv head at once,
//     S = Q K^T,   p = 2^(s - m),   l = sum p,   O = P V,
// and leaves (m, l, O) for the merge with the partials of the requests' own pages and tail rows, which the decode kernel forms.
// The codes of a page are read once per 128 rows instead of once per 8; 4 d flops per token and row are on the tensor cores
// (tcgen05), so it is bound by memory up to 128 rows of a kv head and by the tensor cores and the exponentials beyond.
//
// Roles in a CTA, around two buffers of a token tile (128 tokens; 64 for float32 queries, whose three terms take the room):
//   8 warps   codes from global memory through registers, two tiles ahead, to BF16 keys and f16 values in shared memory.  Both
//             are exact.  Rows are tokens: for S the channels of a row are the contracted dimension, for O the tokens are.
//   1 warp    issues S(i) and then O += P(i - 1) V(i - 1).
//   4 warps   a thread per row: S from tensor memory, the running maximum and sum, P to tensor memory.
// Queries are BF16 operands as they are (float32 ones sums of three), brought near 2^14 by a power of two.  A score is scaled in
// the exponent's multiplication by its page's scale, a weight by its page's V scale after it.  Weights are f16: one number (11
// bits) for BF16 outputs, which are rounded to 8 bits at the end, and two (22 bits) for float32 ones.
#include <cuda.h>

#include "kv8.cuh"

namespace oscar {
namespace {

#include "tc_common.cuh"

constexpr int kSoft = 4, kConv = 8;                       // warps
constexpr int kThreads = 32 * (kSoft + kConv + 1);
constexpr int kRows = 128;
constexpr int kMostPages = 2048;                          // pages of a split
// Tensor memory: scores of two tiles, sums, weights.
constexpr uint32_t kColS = 0, kColO = 256, kColP = 384, kCols = 512;
// A row's reference exponent follows its maximum when it is kLag behind; V scales are relative to a power of two that follows
// the largest when it is 2^kScaleLag behind; a weight of 1 at scale 1 is 2^kBase: below 2^(kLag + kScaleLag + 1 + kBase) = 2^15.
constexpr float kLag = 8.f;
constexpr int kScaleLag = 3, kBase = 3;

template <int D, bool QF32>
struct Lay {
  static constexpr int NT = QF32 ? 64 : 128;              // tokens of a tile
  static constexpr int QT = QF32 ? 3 : 1;                 // BF16 terms of a query
  static constexpr int kQ = kRows * D * 2, kKV = NT * D * 2;
  static constexpr int oQ = 0, oK = oQ + QT * kQ, oV = oK + 2 * kKV, oPages = oV + 2 * kKV;
  static constexpr int kSmem = oPages + kMostPages * 4 + 1024;
  static constexpr int kTasks = NT * D / 16 / (32 * kConv);  // 16-byte chunks of keys (and of values) a thread takes of a tile
};

struct Shared {
  uint64_t k_full[2], k_empty[2], v_full[2], sc_full[2], s_full[2], p_full[2], pv_done[2], end;
  float ks[2][8], vs[2][8];      // per 16 tokens: K scale, V scale relative to 2^E (2^kBase at 1)
  float ratio[2];                // 2^(the E before - E)
  int mask[2], e[2];
  uint32_t tmem;
  int lo, size, shared, tile, holder, abort;
};

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

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

template <int D, int FMT, bool QF32>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefix_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  using L = Lay<D, QF32>;
  constexpr int NT = L::NT, QT = L::QT, NG = NT / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* page_ids = reinterpret_cast<int*>(smem + L::oPages);
  const Geom& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, split = blockIdx.x / a.groups.max_tiles, tile = blockIdx.x % a.groups.max_tiles;
  const int G = g.gq(), P = g.P;
  const int terms = a.out_dtype == kDtypeF32 ? 2 : 1;     // of a weight
  // The grid before this one is the decode kernel of the same call: all that this one reads was there before it.  What it leaves
  // (for the merge, which follows this grid) is waited for at the end.
  pdl_launch_dependents();
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.k_full[b], kConv);
      mbar_init(&sh.k_empty[b], 1);
      mbar_init(&sh.v_full[b], kConv);
      mbar_init(&sh.sc_full[b], 1);
      mbar_init(&sh.s_full[b], 1);
      mbar_init(&sh.p_full[b], kSoft);
      mbar_init(&sh.pv_done[b], 1);
    }
    mbar_init(&sh.end, 1);
    sh.abort = 0;
    fence_barrier_init();
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
  int req = 0, head = 0;
  if (pages > 0 && warp < kSoft) {
    const int r = sh.tile * kRows + tid;
    req = sh.lo + r / G;
    head = h * G + r % G;
    if (r < sh.size * G) {
      const int n = a.seq_lens[req];
      valid = n > 0 && kv8_own_sound(a, n, sh.shared);
    }
  }
  if (!__syncthreads_or(valid)) {                         // no rows, or no pages for them
    pdl_wait();
    return;
  }
  if (warp == kSoft + kConv) tmem_alloc(&sh.tmem, kCols);
  {
    const int* bt = a.block_table + (size_t)sh.holder * a.bt_stride;
    for (int i = tid; i < pages; i += kThreads) {
      int pid = e0 + i < a.bt_stride ? bt[e0 + i] : -1;
      if (pid < 0 || pid >= g.num_pages) {
        flag_error(a.status, kDevBadPage);
        pid = -1;
      }
      page_ids[i] = pid;
    }
  }
  float qs = 0.f;                                         // what a score's raw sum is multiplied by, but for the page's scale
  const bool live = __any_sync(0xffffffffu, valid);
  if (warp < kSoft && live) {
    const size_t at = (size_t)req * a.q_stride + (size_t)head * D;
    float big = 0.f;
    if (valid)
      for (int c = 0; c < D; c += 4) {
        const float4 x = kv8_load4<QF32>(a.q, at + c);
        big = fmaxf(fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
      }
    float up, down;
    power_of_two(big, &up, &down);
    constexpr double kScale = 1.4426950408889634 / (D == 128 ? 11.313708498984761 : 8.0);
    qs = down * (float)kScale;
#pragma unroll 2
    for (int c = 0; c < D; c += 8) {
      float x[8] = {};
      if (valid) {
        const float4 u = kv8_load4<QF32>(a.q, at + c), w = kv8_load4<QF32>(a.q, at + c + 4);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] *= up;
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = pack_bf162(x[2 * k], x[2 * k + 1]);
          x[2 * k] -= bf16_lo(w[k]);
          x[2 * k + 1] -= bf16_hi(w[k]);
        }
        *reinterpret_cast<uint4*>(smem + L::oQ + t * L::kQ + sw128_offset(tid, c, kRows)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int tiles = (pages * P + NT - 1) / NT;
  bool good = true;

  if (warp < kSoft) {
    // ---------------------------------------------------------------- softmax
    const uint32_t base = tmem + ((uint32_t)warp << 21);  // 32 lanes a warp
    const int p_bufs = terms * NT <= 128 ? 2 : 1;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < tiles; ++i) {
      const int b = i & 1, ph = (i >> 1) & 1;
      good = mbar_wait_bounded(&sh.s_full[b], ph, a.status) && mbar_wait_bounded(&sh.sc_full[b], ph, a.status);
      good = __all_sync(0xffffffffu, good);
      if (!good) break;
      tc_fence_after();
      if (live) {
        const uint32_t s_at = base + kColS + 128 * b, p_at = base + kColP + (p_bufs == 2 ? b * terms * (NT / 2) : 0);
        const int mask = sh.mask[b];
        const bool all = mask == (1 << NG) - 1;
        float f[NG], cm[NG], top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NT / 32; ++c) {
          float v[32];
          tmem_ld32(s_at + 32 * c, v);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = 2 * c + u;
            float x = v[16 * u];
#pragma unroll
            for (int j = 1; j < 16; ++j) x = fmaxf(x, v[16 * u + j]);
            f[k] = sh.ks[b][k] * qs;
            cm[k] = all || (mask >> k & 1) ? x : -INFINITY;
            top = fmaxf(top, __fmul_rd(cm[k], f[k]));
          }
        }
        const float ratio = sh.ratio[b];
        const bool follow = top > m + kLag || (m == -INFINITY && top > m);
        if (i == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, follow || ratio != 1.f)) {
          const float m_new = follow ? top : m, alpha = follow ? ex2(m - m_new) : 1.f;
          m = m_new;
          l *= alpha;
          good = mbar_wait_bounded(&sh.pv_done[b ^ 1], ((i - 1) >> 1) & 1, a.status);
          good = __all_sync(0xffffffffu, good);
          if (!good) break;
          tc_fence_after();
          const float scale = alpha * ratio;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float v[32];
            tmem_ld32(base + kColO + c, v);
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j] * scale);
            tmem_st32(base + kColO + c, w);
          }
          tmem_wait_st();
        }
        if (i >= p_bufs) {                                // the sums of the tile whose weights were here
          const int j = i - p_bufs;
          good = mbar_wait_bounded(&sh.pv_done[j & 1], (j >> 1) & 1, a.status);
          good = __all_sync(0xffffffffu, good);
          if (!good) break;
          tc_fence_after();
        }
        const float ref = m == -INFINITY ? 0.f : m;
        // Where scores are so large that a last place of one counts, distances are formed from the raw sums: 0 at a page's largest.
        const bool far = fabsf(ref) >= 4194304.f, any_far = __any_sync(0xffffffffu, far);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < NT / 32; ++c) {
          float v[32];
          tmem_ld32(s_at + 32 * c, v);
          if (!all) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(mask >> (2 * c + j / 16) & 1)) v[j] = -INFINITY;
          }
          uint32_t hi[16], lo[16];
          float part[2] = {0.f, 0.f};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int k = 2 * c + u;
            const float vs = sh.vs[b][k];
            const float bias = far ? fminf(fmaf(cm[k], f[k], -ref), kLag) : -ref;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = v[16 * u + 2 * j + e];
                if (any_far) x = far && cm[k] > -INFINITY ? x - cm[k] : x;
                const float p = ex2(fmaf(x, f[k], bias));
                part[e] += p;
                w[e] = p * vs;
              }
              hi[8 * u + j] = pack_half2(w[0], w[1]);
              const __half2 hh = *reinterpret_cast<const __half2*>(&hi[8 * u + j]);
              lo[8 * u + j] = pack_half2(w[0] - __low2float(hh), w[1] - __high2float(hh));
            }
          }
          sum += part[0] + part[1];
          tmem_st16(p_at + 16 * c, hi);
          if (terms == 2) tmem_st16(p_at + NT / 2 + 16 * c, lo);
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[b]);
    }
    // ---------------------------------------------------------------- the split's partial
    if (good) {
      good = mbar_wait_bounded(&sh.pv_done[(tiles - 1) & 1], ((tiles - 1) >> 1) & 1, a.status);
      good = __all_sync(0xffffffffu, good);
      tc_fence_after();
    }
    if (good && live) {
      const float scale = pow2(sh.e[(tiles - 1) & 1] - kBase);
      float* pp = a.part + (((size_t)req * g.Hq + head) * a.wl.max_splits + split) * (D + 4);
      if (valid) *reinterpret_cast<float2*>(pp) = make_float2(l == l ? m : INFINITY, l);  // (a NaN must not look like no partial)
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float v[32];
        tmem_ld32(base + kColO + c, v);
        if (valid)
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(pp + 4 + c + j) = make_float4(v[j] * scale, v[j + 1] * scale, v[j + 2] * scale, v[j + 3] * scale);
      }
    }
  } else if (warp < kSoft + kConv) {
    // ---------------------------------------------------------------- codes to operands
    constexpr int T = L::kTasks;
    const int ct = tid - 32 * kSoft, p = ct & 7, log_p = 31 - __clz(P);
    const Kv8Geom kg{P, D, g.Hkv};
    const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
    const size_t page_bytes = kg.page_bytes();
    const int pages_per_tile = NT >> log_p;
    // 128-byte line ct / 8 (+ 32, ...) of a tile's codes: its first token, and the logical chunk at place p of it
    const int t0 = D == 128 ? ct >> 3 : 2 * (ct >> 3);    // (+ 32 or 64 tokens a task: the turns stay)
    constexpr int kStep = D == 128 ? 32 : 64;
    auto dest = [&](int turn) {                           // bytes of the chunk's first half, and what leads to its second
      const int idx = p ^ turn, t = D == 128 ? t0 : t0 + (idx >> 2), j = D == 128 ? idx : idx & 3;
      const int u = D == 128 ? j >> 2 : 0;                // (which half goes first: eight lanes then touch every bank once)
      return (uint32_t)((D == 128 ? (j >> 2) * NT * 128 : 0) + t * 128 + (((2 * (j & 3) + u) ^ (t & 7)) << 4)) | (u ? 0x80000000u : 0u);
    };
    const uint32_t dk = dest(D == 128 ? 4 * (t0 & 1) : 0), dv = dest(2 * ((t0 >> 1) & 3));
    const uint32_t nothing = FMT == kKv8Int8 ? 0x80808080u : 0u;
    uint4 kw[2][T], vw[2][T];
    float2 sc[2] = {};
    bool there[2] = {};
    auto load = [&](int i, uint4 (&x)[T], bool is_v) {
#pragma unroll
      for (int k = 0; k < T; ++k) {
        const int t = t0 + k * kStep, e = i * pages_per_tile + (t >> log_p);
        const int pid = e < pages ? page_ids[e] : -1;
        x[k] = make_uint4(nothing, nothing, nothing, nothing);
        if (pid >= 0)
          x[k] = __ldg(reinterpret_cast<const uint4*>(layer + pid * page_bytes + (is_v ? P * D : 0) + (t & (P - 1)) * D + p * 16));
      }
    };
    auto load_scale = [&](int i, float2& s, bool& some) {  // lane k: of the tile's k-th 16 tokens
      if (warp != kSoft || lane >= NG) return;
      const int e = i * pages_per_tile + ((lane * 16) >> log_p);
      const int pid = e < pages ? page_ids[e] : -1;
      some = pid >= 0;
      s = make_float2(1.f, 0.f);
      if (some) s = __ldg(reinterpret_cast<const float2*>(layer + pid * page_bytes + kg.scale_off()));
    };
    auto store = [&](uint8_t* to, uint32_t d, const uint4 (&x)[T], bool is_v) {
      const bool second = d >> 31;
      d &= 0x7FFFFFFFu;
#pragma unroll
      for (int k = 0; k < T; ++k) {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[2 * j] = is_v ? kv8_pair<FMT, 0>(w[j]) : bf16_pair<FMT, 0>(w[j]);
          y[2 * j + 1] = is_v ? kv8_pair<FMT, 1>(w[j]) : bf16_pair<FMT, 1>(w[j]);
        }
        const uint4 first = make_uint4(y[0], y[1], y[2], y[3]), next = make_uint4(y[4], y[5], y[6], y[7]);
        uint8_t* at = to + d + k * kStep * 128;
        *reinterpret_cast<uint4*>(at) = second ? next : first;
        *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(reinterpret_cast<uintptr_t>(at) ^ 16)) = second ? first : next;
      }
    };
    int e_ref = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      load(b, kw[b], false);
      load(b, vw[b], true);
      load_scale(b, sc[b], there[b]);
    }
    for (int i0 = 0; i0 < tiles && good; i0 += 2) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int i = i0 + b;
        if (i >= tiles || !good) continue;
        if (i >= 2) good = mbar_wait_bounded(&sh.k_empty[b], ((i >> 1) - 1) & 1, a.status);
        good = __all_sync(0xffffffffu, good);
        if (!good) continue;
        store(smem + L::oK + b * L::kKV, dk, kw[b], false);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full[b]);
        load(i + 2, kw[b], false);
        if (i >= 2) good = mbar_wait_bounded(&sh.pv_done[b], ((i >> 1) - 1) & 1, a.status);
        good = __all_sync(0xffffffffu, good);
        if (!good) continue;
        if (warp == kSoft) {
          const unsigned mask = __ballot_sync(0xffffffffu, lane < NG && there[b]);
          int e = lane < NG ? max((int)(__float_as_uint(sc[b].y) >> 23) - 127, -110) : -110;
          e = __reduce_max_sync(0xffffffffu, e);
          const int e_new = i == 0 || e > e_ref + kScaleLag ? e : e_ref;
          if (lane < NG) {
            sh.ks[b][lane] = sc[b].x;
            sh.vs[b][lane] = sc[b].y * pow2(kBase - e_new);
          }
          if (lane == 0) {
            sh.ratio[b] = i == 0 ? 1.f : exp2f((float)(e_ref - e_new));
            sh.mask[b] = (int)mask;
            sh.e[b] = e_new;
          }
          e_ref = e_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.sc_full[b]);
          load_scale(i + 2, sc[b], there[b]);
        }
        store(smem + L::oV + b * L::kKV, dv, vw[b], true);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full[b]);
        load(i + 2, vw[b], true);
      }
    }
  } else {
    // ---------------------------------------------------------------- MMA issue
    constexpr uint32_t kIdescS = idesc_bf16_f32(kRows, NT);
    constexpr uint32_t kIdescO = idesc_f16_f32(kRows, D) | (1u << 16);  // the second operand's contracted dimension along its rows
    const uint32_t q_at = smem_u32(smem + L::oQ);
    const int p_bufs = terms * NT <= 128 ? 2 : 1;
    for (int i = 0; i <= tiles; ++i) {
      if (i < tiles) {
        const int b = i & 1;
        good = mbar_wait_bounded(&sh.k_full[b], (i >> 1) & 1, a.status);
        good = __all_sync(0xffffffffu, good);
        if (!good) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t k_at = smem_u32(smem + L::oK + b * L::kKV);
#pragma unroll
          for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma(tmem + kColS + 128 * b, smem_desc_sw128(q_at + t * L::kQ + (kk >> 2) * (kRows * 128) + (kk & 3) * 32),
                     smem_desc_sw128(k_at + (kk >> 2) * (NT * 128) + (kk & 3) * 32), kIdescS, t || kk);
          tc_commit(&sh.s_full[b]);
          tc_commit(&sh.k_empty[b]);
        }
        __syncwarp();
      }
      if (i > 0) {
        const int j = i - 1, b = j & 1, ph = (j >> 1) & 1;
        good = mbar_wait_bounded(&sh.p_full[b], ph, a.status) && mbar_wait_bounded(&sh.v_full[b], ph, a.status);
        good = __all_sync(0xffffffffu, good);
        if (!good) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t v_at = smem_u32(smem + L::oV + b * L::kKV), p_at = tmem + kColP + (p_bufs == 2 ? b * terms * (NT / 2) : 0);
          for (int t = 0; t < terms; ++t)
#pragma unroll
            for (int kk = 0; kk < NT / 16; ++kk)
              tc_mma_ts(tmem + kColO, p_at + t * (NT / 2) + 8 * kk, desc_rows(v_at + kk * 2048, NT * 128), kIdescO, j || t || kk);
          tc_commit(&sh.pv_done[b]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {                                      // nothing is under way when the tensor memory is freed
      tc_commit(&sh.end);
      (void)mbar_wait_bounded(&sh.end, 0, a.status);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoft + kConv) tmem_dealloc(tmem, kCols);
  pdl_wait();
}

}  // namespace

Kv8DecodeWs kv8_shared_plan(const Geom& g, int batch, int n_groups, int max_shared, int max_own, Kv8Groups* groups, int* own_splits) {
  Kv8DecodeWs w = kv8_plan(g, batch, max_own / g.P);
  *own_splits = w.max_splits;
  // The split that takes the fewest rounds of (its units + 3, a CTA's start and end).
  const long long tiles = ((long long)max_shared * g.P + kPrefixUnit - 1) / kPrefixUnit;
  const long long rows = (long long)batch * g.gq(), row_tiles = rows / kRows > n_groups ? rows / kRows : n_groups;
  const long long pairs = row_tiles * g.Hkv > 0 ? row_tiles * g.Hkv : 1;
  const long long most = (long long)kMostPages * g.P / kPrefixUnit;
  const long long all = tiles > 0 ? tiles : 1;
  long long best = most < all ? most : all, cost = -1;
  for (long long rounds = 1; rounds <= 16; ++rounds) {    // as many splits as fill that many rounds
    const long long fit = 152 * rounds / pairs, splits = fit < all ? fit : all;
    if (splits == 0) continue;
    const long long per = (all + splits - 1) / splits;
    const long long c = ((pairs * ((all + per - 1) / per) + 151) / 152) * (per + 3);
    if (per <= most && (cost < 0 || c < cost)) best = per, cost = c;
  }
  groups->n = n_groups;
  groups->max_shared = max_shared;
  groups->max_own = max_own;
  groups->units_per_split = (int)best;
  groups->max_tiles = (int)(rows / kRows + n_groups);
  groups->slots = (int)((all + best - 1) / best);
  w.max_splits += groups->slots;
  w.total = (size_t)batch * g.Hq * w.max_splits * (g.D + 4) * sizeof(float);
  return w;
}

template <int D, int FMT>
static int launch_prefix(const Kv8DecodeArgs& a, cudaStream_t s, bool pdl) {
  const dim3 grid(a.groups.slots * a.groups.max_tiles, a.g.Hkv);
  auto go = [&](auto kern, size_t smem) {
    const cudaError_t e = ensure_smem_limit(kern, smem);
    if (e != cudaSuccess) return (int)e;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, pdl, a);
  };
  return a.q_dtype == kDtypeF32 ? go(kv8_prefix_kernel<D, FMT, true>, Lay<D, true>::kSmem)
                                : go(kv8_prefix_kernel<D, FMT, false>, Lay<D, false>::kSmem);
}

int launch_kv8_shared_prefix(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? launch_prefix<128, kKv8Int8>(a, s, pdl) : launch_prefix<128, kKv8E4m3>(a, s, pdl);
  return a.fmt == kKv8Int8 ? launch_prefix<64, kKv8Int8>(a, s, pdl) : launch_prefix<64, kKv8E4m3>(a, s, pdl);
}

}  // namespace oscar
