// 8-bit cache write and append.
//
// A page is quantised once, when its last token arrives.  For each block (page, kv head, K or V), with m the largest
// finite |x| and M the largest code:
//     scale = m / M,   code = round(x M / m),   and for K: lo, hi = the smallest and largest code of each channel.
// Rounding is monotone, so lo and hi are the codes of a channel's smallest and largest x.  It reads 2 d (or 4 d) bytes
// and writes d + (2 d + 16) / P bytes per K or V row, so it is bound by memory: a group of warps holds a block's P x d
// values in registers as BF16 pairs for both passes over them (the maximum, then the codes), while the next block's rows
// travel to shared memory as one tile.
// 8 x 32K tokens, 8 kv heads of 128 channels, BF16 to E4M3: 249 us, 6.5 TB/s, 0.96 of the measured copy bandwidth.  8 x 8K:
// BF16 0.88 to 0.90 of it at d = 128, 0.71 to 0.78 at d = 64, whose 39 us hold 5 of start and end; float32 rows 0.90 to 0.94
// and 0.83 to 0.89 (0.55 to 0.61 with each thread's 16-byte asynchronous copies instead of tiles, 165 us instead of 107: the
// copies' instructions and their bank conflicts filled the load/store queue).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "kv8.cuh"

namespace oscar {
namespace {

#include "tc_common.cuh"

constexpr int kThreads = 256;
struct Item {
  int b, slot;           // request, its slot
  int page, pages;       // logical pages completed by this item: page, page + 1, ... (pages may be 0)
  int tail0, tail1;      // tokens copied into the tail
  int start, row0;       // first new token and its input row
};

// What request b of the call asks for, if it is sound: its items (0: nothing, or flagged).
// An item is a span of up to `span` pages.
__device__ __forceinline__ int request(const Kv8WriteArgs& a, int span, int b, int* start, int* len, int* row0, int* slot) {
  const Geom& g = a.g;
  *start = a.start_pos[b];
  *row0 = a.cu_seqlens ? a.cu_seqlens[b] : b;
  const long long l = a.cu_seqlens ? (long long)a.cu_seqlens[b + 1] - *row0 : (*start == -1 ? 0 : 1);
  *slot = a.req_slot[b];
  if (l == 0) return 0;
  if (*start < 0 || *row0 < 0 || l < 0 || *row0 + l > a.total_tokens || *start + l > (long long)g.max_pages_per_req * g.P) {
    flag_error(a.status, kDevBadLen);
    return 0;
  }
  if (*slot < 0 || *slot >= g.max_req) {
    flag_error(a.status, kDevBadSlot);
    return 0;
  }
  *len = (int)l;
  return max(((*start + *len) / g.P - *start / g.P + span - 1) / span, 1);
}

// The j-th item of a request.  Item 0 also stores the rows of the page that stays incomplete, after it has read the rows
// of the old one from the same tail.  An append keeps its row in the tail even when it completes the page.
__device__ __forceinline__ Item item_of(const Kv8WriteArgs& a, int span, int b, int j, int start, int len, int row0, int slot) {
  const int P = a.g.P, first = start / P, last = (start + len) / P;
  Item it;
  it.b = b;
  it.slot = slot;
  it.page = first + j * span;
  it.pages = min(span, last - it.page);
  it.start = start;
  it.row0 = row0;
  it.tail0 = j == 0 ? (a.cu_seqlens ? max(last * P, start) : start) : 0;
  it.tail1 = j == 0 ? start + len : 0;
  return it;
}

// One warp finds the item of CTA x.  A request of len rows completes at most len / P + 1 pages, which is at most
// len / (P span) + 1 spans, so request b has the CTAs from cu[b] / (P span) + b on, as many as it can need (the rest end at
// once), and a 32-way search over that bound finds b.
// CTA x also checks request x: one that no CTA works on is reported all the same.
__device__ bool find_item(const Kv8WriteArgs& a, int span, int x, Item* out) {
  const int lane = threadIdx.x & 31, rows = a.g.P * span;
  int start = 0, len = 0, row0 = 0, slot = 0;
  if (a.batch <= 32) {  // every lane its request, one round of loads
    const int cnt = lane < a.batch ? request(a, span, lane, &start, &len, &row0, &slot) : 0;
    const int first = row0 / rows + lane;
    const unsigned hit = __ballot_sync(0xffffffffu, lane < a.batch && first <= x);
    if (hit == 0) return false;
    const int l = 31 - __clz(hit), j = x - __shfl_sync(0xffffffffu, first, l);
    if (j < 0 || j >= __shfl_sync(0xffffffffu, cnt, l)) return false;
    *out = item_of(a, span, l, j, __shfl_sync(0xffffffffu, start, l), __shfl_sync(0xffffffffu, len, l), __shfl_sync(0xffffffffu, row0, l),
                   __shfl_sync(0xffffffffu, slot, l));
    return true;
  }
  if (x < a.batch) (void)request(a, span, x, &start, &len, &row0, &slot);
  int b = 0, n = a.batch;
  while (n > 1) {
    const int step = (n + 31) / 32, at = b + lane * step;
    const bool below = lane * step < n && a.cu_seqlens[at] / rows + at <= x;
    const unsigned hit = __ballot_sync(0xffffffffu, below);
    if (hit == 0) return false;
    const int l = 31 - __clz(hit);
    b += l * step;
    n = min(step, n - l * step);
  }
  const int j = x - (a.cu_seqlens[b] / rows + b);
  if (j < 0 || j >= request(a, span, b, &start, &len, &row0, &slot)) return false;
  *out = item_of(a, span, b, j, start, len, row0, slot);
  return true;
}

// The code nearest x M / m from one multiplication by a float32 near M / m.  A quotient of numbers of 8 and 7 significant
// bits by one of 8 is a tie T between two codes or far from one: x M - T m, where it is not 0, is a whole number of last
// places of numbers of at most 16 bits (INT8: T has 8, m 8) or 13 (E4M3: T has 5), so the quotient misses T by 2^-16 or
// 2^-13 of T at least.  The factor is a little too large (by up to 9 half steps of 2^-24: the approximate reciprocal is off
// by 2 at most, a rounding by 1, and three last places, 3 to 6 of them, are added), so that dropping the product's last 5
// or 8 bits takes what belongs on a tie back to it and carries nothing across one.  Then E4M3 has the hardware's
// rounding, and INT8 the sum with 1.5 2^23 + 128, whose low byte is the code's.
template <int FMT>
struct Quotient {
  float f;
  __device__ __forceinline__ explicit Quotient(float m) {  // 2^-100 <= m
    // m in [2^k, 2^(k+1)) is brought to [2, 4) and back by powers of two, so that nothing leaves the normal numbers
    const int k = (int)(__float_as_uint(m) >> 23) - 127;
    const float s = __uint_as_float((uint32_t)(128 - k) << 23);
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(m * s));
    f = __uint_as_float(__float_as_uint(r * (FMT == kKv8Int8 ? 127.f : 448.f) * s) + 3u);
  }
  __device__ __forceinline__ float operator()(float x) const {
    return __uint_as_float(__float_as_uint(x * f) & (FMT == kKv8Int8 ? 0xffffffe0u : 0xffffff00u));
  }
  __device__ __forceinline__ uint32_t byte(float x) const { return __float_as_uint((*this)(x) + 12583040.f); }
};

// Codes of four finite values as one word.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const Quotient<FMT>& quo, uint32_t x01, uint32_t x23) {
  const float x0 = bf16_lo(x01), x1 = bf16_hi(x01), x2 = bf16_lo(x23), x3 = bf16_hi(x23);
  if constexpr (FMT == kKv8Int8) {
    return prmt(prmt(quo.byte(x0), quo.byte(x1), 0x0040u), prmt(quo.byte(x2), quo.byte(x3), 0x0040u), 0x5410u);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(quo(x1)), "f"(quo(x0)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(quo(x3)), "f"(quo(x2)));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

// Smaller and larger BF16 pairs, and the larger in magnitude (a NaN stays one).
__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t babs2(uint32_t a) { return a & 0x7fff7fffu; }

// Eight float32 values as BF16 pairs.
__device__ __forceinline__ uint4 to_bf16(const uint4& x, const uint4& y) {
  return make_uint4(pack_bf162(__uint_as_float(x.x), __uint_as_float(x.y)), pack_bf162(__uint_as_float(x.z), __uint_as_float(x.w)),
                    pack_bf162(__uint_as_float(y.x), __uint_as_float(y.y)), pack_bf162(__uint_as_float(y.z), __uint_as_float(y.w)));
}

__device__ __forceinline__ void copy_async(void* smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(src) : "memory");
}

// A block of P x D values is a group of T threads' work, V vectors of eight channels each, the channels of a thread the
// same in all of them; a CTA holds NU groups, and works on a span of NU pages: as much for any P and D.  (With one block a
// CTA, P = 16 and d = 128 ran at 0.42 of the measured copy bandwidth instead of 0.85: most of a CTA's time was its look-up
// and barriers.  Four vectors a thread instead of eight, and two units ahead, took 265 us at 8 x 32K tokens instead of 250:
// what a unit costs beside its elements counts, the kernel issues instructions 0.65 of its cycles.)
template <int D, int P>
struct Shape {
  static constexpr int V = P * D >= 2048 ? 8 : 4;
  static constexpr int T = P * D / 8 / V;
  static constexpr int NU = kThreads / T, SPAN = NU;
  static constexpr int CH = D / 8;       // threads of a row
  static constexpr int RS = T / CH;      // rows between a thread's vectors
  static_assert(T >= 32 && T % 32 == 0 && T % CH == 0, "a group is whole warps and whole rows");
  __device__ __forceinline__ static void sync(int group) {
    if constexpr (T == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
  }
};

// The row tensors of a write as tiles of P rows of one head.
struct RowMaps {
  CUtensorMap k, v;
};
struct NoMaps {};

// TILED: a write, whose pages' rows come as one tile a unit; otherwise an append, where all but the new row of a completed page
// are in the tail.
template <int D, int P, bool F32, bool TILED>
struct Ahead {
  using S = Shape<D, P>;
  static constexpr int WD = F32 && TILED ? 2 : 1;        // 16-byte words of eight values
  // units of a group on their way (BF16 rows at 8 x 8K tokens, d = 128: two 66 to 69 us, one 68 to 70)
  static constexpr int NB = F32 || !TILED ? 1 : 2;
  static constexpr int kWords = S::V * S::T * WD;        // of a unit
  // CTAs an SM.  (8 x 8K tokens, BF16 rows, a group a warp: four 42.6, 38.5 and 67.9 us at d = 64 with P = 16, 32 and d = 128
  // with P = 16, three 44.7, 39.6 and 69.1; float32 rows 57.8, 59.9 and 112 against 60.4, 56.5 and 107.)
  static constexpr int kResident = S::T == 32 && !F32 ? 4 : 3;
  static constexpr int kBytes = S::NU * NB * kWords * 16;
};

template <int D, int P, int FMT, bool F32, bool TILED>
__global__ void __launch_bounds__(kThreads, (Ahead<D, P, F32, TILED>::kResident))
    kv8_write_kernel(const __grid_constant__ Kv8WriteArgs a, const __grid_constant__ std::conditional_t<TILED, RowMaps, NoMaps> maps) {
  using S = Shape<D, P>;
  using A = Ahead<D, P, F32, TILED>;
  constexpr int W = S::T / 32;             // warps of a group
  constexpr float M = FMT == kKv8Int8 ? 127.f : 448.f;
  constexpr int kGaveUp = 0x10000;         // above every magnitude's bits: a wait of the group ran out
  __shared__ Item s_item;
  __shared__ int s_have, s_pid[S::SPAN];
  __shared__ int s_max_all[kThreads / 32], s_fin_all[kThreads / 32];
  __shared__ uint4 s_lo_all[kThreads / 32][S::CH], s_hi_all[kThreads / 32][S::CH];
  __shared__ uint64_t full_all[S::NU][A::NB];
  extern __shared__ uint8_t ahead_raw[];
  const Geom& g = a.g;
  const Kv8Geom kg{P, D, g.Hkv};
  const int group = threadIdx.x / S::T, tid = threadIdx.x % S::T, warp = tid >> 5, lane = tid & 31;   // in the group
  int* s_max = s_max_all + group * W;
  int* s_fin = s_fin_all + group * W;
  auto s_lo = s_lo_all + group * W;
  auto s_hi = s_hi_all + group * W;
  uint64_t* full = full_all[group];
  uint4* ahead = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(ahead_raw) + 127) & ~uintptr_t(127)) +
                 group * A::NB * A::kWords;
  if constexpr (TILED) {
    if (tid == 0) {
      for (int i = 0; i < A::NB; ++i) mbar_init(&full[i], 1);
      fence_barrier_init();
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 32) {
    Item it;
    bool have;
    if constexpr (TILED) {
      have = find_item(a, S::SPAN, blockIdx.x, &it);
    } else {
      int start, len, row0, slot;
      have = request(a, S::SPAN, blockIdx.x, &start, &len, &row0, &slot) > 0;
      if (have) it = item_of(a, S::SPAN, blockIdx.x, 0, start, len, row0, slot);
    }
    if (threadIdx.x == 0) {
      s_item = it;
      s_have = have;
    }
  }
  __syncthreads();
  if (!s_have) return;
  const Item it = s_item;
  const int row = tid / S::CH, ch = (tid % S::CH) * 8;   // this thread's first row and its channels
  const int k_place = kv8_place<D, false>(row, ch), v_place = kv8_place<D, true>(row, ch);
  if (threadIdx.x < it.pages) {            // (SPAN <= 8 pages)
    const int lp = it.page + threadIdx.x;
    int pid = lp < a.bt_stride ? a.block_table[(size_t)it.b * a.bt_stride + lp] : -1;
    if (pid < 0 || pid >= g.num_pages) {
      pid = -1;
      flag_error(a.status, kDevBadPage);
    }
    s_pid[threadIdx.x] = pid;
  }
  // this thread's channels of head h of input row t of K or V, as BF16 pairs
  auto input = [&](int kv, int h, int t) {
    const size_t i = (size_t)((long long)(it.row0 + (t - it.start)) * (kv ? a.v_stride : a.k_stride) + h * D + ch);
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? a.V : a.K) + i * (F32 ? 4 : 2));
    if constexpr (F32) return to_bf16(p[0], p[1]);
    return p[0];
  };
  auto tail_of = [&](int unit) {
    return a.tail + ((size_t)a.layer * g.max_req + it.slot) * kv8_tail_req_elems(g) + (size_t)unit * P * D;
  };
  // A unit is (kv head, K | V) of a page of the span.  The next one's (or two's) rows are on their way to shared memory
  // while this one's are worked on.
  const int units = 2 * g.Hkv, step = gridDim.y * S::NU;
  // (page of the span, unit) of this group's current work and of the next to fetch
  auto advance = [&](int& page, int& unit) {
    for (unit += step; unit >= units; unit -= units) ++page;
  };
  int page = 0, unit = blockIdx.y * S::NU + group;
  for (; unit >= units; unit -= units) ++page;
  int next_page = page, next_unit = unit, issued = 0, taken = 0;
  auto fetch = [&] {
    if constexpr (TILED) {                  // (one thread of the group)
      if (next_page < it.pages) {
        uint64_t* bar = &full[issued % A::NB];
        mbar_arrive_expect_tx(bar, A::kWords * 16);
        tma_load_2d_tc(ahead + issued % A::NB * A::kWords, (next_unit & 1) ? &maps.v : &maps.k, (next_unit >> 1) * D,
                       it.row0 + ((it.page + next_page) * P - it.start), bar);
        ++issued;
      }
    } else {                                // words that only this thread reads again
      if (next_page < it.pages) {
#pragma unroll
        for (int k = 0; k < S::V; ++k)
          if (row + k * S::RS < P - 1) copy_async(ahead + tid + k * S::T, tail_of(next_unit) + (size_t)(row + k * S::RS) * D + ch);
      }
    }
    advance(next_page, next_unit);
  };
  if (!TILED || tid == 0)
    for (int i = 0; i < A::NB; ++i) fetch();
  __syncthreads();                          // (the pages' ids)
  for (const int pages = max(it.pages, 1); page < pages; advance(page, unit)) {
    const int kv = unit & 1, h = unit >> 1;
    uint16_t* tail = tail_of(unit);
    if (it.pages > 0) {
      const int pid = s_pid[page];
      uint4 x[S::V];
      bool good = true;
      if constexpr (TILED) {
        good = mbar_wait_bounded(&full[taken % A::NB], (taken / A::NB) & 1, a.status);
        good = __all_sync(0xffffffffu, good);
        const uint4* from = ahead + taken % A::NB * A::kWords;
        ++taken;
#pragma unroll
        for (int k = 0; k < S::V; ++k) {
          if constexpr (F32) {  // every other four threads take their second word first: no bank is met twice
            const int i = 2 * (tid + k * S::T), turn = (tid >> 2) & 1;
            const uint4 u = from[i + turn], v = from[i + 1 - turn];
            const uint2 pu = make_uint2(pack_bf162(__uint_as_float(u.x), __uint_as_float(u.y)), pack_bf162(__uint_as_float(u.z), __uint_as_float(u.w)));
            const uint2 pv = make_uint2(pack_bf162(__uint_as_float(v.x), __uint_as_float(v.y)), pack_bf162(__uint_as_float(v.z), __uint_as_float(v.w)));
            x[k] = turn ? make_uint4(pv.x, pv.y, pu.x, pu.y) : make_uint4(pu.x, pu.y, pv.x, pv.y);
          } else {
            x[k] = from[tid + k * S::T];
          }
        }
        const int old = it.start - (it.page + page) * P;   // the page's first rows may be in the tail
        if (old > 0) {
#pragma unroll
          for (int k = 0; k < S::V; ++k)
            if (row + k * S::RS < old) x[k] = *reinterpret_cast<const uint4*>(tail + (size_t)(row + k * S::RS) * D + ch);
        }
      } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int k = 0; k < S::V; ++k)
          x[k] = row + k * S::RS < P - 1 ? ahead[tid + k * S::T] : input(kv, h, it.start);
        fetch();
      }
      // the channels' smallest and largest values (K), and from them, or directly (V), the largest magnitude
      uint4 lo = x[0], hi = x[0];
      auto fold = [&](const uint4& l, const uint4& u) {
        lo = make_uint4(bmin2(lo.x, l.x), bmin2(lo.y, l.y), bmin2(lo.z, l.z), bmin2(lo.w, l.w));
        hi = make_uint4(bmax2(hi.x, u.x), bmax2(hi.y, u.y), bmax2(hi.z, u.z), bmax2(hi.w, u.w));
      };
      uint32_t m2;
      if (!kv) {
#pragma unroll
        for (int k = 1; k < S::V; ++k) fold(x[k], x[k]);
        m2 = bmax2(bmax2(bmax2(babs2(lo.x), babs2(lo.y)), bmax2(babs2(lo.z), babs2(lo.w))),
                   bmax2(bmax2(babs2(hi.x), babs2(hi.y)), bmax2(babs2(hi.z), babs2(hi.w))));
      } else {
        m2 = 0;
#pragma unroll
        for (int k = 0; k < S::V; ++k)
          m2 = bmax2(m2, bmax2(bmax2(babs2(x[k].x), babs2(x[k].y)), bmax2(babs2(x[k].z), babs2(x[k].w))));
      }
      int big = good ? (int)__reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16)) : kGaveUp;
      if (W > 1 && lane == 0) s_max[warp] = big;
      S::sync(group);   // (and a tile's words are read)
      if constexpr (W > 1) big = (int)__reduce_max_sync(0xffffffffu, (unsigned)s_max[lane % W]);
      if constexpr (TILED) {
        if (big == kGaveUp) {  // let the tiles in flight land before the CTA ends
          if (tid == 0)
            for (int i = taken - 1; i < issued; ++i) (void)mbar_wait_bounded(&full[i % A::NB], (i / A::NB) & 1, nullptr);
          return;
        }
        if (tid == 0) fetch();
      }
      if (big >= 0x7f80) {
        // infinities and NaNs: the scale is the finite values'; an infinity becomes the largest of them, a NaN 0
        if (tid == 0) flag_error(a.status, kDevBadValue);
        int fin = 0;
        uint16_t* e = reinterpret_cast<uint16_t*>(x);
        for (int i = 0; i < 8 * S::V; ++i) {
          const int v = e[i] & 0x7fff;
          if (v < 0x7f80) fin = max(fin, v);
        }
        fin = (int)__reduce_max_sync(0xffffffffu, (unsigned)fin);
        if (lane == 0) s_fin[warp] = fin;
        S::sync(group);
        big = (int)__reduce_max_sync(0xffffffffu, (unsigned)s_fin[lane % W]);
        for (int i = 0; i < 8 * S::V; ++i) {
          const int v = e[i] & 0x7fff;
          if (v >= 0x7f80) e[i] = (uint16_t)(v == 0x7f80 ? (e[i] & 0x8000) | big : 0);
        }
        lo = hi = x[0];
#pragma unroll
        for (int k = 1; k < S::V; ++k) fold(x[k], x[k]);
      }
      const float m = __uint_as_float((uint32_t)big << 16);
      const bool some = m >= kKv8Smallest;
      const Quotient<FMT> quo(some ? m : 1.f);
      constexpr uint32_t kZero = FMT == kKv8Int8 ? 0x80808080u : 0u;
      uint8_t* block = a.pool + ((size_t)a.layer * g.num_pages + (pid < 0 ? 0 : pid)) * kg.page_bytes() + (size_t)h * kg.block_bytes();
      if (pid >= 0) {
#pragma unroll
        for (int k = 0; k < S::V; ++k) {
          uint2 code = make_uint2(kZero, kZero);
          if (some) code = make_uint2(encode4<FMT>(quo, x[k].x, x[k].y), encode4<FMT>(quo, x[k].z, x[k].w));
          // V's turn in rows k RS on: the same at RS = 8, 4 chunks off at every second k at RS = 4, 2 (k & 3) at RS = 2
          const int off = kv ? v_place ^ ((k * S::RS / 2 & 3) * 32) : k_place;
          *reinterpret_cast<uint2*>(block + off + (kv ? P * D : 0) + k * S::RS * D) = code;
        }
        if (tid == 0) reinterpret_cast<float*>(block + kg.scale_off())[kv] = some ? __fdiv_rn(m, M) : 0.f;
      }
      if (!kv) {
#pragma unroll
        for (int o = S::CH; o < 32; o <<= 1) {
          uint4 l, u;
          l.x = __shfl_xor_sync(0xffffffffu, lo.x, o), l.y = __shfl_xor_sync(0xffffffffu, lo.y, o);
          l.z = __shfl_xor_sync(0xffffffffu, lo.z, o), l.w = __shfl_xor_sync(0xffffffffu, lo.w, o);
          u.x = __shfl_xor_sync(0xffffffffu, hi.x, o), u.y = __shfl_xor_sync(0xffffffffu, hi.y, o);
          u.z = __shfl_xor_sync(0xffffffffu, hi.z, o), u.w = __shfl_xor_sync(0xffffffffu, hi.w, o);
          fold(l, u);
        }
        if (lane < S::CH) {
          s_lo[warp][lane] = lo;
          s_hi[warp][lane] = hi;
        }
        S::sync(group);
        if (tid < S::CH && pid >= 0) {
          for (int w = 0; w < W; ++w) fold(s_lo[w][tid], s_hi[w][tid]);
          uint2 l = make_uint2(kZero, kZero), u = l;
          if (some) {
            l = make_uint2(encode4<FMT>(quo, lo.x, lo.y), encode4<FMT>(quo, lo.z, lo.w));
            u = make_uint2(encode4<FMT>(quo, hi.x, hi.y), encode4<FMT>(quo, hi.z, hi.w));
            if constexpr (FMT == kKv8E4m3) {  // -0 is stored as +0
              l = make_uint2(l.x & ~__vcmpeq4(l.x, 0x80808080u), l.y & ~__vcmpeq4(l.y, 0x80808080u));
              u = make_uint2(u.x & ~__vcmpeq4(u.x, 0x80808080u), u.y & ~__vcmpeq4(u.y, 0x80808080u));
            }
          }
          *reinterpret_cast<uint2*>(block + kg.lo_off() + ch) = l;
          *reinterpret_cast<uint2*>(block + kg.hi_off() + ch) = u;
        }
      }
      S::sync(group);   // every row of the old tail is read, and the shared words are free
    }
    if (page == 0)
      for (int t = it.tail0 + row; t < it.tail1; t += S::RS) *reinterpret_cast<uint4*>(tail + (size_t)(t % P) * D + ch) = input(kv, h, t);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// [total_tokens][Hkv x D] rows in boxes of P rows of one head.  (The values pass unread, as words of their size.)
template <int D, int P>
int row_map(CUtensorMap* map, const void* base, long long row_stride, const Kv8WriteArgs& a) {
  auto encode = tensor_map_encoder();
  if (!encode) return (int)cudaErrorNotSupported;
  const bool f32 = a.dtype == kDtypeF32;
  const cuuint64_t dims[2] = {(cuuint64_t)a.g.Hkv * D, (cuuint64_t)a.total_tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)row_stride * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {D, P}, ones[2] = {1, 1};
  const CUresult r = encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(base), dims,
                            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : (int)cudaErrorInvalidValue;
}

template <int D, int P, int FMT>
int launch_write(const Kv8WriteArgs& a, cudaStream_t s, bool pdl) {
  using S = Shape<D, P>;
  const int items = a.cu_seqlens ? a.total_tokens / (P * S::SPAN) + a.batch : a.batch;
  // Several units a group where there are CTAs enough: one look-up of the item, and loads that never pause.  (A CTA for
  // each unit took 411 us at 8 x 32K tokens.  At 8 x 8K, half again as many CTAs took up to 5 % more with BF16 rows and up to
  // 4 % less with float32 rows, three quarters of them up to 5 % more.)
  const int rounds = a.cu_seqlens ? 2 * a.g.Hkv : (2 * a.g.Hkv + S::NU - 1) / S::NU;   // a CTA's, were it alone with its item
  long long per = (long long)items * rounds / (152LL * 4 * 2);
  if (per < 1) per = 1;
  if (per > rounds) per = rounds;
  const dim3 grid(items, (unsigned)((rounds + per - 1) / per));
  const bool f32 = a.dtype == kDtypeF32;
  auto go = [&](auto kern, size_t bytes, const auto& maps) {
    const size_t smem = bytes + 128;
    const cudaError_t e = ensure_smem_limit(kern, smem, true);
    return e != cudaSuccess ? (int)e : launch_pdl(kern, grid, dim3(kThreads), smem, s, pdl, a, maps);
  };
  if (!a.cu_seqlens)
    return f32 ? go(kv8_write_kernel<D, P, FMT, true, false>, Ahead<D, P, true, false>::kBytes, NoMaps{})
               : go(kv8_write_kernel<D, P, FMT, false, false>, Ahead<D, P, false, false>::kBytes, NoMaps{});
  RowMaps maps;
  int e = row_map<D, P>(&maps.k, a.K, a.k_stride, a);
  if (!e) e = row_map<D, P>(&maps.v, a.V, a.v_stride, a);
  if (e) return e;
  return f32 ? go(kv8_write_kernel<D, P, FMT, true, true>, Ahead<D, P, true, true>::kBytes, maps)
             : go(kv8_write_kernel<D, P, FMT, false, true>, Ahead<D, P, false, true>::kBytes, maps);
}

template <int D, int P>
int launch_fmt(const Kv8WriteArgs& a, cudaStream_t s, bool pdl) {
  return a.fmt == kKv8Int8 ? launch_write<D, P, kKv8Int8>(a, s, pdl) : launch_write<D, P, kKv8E4m3>(a, s, pdl);
}

template <int D>
int launch_page(const Kv8WriteArgs& a, cudaStream_t s, bool pdl) {
  if (a.g.P == 64) return launch_fmt<D, 64>(a, s, pdl);
  return a.g.P == 32 ? launch_fmt<D, 32>(a, s, pdl) : launch_fmt<D, 16>(a, s, pdl);
}

}  // namespace

int launch_kv8_write(const Kv8WriteArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.g.D == 128 ? launch_page<128>(a, s, pdl) : launch_page<64>(a, s, pdl);
}

}  // namespace oscar
