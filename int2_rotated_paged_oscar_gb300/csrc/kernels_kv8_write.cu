// 8-bit cache write and append.
//
// A page is quantised once, when its last token arrives.  For each block (page, kv head, K or V), with m the largest
// finite |x| and M the largest code:
//     scale = m / M,   code = round(x M / m),   and for K: lo, hi = the smallest and largest code of each channel.
// Rounding is monotone, so lo and hi are the codes of a channel's smallest and largest x.  It reads 2 d (or 4 d) bytes
// and writes d + (2 d + 16) / P bytes per K or V row, so it is bound by memory: one CTA holds a block's P x d values in
// registers as BF16 pairs, from 16-byte copies, for both passes over them (the maximum, then the codes).
// 8 x 32K tokens, 8 kv heads of 128 channels, BF16 to E4M3: 265 us, 6.1 TB/s, 0.90 of the measured copy bandwidth.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kMaxThreads = 256;
// Units on their way: 1, 2 and 3 took 291, 265 and 270 us for 8 x 32K tokens (8 kv heads of 128, BF16, E4M3).
constexpr int kAhead = 2;

struct Item {
  int b, page;           // request, logical page completed by this item (-1: none)
  int tail0, tail1;      // tokens copied into the tail
  int start, row0;       // first new token and its input row
};

// What request b of the call asks for, if it is sound: cnt items (0: nothing, or flagged).
__device__ __forceinline__ int request(const Kv8WriteArgs& a, int b, int* start, int* len, int* row0) {
  const Geom& g = a.g;
  *start = a.start_pos[b];
  *row0 = a.cu_seqlens ? a.cu_seqlens[b] : b;
  const long long l = a.cu_seqlens ? (long long)a.cu_seqlens[b + 1] - *row0 : (*start == -1 ? 0 : 1);
  const int slot = a.req_slot[b];
  if (l == 0) return 0;
  if (*start < 0 || *row0 < 0 || l < 0 || *row0 + l > a.total_tokens || *start + l > (long long)g.max_pages_per_req * g.P) {
    flag_error(a.status, kDevBadLen);
    return 0;
  }
  if (slot < 0 || slot >= g.max_req) {
    flag_error(a.status, kDevBadSlot);
    return 0;
  }
  *len = (int)l;
  return max((*start + *len) / g.P - *start / g.P, 1);
}

// The j-th item of a request.  A request whose chunk completes c pages has max(c, 1) items: item j quantises its j-th
// page, item 0 also stores the rows of the page that stays incomplete, after it has read the rows of the old one from
// the same tail.  An append keeps its row in the tail even when it completes the page.
__device__ __forceinline__ Item item_of(const Kv8WriteArgs& a, int b, int j, int start, int len, int row0) {
  const int P = a.g.P, first = start / P, last = (start + len) / P;
  Item it;
  it.b = b;
  it.page = first + j < last ? first + j : -1;
  it.start = start;
  it.row0 = row0;
  it.tail0 = j == 0 ? (a.cu_seqlens ? max(last * P, start) : start) : 0;
  it.tail1 = j == 0 ? start + len : 0;
  return it;
}

// One warp finds the item of CTA x.  A request of len rows completes at most len / P + 1 pages, so request b has the CTAs
// from cu[b] / P + b on, as many as it can need (the rest end at once), and a 32-way search over that bound finds b.
// CTA x also checks request x: one that no CTA works on is reported all the same.
__device__ bool find_item(const Kv8WriteArgs& a, int x, Item* out) {
  const int lane = threadIdx.x & 31, P = a.g.P;
  int start, len, row0;
  if (x < a.batch) (void)request(a, x, &start, &len, &row0);
  int b = 0, n = a.batch;
  while (n > 1) {
    const int step = (n + 31) / 32, at = b + lane * step;
    const bool below = lane * step < n && a.cu_seqlens[at] / P + at <= x;
    const unsigned hit = __ballot_sync(0xffffffffu, below);
    if (hit == 0) return false;
    const int l = 31 - __clz(hit);
    b += l * step;
    n = min(step, n - l * step);
  }
  const int j = x - (a.cu_seqlens[b] / P + b);
  if (j < 0 || j >= request(a, b, &start, &len, &row0)) return false;
  *out = item_of(a, b, j, start, len, row0);
  return true;
}

// x M / m, correctly rounded, from x (2^e M) and m 2^e in [2, 4): with r the correctly rounded reciprocal of the latter,
// one correction of x r by its exact remainder (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Numbers below float32's normal range only arise where the code is 0.
struct Quotient {
  float up, den, rec;
  __device__ __forceinline__ Quotient(float m, float M) {
    const int k = (int)(__float_as_uint(m) >> 23) - 127;  // m in [2^k, 2^(k+1)), -100 <= k <= 127
    const float s = __uint_as_float((uint32_t)(128 - k) << 23);
    up = s * M;
    den = m * s;
    rec = __frcp_rn(den);
  }
  __device__ __forceinline__ float operator()(float x) const {
    const float t = x * up, q = t * rec;
    return fmaf(-fmaf(q, den, -t), rec, q);   // (in these signs a -0 stays one)
  }
};

// Codes of four finite values as one word.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(const Quotient& quo, uint32_t x01, uint32_t x23) {
  const float y0 = quo(bf16_lo(x01)), y1 = quo(bf16_hi(x01)), y2 = quo(bf16_lo(x23)), y3 = quo(bf16_hi(x23));
  if constexpr (FMT == kKv8Int8) {
    // 1.5 2^23 + 128 + y: the sum's rounding is the code's, its low byte the stored byte
    const uint32_t a = __float_as_uint(y0 + 12583040.f), b = __float_as_uint(y1 + 12583040.f);
    const uint32_t c = __float_as_uint(y2 + 12583040.f), d = __float_as_uint(y3 + 12583040.f);
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y1), "f"(y0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y3), "f"(y2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight float32 values as BF16 pairs.
__device__ __forceinline__ uint4 to_bf16(const uint4& x, const uint4& y) {
  return make_uint4(pack_bf162(__uint_as_float(x.x), __uint_as_float(x.y)), pack_bf162(__uint_as_float(x.z), __uint_as_float(x.w)),
                    pack_bf162(__uint_as_float(y.x), __uint_as_float(y.y)), pack_bf162(__uint_as_float(y.z), __uint_as_float(y.w)));
}

__device__ __forceinline__ void copy_async(void* smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(src) : "memory");
}

// A block of P x D values: T threads, V vectors of eight channels each, the channels of a thread the same in all of them.
template <int D, int P>
struct Shape {
  static constexpr int T = P * D / 8 < kMaxThreads ? P * D / 8 : kMaxThreads;
  static constexpr int V = P * D / 8 / T;
  static constexpr int CH = D / 8;       // threads of a row
  static constexpr int RS = T / CH;      // rows between a thread's vectors
};

template <int D, int P, int FMT, bool F32>
__global__ void __launch_bounds__(Shape<D, P>::T) kv8_write_kernel(const __grid_constant__ Kv8WriteArgs a) {
  using S = Shape<D, P>;
  constexpr int W = S::T / 32;
  constexpr float M = FMT == kKv8Int8 ? 127.f : 448.f;
  __shared__ Item s_item;
  __shared__ int s_have;
  __shared__ int s_max[W], s_fin[W];
  __shared__ uint4 s_lo[W][S::CH], s_hi[W][S::CH];
  extern __shared__ uint4 ahead[];         // [kAhead][V][words][T]
  const Geom& g = a.g;
  const Kv8Geom kg{P, D, g.Hkv};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (tid < 32) {
    Item it;
    bool have;
    if (a.cu_seqlens) {
      have = find_item(a, blockIdx.x, &it);
    } else {
      int start, len, row0;
      have = request(a, blockIdx.x, &start, &len, &row0) > 0;
      if (have) it = item_of(a, blockIdx.x, 0, start, len, row0);
    }
    if (tid == 0) {
      s_item = it;
      s_have = have;
    }
  }
  __syncthreads();
  if (!s_have) return;
  const Item it = s_item;
  const int row = tid / S::CH, ch = (tid % S::CH) * 8;   // this thread's first row and its channels
  const int slot = a.req_slot[it.b];
  int pid = -1;
  if (it.page >= 0) {
    if (it.page < a.bt_stride) pid = a.block_table[(size_t)it.b * a.bt_stride + it.page];
    if (pid < 0 || pid >= g.num_pages) {
      pid = -1;
      if (tid == 0) flag_error(a.status, kDevBadPage);
    }
  }
  // eight values of an input row
  auto input_at = [&](int kv, int h, int t) -> const void* {
    const size_t i = (size_t)(it.row0 + (t - it.start)) * (size_t)(kv ? a.v_stride : a.k_stride) + (size_t)h * D + ch;
    if constexpr (F32) return static_cast<const float*>(kv ? a.V : a.K) + i;
    return static_cast<const uint16_t*>(kv ? a.V : a.K) + i;
  };
  auto input = [&](int kv, int h, int t) {  // as BF16 pairs
    const uint4* p = static_cast<const uint4*>(input_at(kv, h, t));
    if constexpr (F32) return to_bf16(p[0], p[1]);
    return p[0];
  };
  auto tail_of = [&](int unit) {
    return a.tail + ((size_t)a.layer * g.max_req + slot) * kv8_tail_req_elems(g) + (size_t)unit * P * D;
  };
  // A unit is (kv head, K | V).  The next ones' rows are on their way, by asynchronous copies into words of shared
  // memory that only this thread reads again, while this one's are worked on.
  constexpr int WD = F32 ? 2 : 1;           // 16-byte words of eight input values
  const int units = 2 * g.Hkv;
  auto fetch = [&](int i) {                 // the i-th unit of this CTA
    const int unit = blockIdx.y + i * gridDim.y;
    if (unit < units) {
      const uint16_t* tail = tail_of(unit);
#pragma unroll
      for (int k = 0; k < S::V; ++k) {
        const int r = row + k * S::RS, t = it.page * P + r;
        uint4* to = ahead + ((i % kAhead * S::V + k) * WD) * S::T + tid;
        if (t < it.start) {
          copy_async(to, tail + (size_t)r * D + ch);
        } else {
          const uint4* from = static_cast<const uint4*>(input_at(unit & 1, unit >> 1, t));
#pragma unroll
          for (int w = 0; w < WD; ++w) copy_async(to + w * S::T, from + w);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (it.page >= 0)
    for (int i = 0; i < kAhead; ++i) fetch(i);
  for (int i = 0, unit = blockIdx.y; unit < units; ++i, unit += gridDim.y) {
    const int kv = unit & 1, h = unit >> 1;
    uint16_t* tail = tail_of(unit);
    if (it.page >= 0) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      uint4 x[S::V];
#pragma unroll
      for (int k = 0; k < S::V; ++k) {
        const uint4* from = ahead + ((i % kAhead * S::V + k) * WD) * S::T + tid;
        x[k] = from[0];
        if constexpr (F32) {
          if (it.page * P + row + k * S::RS >= it.start) x[k] = to_bf16(x[k], from[S::T]);
        }
      }
      fetch(i + kAhead);
      uint32_t m2 = 0;
#pragma unroll
      for (int k = 0; k < S::V; ++k) {
        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu),
                                   __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu)));
      }
      int big = (int)__reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
      if (lane == 0) s_max[warp] = big;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) big = max(big, s_max[w]);
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
        __syncthreads();
        big = 0;
        for (int w = 0; w < W; ++w) big = max(big, s_fin[w]);
        for (int i = 0; i < 8 * S::V; ++i) {
          const int v = e[i] & 0x7fff;
          if (v >= 0x7f80) e[i] = (uint16_t)(v == 0x7f80 ? (e[i] & 0x8000) | big : 0);
        }
      }
      const float m = __uint_as_float((uint32_t)big << 16);
      const bool some = m >= kKv8Smallest;
      const Quotient quo(some ? m : 1.f, M);
      constexpr uint32_t kZero = FMT == kKv8Int8 ? 0x80808080u : 0u;
      uint8_t* block = a.pool + ((size_t)a.layer * g.num_pages + (pid < 0 ? 0 : pid)) * kg.page_bytes() + (size_t)h * kg.block_bytes();
      if (pid >= 0) {
#pragma unroll
        for (int k = 0; k < S::V; ++k) {
          const int r = row + k * S::RS;
          uint2 code = make_uint2(kZero, kZero);
          if (some) code = make_uint2(encode4<FMT>(quo, x[k].x, x[k].y), encode4<FMT>(quo, x[k].z, x[k].w));
          uint8_t* at = kv ? block + kg.v_off() + kv8_place<D, true>(r, ch) : block + kv8_place<D, false>(r, ch);
          *reinterpret_cast<uint2*>(at) = code;
        }
        if (tid == 0) reinterpret_cast<float*>(block + kg.scale_off())[kv] = some ? __fdiv_rn(m, M) : 0.f;
      }
      if (!kv) {
        uint4 lo = x[0], hi = x[0];
        auto fold = [&](const uint4& l, const uint4& u) {
          lo = make_uint4(bmin2(lo.x, l.x), bmin2(lo.y, l.y), bmin2(lo.z, l.z), bmin2(lo.w, l.w));
          hi = make_uint4(bmax2(hi.x, u.x), bmax2(hi.y, u.y), bmax2(hi.z, u.z), bmax2(hi.w, u.w));
        };
#pragma unroll
        for (int k = 1; k < S::V; ++k) fold(x[k], x[k]);
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
        __syncthreads();
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
      __syncthreads();   // every row of the old tail is read, and the shared words are free
    }
    for (int t = it.tail0 + row; t < it.tail1; t += S::RS) *reinterpret_cast<uint4*>(tail + (size_t)(t % P) * D + ch) = input(kv, h, t);
  }
}

template <int D, int P, int FMT>
int launch_write(const Kv8WriteArgs& a, cudaStream_t s, bool pdl) {
  const int items = a.cu_seqlens ? a.total_tokens / P + a.batch : a.batch;
  // several units a CTA where there are CTAs enough: one look-up of the item, and loads that never pause
  // (16 units each at 8 x 32K tokens: 265 us, 8 each 271 us; one each without prefetch 411 us)
  const int units = 2 * a.g.Hkv;
  long long per = (long long)items * units / (152LL * 4 * 4);
  if (per < 1) per = 1;
  if (per > units) per = units;
  const dim3 grid(items, (unsigned)((units + per - 1) / per));
  using S = Shape<D, P>;
  const bool f32 = a.dtype == kDtypeF32;
  const size_t smem = (size_t)kAhead * S::V * S::T * (f32 ? 2 : 1) * sizeof(uint4);
  auto go = [&](auto kern) {
    const cudaError_t e = ensure_smem_limit(kern, smem, true);
    return e != cudaSuccess ? (int)e : launch_pdl(kern, grid, dim3(S::T), smem, s, pdl, a);
  };
  return f32 ? go(kv8_write_kernel<D, P, FMT, true>) : go(kv8_write_kernel<D, P, FMT, false>);
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
