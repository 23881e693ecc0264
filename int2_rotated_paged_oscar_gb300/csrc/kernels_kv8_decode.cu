// Decode attention over the 8-bit cache: every complete page of a request, or a selected list of them
// per kv head, and the BF16 tail rows of the page that is not complete.
//
// o = softmax(q K^T / sqrt d) V is split along the tokens: CTA (split, kv head, request) reads its pages
// once for all query heads of the kv head and leaves (m, l, acc) with weights 2^(s - m); a second kernel
// merges the partials.  What it must read is 2 d bytes per token and kv head, so it is bound by memory;
// 4 d flops per token and query head run on the tensor cores.
//
// A CTA has one producer warp and four consumer warps around a ring of stages of 64 tokens (64 / P pages,
// each one bulk copy of codes and scales).  Consumer warp w takes tokens 16 w .. 16 w + 15 of a stage:
//   scores: A = 16 tokens x 16 channels of codes, B = the query as f16 (a power of two brings its largest
//           component to 2^14; BF16 queries are exact in one f16, float32 ones take a high and a low half);
//           channels are taken in the order in which a lane's 16-byte loads hold them.
//   values: A = 16 channels x 16 tokens of codes, B = the weights as f16 high and low halves (24 bits
//           relative to the block's largest).
// Codes are exact f16 numbers, so the only roundings are float32's.  The block's scales multiply scores
// and sums in float32, and the weights are relative to the 16-token block's own maximum, so a quiet page
// next to a loud one keeps its digits.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kConsumers = 4;
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kStages = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Layout {
  static constexpr int kPad = 128;  // scales, and the 128-byte alignment of the next page
  OSCAR_HD static int page_stride(int P) { return 2 * P * D + kPad; }
  OSCAR_HD static int stage_bytes(int P) { return (kKv8StageTokens / P) * page_stride(P); }
  static constexpr int kTailRow = 2 * D + 16;  // bytes of a staged tail row of K (padded: no bank conflicts)
  // tail CTA: K rows | V rows | q [8][D] | weights [64][8] | (m, l) [8]
  static constexpr int kTailBytes = 64 * kTailRow + 64 * 2 * D + 8 * D * 4 + 64 * 8 * 4 + 64;
  static size_t smem(int P) {
    const size_t ring = (size_t)kStages * stage_bytes(P);
    const size_t merge = kConsumers * 8 * (D + 2) * sizeof(float);
    size_t n = ring > kTailBytes ? ring : (size_t)kTailBytes;
    if (merge > n) n = merge;
    return n + 128;
  }
};

__device__ __forceinline__ bool length_ok(const Kv8DecodeArgs& a, int n) {
  return n >= 0 && n <= (a.page_idx ? (long long)a.g.max_pages_per_req * a.g.P : (long long)a.max_seq);
}

__device__ __forceinline__ float* partial(const Kv8DecodeArgs& a, int b, int head, int split, int D) {
  return a.part + (((size_t)b * a.g.Hq + head) * (1 + a.wl.max_splits) + split) * (D + 4);
}

// ------------------------------------------------------------------ tail rows
// At most 63 BF16 rows, in float32 on the CUDA cores: a thread per (token, head) for the scores, a thread
// per two channels and every (256 / D)-th head for the sums.
template <int D>
__device__ void tail_rows(const Kv8DecodeArgs& a, int b, int h, int cnt, uint8_t* smem) {
  using L = Layout<D>;
  const Geom& g = a.g;
  const int G = g.gq(), tid = threadIdx.x;
  uint8_t* ks = smem;
  uint8_t* vs = ks + 64 * L::kTailRow;
  float* qs = reinterpret_cast<float*>(vs + 64 * 2 * D);
  float* ps = qs + 8 * D;
  float* ml = ps + 64 * 8;
  const uint16_t* rows = a.tail + ((size_t)a.layer * g.max_req + a.req_slot[b]) * kv8_tail_req_elems(g) + (size_t)h * 2 * g.P * D;
  constexpr int kVec = D / 8;
  for (int i = tid; i < cnt * kVec; i += kThreads) {
    const int t = i / kVec, c = i % kVec;
    *reinterpret_cast<uint4*>(ks + t * L::kTailRow + c * 16) = reinterpret_cast<const uint4*>(rows)[t * kVec + c];
    reinterpret_cast<uint4*>(vs)[i] = reinterpret_cast<const uint4*>(rows + (size_t)g.P * D)[i];
  }
  for (int i = tid; i < G * D; i += kThreads)
    qs[i] = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)h * G * D + i, a.q_dtype);
  __syncthreads();
  const float scale = kLog2e * rsqrtf((float)D);
  for (int i = tid; i < 64 * G; i += kThreads) {
    const int t = i & 63, hh = i >> 6;
    if (t >= cnt) continue;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
    for (int c = 0; c < kVec; ++c) {
      const uint4 k = *reinterpret_cast<const uint4*>(ks + t * L::kTailRow + c * 16);
      const float4 x = reinterpret_cast<const float4*>(qs + hh * D)[2 * c], y = reinterpret_cast<const float4*>(qs + hh * D)[2 * c + 1];
      s0 = fmaf(x.x, bf16_lo(k.x), s0);
      s1 = fmaf(x.y, bf16_hi(k.x), s1);
      s0 = fmaf(x.z, bf16_lo(k.y), s0);
      s1 = fmaf(x.w, bf16_hi(k.y), s1);
      s0 = fmaf(y.x, bf16_lo(k.z), s0);
      s1 = fmaf(y.y, bf16_hi(k.z), s1);
      s0 = fmaf(y.z, bf16_lo(k.w), s0);
      s1 = fmaf(y.w, bf16_hi(k.w), s1);
    }
    ps[t * 8 + hh] = (s0 + s1) * scale;
  }
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  for (int hh = warp; hh < G; hh += kThreads / 32) {
    const float x = lane < cnt ? ps[lane * 8 + hh] : -INFINITY, y = lane + 32 < cnt ? ps[(lane + 32) * 8 + hh] : -INFINITY;
    float m = fmaxf(x, y);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = warp_max_xor(m, o);
    const float px = lane < cnt ? ex2(x - m) : 0.f, py = lane + 32 < cnt ? ex2(y - m) : 0.f;
    float l = px + py;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane < cnt) ps[lane * 8 + hh] = px;
    if (lane + 32 < cnt) ps[(lane + 32) * 8 + hh] = py;
    if (lane == 0) {
      ml[2 * hh] = m;
      ml[2 * hh + 1] = l;
    }
  }
  __syncthreads();
  constexpr int kGroups = 256 / D;      // 128 threads cover D / 2 channel pairs this many times
  constexpr int kHeads = 8 / kGroups;
  if (tid >= 128) return;
  const int cp = tid % (D / 2), g0 = tid / (D / 2);
  float2 acc[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int t = 0; t < cnt; ++t) {
    const uint32_t v = reinterpret_cast<const uint32_t*>(vs)[t * (D / 2) + cp];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int hh = g0 + i * kGroups;
      if (hh < G) {
        const float p = ps[t * 8 + hh];
        acc[i].x = fmaf(p, bf16_lo(v), acc[i].x);
        acc[i].y = fmaf(p, bf16_hi(v), acc[i].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int hh = g0 + i * kGroups;
    if (hh < G) {
      float* pp = partial(a, b, h * G + hh, 0, D);
      *reinterpret_cast<float2*>(pp + 4 + 2 * cp) = acc[i];
      if (cp == 0) {
        pp[0] = ml[2 * hh];
        pp[1] = ml[2 * hh + 1];
      }
    }
  }
}

// ------------------------------------------------------------------ pages
// G8: eight query heads per kv head (an MMA column is a head, low halves go through a second MMA); otherwise
// up to four (columns 2 h and 2 h + 1 are the high and the low half of head h).
template <int D, int FMT, bool G8, bool QF32>
__global__ void __launch_bounds__(kThreads, 3) kv8_decode_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  using L = Layout<D>;
  constexpr int KS = D / 16;               // k-steps of a score, and channel tiles of a sum
  constexpr int NH = G8 ? 2 : 1;           // heads whose weights a lane holds
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ uint32_t mapped[kStages];     // bit i: page i of the stage is there
  __shared__ int abort_flag, issued;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const Geom& g = a.g;
  const int b = blockIdx.z, h = blockIdx.y, split = (int)blockIdx.x - 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = g.gq(), P = g.P;
  const int per_stage = kKv8StageTokens / P;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b];
  if (!length_ok(a, n)) {
    if (tid == 0 && split < 0) flag_error(a.status, kDevBadLen);
    return;
  }
  const int pages = n / P;
  if (split < 0) {
    if (n % P == 0) return;
    const int slot = a.req_slot[b];
    if (slot < 0 || slot >= g.max_req) {
      if (tid == 0) flag_error(a.status, kDevBadSlot);
      return;
    }
    tail_rows<D>(a, b, h, n % P, smem);
    return;
  }
  const int have = a.page_idx ? a.n_select : pages;
  const int e0 = split * a.wl.stages_per_split * per_stage;
  if (e0 >= have) return;
  const int e1 = min(e0 + a.wl.stages_per_split * per_stage, have);
  const int stages = (e1 - e0 + per_stage - 1) / per_stage;
  const int page_stride = L::page_stride(P), stage_bytes = L::stage_bytes(P);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumers);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const float sm_log2 = kLog2e * rsqrtf((float)D);
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

  if (warp == kConsumers) {
    // ---------------------------------------------------------------- producer
    const Kv8Geom kg{P, D, g.Hkv};
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t bytes = 2 * P * D + 16;
    const uint8_t* layer = a.pool + (size_t)a.layer * g.num_pages * kg.page_bytes() + (size_t)h * kg.block_bytes();
    const int* bt = a.block_table + (size_t)b * a.bt_stride;
    const int* list = a.page_idx ? a.page_idx + ((size_t)b * g.Hkv + h) * a.n_select : nullptr;
    // lane i looks up entry e0 + base + i; -1: nothing to copy
    auto lookup = [&](int e) {
      if (e >= e1) return -1;
      int lp = e;
      if (list) {
        lp = list[e];
        const int before = e > 0 ? list[e - 1] : -1;
        if (lp < 0) return -1;
        if (lp >= pages || (e > 0 && before < 0) || before >= lp) {
          flag_error(a.status, kDevBadPage);
          return -1;
        }
      }
      const int pid = lp < a.bt_stride ? bt[lp] : -1;
      if (pid < 0 || pid >= g.num_pages) {
        flag_error(a.status, kDevBadPage);
        return -1;
      }
      return pid;
    };
    int pid_now = lookup(e0 + lane), pid_next = lookup(e0 + 32 + lane);
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
        pid_next = lookup(e0 + at + 32 + lane);
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
          float4 v;
          if constexpr (QF32) {
            v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + i);
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + i);
            v = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
          }
          float* y = x[4 * c + w];
          y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
#pragma unroll
          for (int k = 0; k < 4; ++k) big = fmaxf(big, fabsf(y[k]));
        }
      big = warp_max_xor(big, 1);
      big = warp_max_xor(big, 2);
      const int k = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - k) << 23), down = __uint_as_float((uint32_t)(127 - 14 + k) << 23);
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
        qs[i] = __shfl_sync(0xffffffffu, down, (G8 ? 2 * tig + i : 2 * tig) * 4) * sm_log2;
    }
    const int pi = warp * 16 / P;                       // page of the stage, and the block's first token in it
    const int t0 = warp * 16 % P;
    // byte offsets inside a page: K row gid (+ 8), chunk tig (+ 4); V rows 2 tig (+ 1, + 8, + 9), chunk of channels gid D / 8
    const uint32_t k_off = D == 128 ? (t0 + gid) * 128 + ((tig ^ (4 * (gid & 1))) << 4) : (t0 + gid) * 64 + tig * 16;
    const uint32_t v_off = P * D + (D == 128 ? (t0 + 2 * tig) * 128 + ((gid ^ (2 * tig)) << 4)
                                             : (t0 / 2 + tig) * 128 + (((gid >> 1) ^ (2 * tig)) << 4) + (gid & 1) * 8);
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
        uint32_t kw[2][KS];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < KS / 4; ++c) {
            const uint32_t at = D == 128 ? (k_off ^ (64 * c)) + r * 8 * D : k_off + r * 8 * D;
            const uint4 v = *reinterpret_cast<const uint4*>(page + at);
            kw[r][4 * c] = v.x, kw[r][4 * c + 1] = v.y, kw[r][4 * c + 2] = v.z, kw[r][4 * c + 3] = v.w;
          }
        float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
          const uint32_t a0 = kv8_pair<FMT, 0>(kw[0][kk]), a1 = kv8_pair<FMT, 0>(kw[1][kk]);
          const uint32_t a2 = kv8_pair<FMT, 1>(kw[0][kk]), a3 = kv8_pair<FMT, 1>(kw[1][kk]);
          mma_f16(sc, a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
          if constexpr (G8 && QF32) mma_f16(sc, a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
        }
        // weights relative to the block's maximum
        float w_acc[NH], alpha[NH];
        uint32_t pb[G8 ? 4 : 2];
        float pr[NH][2];
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          const float f = sc2.x * qs[i];
          const float sa = (G8 ? sc[i] : sc[0] + sc[1]) * f, sb = (G8 ? sc[2 + i] : sc[2] + sc[3]) * f;
          float m = fmaxf(sa, sb);
          m = warp_max_xor(m, 4);
          m = warp_max_xor(m, 8);
          m = warp_max_xor(m, 16);
          const float m_new = fmaxf(m_run[i], m);
          alpha[i] = ex2(m_run[i] - m_new);
          const float beta = ex2(m - m_new);
          pr[i][0] = ex2(sa - m);
          pr[i][1] = ex2(sb - m);
          l_run[i] = fmaf(l_run[i], alpha[i], beta * (pr[i][0] + pr[i][1]));
          m_run[i] = m_new;
          w_acc[i] = beta * sc2.y;
        }
        if constexpr (G8) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t hi = pack_half2(pr[0][r], pr[1][r]);
            const __half2 hh = *reinterpret_cast<const __half2*>(&hi);
            pb[r] = transpose_8x8(hi);
            pb[2 + r] = transpose_8x8(pack_half2(pr[0][r] - __low2float(hh), pr[1][r] - __high2float(hh)));
          }
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float hi = __half2float(__float2half_rn(pr[0][r]));
            pb[r] = transpose_8x8(pack_half2(hi, pr[0][r] - hi));
          }
        }
        // sums
        uint32_t vw[4][KS / 2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(page + v_off + ((j & 1) + 8 * (j >> 1)) * 128);
            vw[j][0] = v.x, vw[j][1] = v.y, vw[j][2] = v.z, vw[j][3] = v.w;
          } else {
            // row 2 tig + 1 is the other half of the 128-byte line: four chunks on
            const uint2 v = *reinterpret_cast<const uint2*>(page + ((v_off - P * D) ^ (64 * (j & 1))) + P * D + (j >> 1) * 512);
            vw[j][0] = v.x, vw[j][1] = v.y;
          }
        }
#pragma unroll
        for (int w = 0; w < KS / 2; ++w)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x01 = prmt(vw[0][w], vw[1][w], u ? 0x7362u : 0x5140u);
            const uint32_t x23 = prmt(vw[2][w], vw[3][w], u ? 0x7362u : 0x5140u);
            const uint32_t a0 = kv8_pair<FMT, 0>(x01), a1 = kv8_pair<FMT, 1>(x01);
            const uint32_t a2 = kv8_pair<FMT, 0>(x23), a3 = kv8_pair<FMT, 1>(x23);
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(o, a0, a1, a2, a3, pb[0], pb[1]);
            if constexpr (G8) mma_f16(o, a0, a1, a2, a3, pb[2], pb[3]);
            const int mt = 2 * w + u;
            if constexpr (G8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[mt][i] = fmaf(acc[mt][i], alpha[i & 1], o[i] * w_acc[i & 1]);
            } else {
              acc[mt][0] = fmaf(acc[mt][0], alpha[0], (o[0] + o[1]) * w_acc[0]);
              acc[mt][1] = fmaf(acc[mt][1], alpha[0], (o[2] + o[3]) * w_acc[0]);
            }
          }
      }
      __syncwarp();
      if (lane == 0) {
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[s])) : "memory");
      }
    }
  }
  __syncthreads();
  if (abort_flag) {  // a wait ran out: let the copies in flight land before the CTA ends
    if (tid == 0)
      for (int k = max(issued - kStages, 0); k < issued; ++k)
        (void)mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, nullptr);
    __syncthreads();
    return;
  }
  // merge the four warps' partials: [warp][head][D + 2] in the ring's memory
  float* mg = reinterpret_cast<float*>(smem);
  if (warp < kConsumers) {
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
    float* pp = partial(a, b, h * G + hh, 1 + split, D);
    pp[4 + ch] = o;
    if (ch == 0) {
      pp[0] = M;
      pp[1] = l;
    }
  }
}

// ------------------------------------------------------------------ merge of the splits
// One CTA per (query head, request): warp w takes every fourth split, a lane D / 32 channels.
template <int D>
__global__ void __launch_bounds__(128) kv8_combine_kernel(const __grid_constant__ Kv8DecodeArgs a) {
  constexpr int C = D / 32;
  __shared__ float s_o[4][D], s_l[4];
  const Geom& g = a.g;
  const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.seq_lens[b], slot = a.req_slot[b];
  const bool ok = length_ok(a, n);
  const int have = !ok ? 0 : a.page_idx ? a.n_select : n / g.P;
  const int per_split = a.wl.stages_per_split * (kKv8StageTokens / g.P);
  const int last = 1 + (have + per_split - 1) / per_split;
  const int first = ok && n % g.P && slot >= 0 && slot < g.max_req ? 0 : 1;
  const float* base = partial(a, b, head, 0, D);
  float M = -INFINITY;
  for (int i = first + lane; i < last; i += 32) M = fmaxf(M, base[(size_t)i * (D + 4)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = warp_max_xor(M, o);
  float l = 0.f, r[C];
#pragma unroll
  for (int c = 0; c < C; ++c) r[c] = 0.f;
#pragma unroll 4
  for (int i = first + warp; i < last; i += 4) {
    const float* p = base + (size_t)i * (D + 4);
    const float m = p[0];
    const float w = m == -INFINITY ? 0.f : ex2(m - M);
    l = fmaf(w, p[1], l);
    float v[C];
    if constexpr (C == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + 4 + lane * 4);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(p + 4 + lane * 2);
      v[0] = x.x, v[1] = x.y;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = fmaf(w, v[c], r[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_o[warp][lane * C + c] = r[c];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (tid >= D) return;
  const float sum = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
  const float o = (s_o[0][tid] + s_o[1][tid]) + (s_o[2][tid] + s_o[3][tid]);
  const float y = sum > 0.f ? o / sum : 0.f;
  const size_t at = ((size_t)b * g.Hq + head) * D + tid;
  if (a.out_dtype == kDtypeBF16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  else static_cast<float*>(a.out)[at] = y;
}

template <int D, int FMT>
int launch_pages(const Kv8DecodeArgs& a, cudaStream_t s, bool pdl) {
  const dim3 grid(1 + a.wl.max_splits, a.g.Hkv, a.batch);
  const size_t smem = Layout<D>::smem(a.g.P);
  auto go = [&](auto kern) {
    const cudaError_t e = ensure_smem_limit(kern, smem, true);
    if (e != cudaSuccess) return (int)e;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, pdl, a);
  };
  const bool f32 = a.q_dtype == kDtypeF32;
  if (a.g.gq() == 8) return f32 ? go(kv8_decode_kernel<D, FMT, true, true>) : go(kv8_decode_kernel<D, FMT, true, false>);
  return f32 ? go(kv8_decode_kernel<D, FMT, false, true>) : go(kv8_decode_kernel<D, FMT, false, false>);
}

}  // namespace

Kv8DecodeWs kv8_plan(const Geom& g, int batch, long long max_pages) {
  Kv8DecodeWs w{};
  const int per_stage = kKv8StageTokens / g.P;
  const long long stages = (max_pages + per_stage - 1) / per_stage;
  const long long pairs = (long long)batch * g.Hkv > 0 ? (long long)batch * g.Hkv : 1;
  const long long wave = 152LL * 3;        // resident CTAs
  // one wave where CTAs of up to 16 stages fill it, else CTAs of at least 16 stages in up to eight waves
  long long ctas = pairs * stages / 16;
  if (ctas < wave) ctas = wave;
  if (ctas > 8 * wave) ctas = 8 * wave;
  long long splits = ctas / pairs;
  if (splits < 1) splits = 1;
  long long per = stages > 0 ? (stages + splits - 1) / splits : 1;
  w.stages_per_split = (int)per;
  w.max_splits = stages > 0 ? (int)((stages + per - 1) / per) : 0;
  w.total = (size_t)batch * g.Hq * (1 + w.max_splits) * (g.D + 4) * sizeof(float);
  return w;
}

int launch_kv8_decode(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.g.D == 128) return a.fmt == kKv8Int8 ? launch_pages<128, kKv8Int8>(a, s, pdl) : launch_pages<128, kKv8E4m3>(a, s, pdl);
  return a.fmt == kKv8Int8 ? launch_pages<64, kKv8Int8>(a, s, pdl) : launch_pages<64, kKv8E4m3>(a, s, pdl);
}

int launch_kv8_combine(const Kv8DecodeArgs& a, void* stream, bool pdl) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(a.g.Hq, a.batch);
  if (a.g.D == 128) return launch_pdl(kv8_combine_kernel<128>, grid, dim3(128), 0, s, pdl, a);
  return launch_pdl(kv8_combine_kernel<64>, grid, dim3(128), 0, s, pdl, a);
}

}  // namespace oscar
