// Decode attention over the 8-bit cache (all complete pages, or a selected list of them) and
// the BF16 tail rows; split along the tokens, partials merged by a second kernel.
#include "kv8.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 16;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) kv8_decode_kernel(Kv8DecodeArgs a) {
  __shared__ float qs[8][D], ks[kTile][D + 1], vs[kTile][D], sc[8][kTile], s_corr[8], s_m[8], s_l[8];
  const Geom& g = a.g;
  const Kv8Geom kg{g.P, D, g.Hkv};
  const int b = blockIdx.z, h = blockIdx.y, split = (int)blockIdx.x - 1, tid = threadIdx.x;
  const int G = g.gq();
  const int n = a.seq_lens[b];
  const long long cap = a.page_idx ? (long long)g.max_pages_per_req * g.P : a.max_seq;
  if (n < 0 || n > cap) {
    if (tid == 0 && split < 0) flag_error(a.status, kDevBadLen);
    return;
  }
  const int pages = n / g.P, tail_n = n % g.P;
  const int have = a.page_idx ? a.n_select : pages;
  const int per_stage = kKv8StageTokens / g.P;
  const int p0 = split < 0 ? 0 : split * a.wl.stages_per_split * per_stage;
  const int p1 = split < 0 ? 0 : min(p0 + a.wl.stages_per_split * per_stage, have);
  if (split < 0 ? tail_n == 0 : p0 >= have) return;
  const int slot = a.req_slot[b];
  if (split < 0 && (slot < 0 || slot >= g.max_req)) {
    if (tid == 0) flag_error(a.status, kDevBadSlot);
    return;
  }
  for (int i = tid; i < G * D; i += kThreads)
    qs[i / D][i % D] = kv8_load(a.q, (size_t)b * a.q_stride + (size_t)h * G * D + i, a.q_dtype);
  if (tid < 8) {
    s_m[tid] = -INFINITY;
    s_l[tid] = 0.f;
  }
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  const int tokens = split < 0 ? tail_n : (p1 - p0) * g.P;
  const float scale = kLog2e * rsqrtf((float)D);
  const uint16_t* tail = a.tail + ((size_t)a.layer * g.max_req + (split < 0 ? slot : 0)) * kv8_tail_req_elems(g) +
                         (size_t)h * 2 * g.P * D;
  for (int t0 = 0; t0 < tokens; t0 += kTile) {
    const int cnt = min(kTile, tokens - t0);
    bool live = true;
    __syncthreads();
    if (split < 0) {
      for (int i = tid; i < cnt * D; i += kThreads) {
        ks[i / D][i % D] = __uint_as_float((uint32_t)tail[(size_t)t0 * D + i] << 16);
        vs[i / D][i % D] = __uint_as_float((uint32_t)tail[(size_t)(g.P + t0) * D + i] << 16);
      }
    } else {
      const int e = p0 + t0 / g.P;
      int lp = e;
      if (a.page_idx) {
        const int* list = a.page_idx + ((size_t)b * g.Hkv + h) * a.n_select;
        lp = list[e];
        if (lp >= pages || (lp >= 0 && e > 0 && list[e - 1] >= lp) || (lp >= 0 && e > 0 && list[e - 1] < 0)) {
          if (tid == 0) flag_error(a.status, kDevBadPage);
          lp = -1;
        }
      }
      int pid = -1;
      if (lp >= 0) {
        pid = lp < a.bt_stride ? a.block_table[(size_t)b * a.bt_stride + lp] : -1;
        if (pid < 0 || pid >= g.num_pages) {
          if (tid == 0) flag_error(a.status, kDevBadPage);
          pid = -1;
        }
      }
      live = pid >= 0;
      if (live) {
        const uint8_t* block = a.pool + ((size_t)a.layer * g.num_pages + pid) * kg.page_bytes() + (size_t)h * kg.block_bytes();
        const float sk = reinterpret_cast<const float*>(block + kg.scale_off())[0];
        const float sv = reinterpret_cast<const float*>(block + kg.scale_off())[1];
        for (int i = tid; i < kTile * D; i += kThreads) {
          const int t = t0 % g.P + i / D, ch = i % D;
          ks[i / D][ch] = kv8_value<FMT>(block[kv8_place<D, false>(t, ch)]) * sk;
          vs[i / D][ch] = kv8_value<FMT>(block[kg.v_off() + kv8_place<D, true>(t, ch)]) * sv;
        }
      }
    }
    if (!live) continue;
    __syncthreads();
    for (int i = tid; i < G * kTile; i += kThreads) {
      const int hh = i / kTile, t = i % kTile;
      float s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(qs[hh][c], ks[t][c], s);
      sc[hh][t] = t < cnt ? s * scale : -INFINITY;
    }
    __syncthreads();
    if (tid < G) {
      float m = s_m[tid];
      for (int t = 0; t < cnt; ++t) m = fmaxf(m, sc[tid][t]);
      const float corr = m == -INFINITY ? 1.f : ex2(s_m[tid] - m);
      float l = s_l[tid] * corr;
      for (int t = 0; t < cnt; ++t) {
        const float p = sc[tid][t] == -INFINITY ? 0.f : ex2(sc[tid][t] - m);
        sc[tid][t] = p;
        l += p;
      }
      s_m[tid] = m;
      s_l[tid] = l;
      s_corr[tid] = corr;
    }
    __syncthreads();
    if (tid < D)
      for (int hh = 0; hh < G; ++hh) {
        float r = acc[hh] * s_corr[hh];
        for (int t = 0; t < cnt; ++t) r = fmaf(sc[hh][t], vs[t][tid], r);
        acc[hh] = r;
      }
  }
  __syncthreads();
  const int stride = 1 + a.wl.max_splits;
  for (int hh = 0; hh < G; ++hh) {
    float* pp = a.part + (((size_t)b * g.Hq + (size_t)h * G + hh) * stride + 1 + split) * (D + 4);
    if (tid < D) pp[4 + tid] = acc[hh];
    if (tid == 0) {
      pp[0] = s_m[hh];
      pp[1] = s_l[hh];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(D) kv8_combine_kernel(Kv8DecodeArgs a) {
  const Geom& g = a.g;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n = a.seq_lens[b];
  const long long cap = a.page_idx ? (long long)g.max_pages_per_req * g.P : a.max_seq;
  const bool ok = n >= 0 && n <= cap;
  const int have = !ok ? 0 : a.page_idx ? a.n_select : n / g.P;
  const int per_split = a.wl.stages_per_split * (kKv8StageTokens / g.P);
  const int last = 1 + (have + per_split - 1) / per_split;
  const int slot = a.req_slot[b];
  const int first = ok && n % g.P && slot >= 0 && slot < g.max_req ? 0 : 1;
  const float* base = a.part + ((size_t)b * g.Hq + h) * (1 + a.wl.max_splits) * (D + 4);
  float M = -INFINITY, L = 0.f, r = 0.f;
  for (int i = first; i < last; ++i) M = fmaxf(M, base[(size_t)i * (D + 4)]);
  for (int i = first; i < last; ++i) {
    const float m = base[(size_t)i * (D + 4)];
    if (m == -INFINITY) continue;
    const float w = ex2(m - M);
    L = fmaf(w, base[(size_t)i * (D + 4) + 1], L);
    r = fmaf(w, base[(size_t)i * (D + 4) + 4 + tid], r);
  }
  const float o = L > 0.f ? r / L : 0.f;
  const size_t at = ((size_t)b * g.Hq + h) * D + tid;
  if (a.out_dtype == kDtypeBF16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(o);
  else static_cast<float*>(a.out)[at] = o;
}

}  // namespace

Kv8DecodeWs kv8_plan(const Geom& g, int batch, long long max_pages) {
  Kv8DecodeWs w{};
  const int per_stage = kKv8StageTokens / g.P;
  const long long stages = (max_pages + per_stage - 1) / per_stage;
  const long long pairs = (long long)batch * g.Hkv > 0 ? (long long)batch * g.Hkv : 1;
  long long splits = 152LL * 4 / pairs;
  if (splits < 1) splits = 1;
  long long per = stages > 0 ? (stages + splits - 1) / splits : 1;
  w.stages_per_split = (int)per;
  w.max_splits = stages > 0 ? (int)((stages + per - 1) / per) : 0;
  w.total = (size_t)batch * g.Hq * (1 + w.max_splits) * (g.D + 4) * sizeof(float);
  return w;
}

int launch_kv8_decode(const Kv8DecodeArgs& a, void* stream, bool) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(1 + a.wl.max_splits, a.g.Hkv, a.batch);
  if (a.g.D == 128) {
    if (a.fmt == kKv8Int8) kv8_decode_kernel<128, kKv8Int8><<<grid, kThreads, 0, s>>>(a);
    else kv8_decode_kernel<128, kKv8E4m3><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (a.fmt == kKv8Int8) kv8_decode_kernel<64, kKv8Int8><<<grid, kThreads, 0, s>>>(a);
    else kv8_decode_kernel<64, kKv8E4m3><<<grid, kThreads, 0, s>>>(a);
  }
  return (int)cudaGetLastError();
}

int launch_kv8_combine(const Kv8DecodeArgs& a, void* stream, bool) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(a.g.Hq, a.batch);
  if (a.g.D == 128) kv8_combine_kernel<128><<<grid, 128, 0, s>>>(a);
  else kv8_combine_kernel<64><<<grid, 64, 0, s>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace oscar
