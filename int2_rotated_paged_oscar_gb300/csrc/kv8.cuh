// Device helpers of the 8-bit paged cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv8_internal.h"

namespace oscar {

// Byte of (token t, channel ch) inside a code section.
template <int D, bool IS_V>
__device__ __forceinline__ int kv8_place(int t, int ch) {
  const int c = (t * D + ch) >> 4;
  const int turn = IS_V ? 2 * ((t >> 1) & 3) : (D == 128 ? 4 * (t & 1) : 0);
  return (((c & ~7) | ((c & 7) ^ turn)) << 4) | (ch & 15);
}

// The number a code byte stands for (before the block's scale).
template <int FMT>
__device__ __forceinline__ float kv8_value(uint32_t b) {
  if constexpr (FMT == kKv8Int8) return (float)((int)b - 128);
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
  return __half2float(__half(h));
}

// Two neighbouring code bytes of a word as an f16 pair: bytes 0, 1 (HALF = 0) or 2, 3 (HALF = 1).
// Both are exact.  INT8: the byte under the exponent of 1024 is 1024 + byte; less 1152 that is
// byte - 128.  E4M3: the hardware's conversion.
template <int FMT, int HALF>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t w) {
  if constexpr (FMT == kKv8Int8) {
    const uint32_t x = prmt(w, 0x64646464u, HALF ? 0x4342u : 0x4140u);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    uint32_t r;
    const uint16_t b = (uint16_t)(HALF ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
    return r;
  }
}

// Transpose of an 8 x 8 matrix of 16-bit elements held as an MMA fragment (lane: row lane / 4,
// columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 2^e and its inverse with big 2^e in [2^14, 2^15).
__device__ __forceinline__ void power_of_two(float big, float* up, float* down) {
  const int k = min(max((int)(__float_as_uint(big) >> 23) - 127, -100), 127);
  *up = __uint_as_float((uint32_t)(127 + 14 - k) << 23);
  *down = __uint_as_float((uint32_t)(127 - 14 + k) << 23);
}

// Four neighbouring query components.
template <bool QF32>
__device__ __forceinline__ float4 kv8_load4(const void* q, size_t i) {
  if constexpr (QF32) return *reinterpret_cast<const float4*>(static_cast<const float*>(q) + i);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + i);
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}

__device__ __forceinline__ float kv8_load(const void* p, size_t i, int dtype) {
  if (dtype == kDtypeBF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

// ------------------------------------------------------------------ requests in groups
// Whether length n >= 0 of request b, in a group with `shared` shared pages, is one that the call allows.
__device__ __forceinline__ bool kv8_own_sound(const Kv8DecodeArgs& a, int n, int shared) {
  const long long own = n - (long long)shared * a.g.P;
  return shared >= 0 && shared <= a.groups.max_shared && own >= 0 && own <= a.groups.max_own &&
         n <= (long long)a.g.max_pages_per_req * a.g.P;
}

// Shared pages of the group that holds request b, found by a whole warp: 0 .. max_shared, so that a page index formed from them
// cannot wrap, or -1 where no group holds it or the group's word is another one.
__device__ __forceinline__ int kv8_shared_of(const Kv8DecodeArgs& a, int b) {
  int c = 0;
  for (int i = threadIdx.x & 31; i < a.groups.n; i += 32) c += a.groups.starts[i] <= b;
  const int at = __reduce_add_sync(0xffffffffu, c) - 1;
  if (at < 0) return -1;
  const int lo = a.groups.starts[at], hi = a.groups.starts[at + 1], s = a.groups.shared[at];
  return lo >= 0 && lo <= b && b < hi && hi <= a.batch && s >= 0 && s <= a.groups.max_shared ? s : -1;
}

// Prefix partials of a row whose group shares s pages.
__device__ __forceinline__ int kv8_prefix_splits(const Kv8DecodeArgs& a, int s) {
  const int per = a.groups.units_per_split * (kPrefixUnit / a.g.P);
  return (s + per - 1) / per;
}

}  // namespace oscar
