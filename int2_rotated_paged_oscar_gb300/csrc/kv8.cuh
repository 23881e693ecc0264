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

// x / m * M rounded to a code.  x M is exact (x and M have 8 and at most 7 significant bits),
// and a quotient of two numbers that short lies no nearer to a code border than float32's
// rounding unless it is on it, so the one rounding of the division loses nothing.
// An infinity saturates and a NaN gives the code of 0.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode(float x, float m) {
  constexpr float M = FMT == kKv8Int8 ? 127.f : 448.f;
  float y = __fdiv_rn(x * M, m);
  if (!(y == y)) y = 0.f;
  if constexpr (FMT == kKv8Int8) {
    return (uint32_t)((int)rintf(fminf(fmaxf(y, -127.f), 127.f)) + 128);
  } else {
    return (uint32_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  }
}

// Code bytes as unsigned keys in the order of their values (-0 counts as +0), and back.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_key(uint32_t b) {
  if constexpr (FMT == kKv8Int8) return b;
  if (b == 0x80u) b = 0;
  return (b & 0x80u) ? (0xFFu & ~b) : (b | 0x80u);
}
template <int FMT>
__device__ __forceinline__ uint32_t kv8_unkey(uint32_t k) {
  if constexpr (FMT == kKv8Int8) return k;
  return (k & 0x80u) ? (k & 0x7Fu) : (0xFFu & ~k);
}

__device__ __forceinline__ float kv8_load(const void* p, size_t i, int dtype) {
  if (dtype == kDtypeBF16) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}

}  // namespace oscar
