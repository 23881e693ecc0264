// Page management on the device: tail rows of a fork, page moves, block-table rewriting.  All three only move bytes, so
// they are bound by memory: 16-byte accesses, enough of them in flight, every source byte read once.
#include "common.cuh"
#include "kv8_internal.h"

namespace oscar {
namespace {

// One vector of the source's rows and its copies.  Eight forks of a 37-row tail, 36 layers, 8 kv heads of 128 channels
// (49 MB): 10 us, 4.9 TB/s, the launch included.
template <int N>
__global__ void __launch_bounds__(256) fork_tail_kernel(Geom g, uint16_t* tail, int src, const __grid_constant__ IntPairs<N> p,
                                                        int n_rows) {
  const int layer = blockIdx.z, hk = blockIdx.y;  // hk: kv head * 2 + (K|V)
  const int vecs = n_rows * g.D / 8;
  const size_t req = kv8_tail_req_elems(g) / 8, sect = (size_t)hk * g.P * g.D / 8;
  uint4* base = reinterpret_cast<uint4*>(tail) + (size_t)layer * g.max_req * req + sect;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= vecs) return;
  const uint4 x = base[src * req + i];
  for (int k = 0; k < p.n; ++k) base[p.dst[k] * req + i] = x;
}

// Four vectors a thread on their way at once.  62 pages of 36 layers (134 KB each, 299 MB): 94 us, 6.4 TB/s read and
// written, 0.94 of the measured copy bandwidth.
template <int N>
__global__ void __launch_bounds__(256) copy_pages_kernel(uint4* pool, int num_pages, size_t vecs, const __grid_constant__ IntPairs<N> p) {
  const size_t layer = (size_t)blockIdx.z * num_pages;
  const uint4* src = pool + (layer + p.src[blockIdx.y]) * vecs;
  uint4* dst = pool + (layer + p.dst[blockIdx.y]) * vecs;
  const size_t step = (size_t)gridDim.x * blockDim.x;
  size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (; i + 3 * step < vecs; i += 4 * step) {
    const uint4 a = src[i], b = src[i + step], c = src[i + 2 * step], d = src[i + 3 * step];
    dst[i] = a;
    dst[i + step] = b;
    dst[i + 2 * step] = c;
    dst[i + 3 * step] = d;
  }
  for (; i < vecs; i += step) dst[i] = src[i];
}

template <int N>
__global__ void __launch_bounds__(256) remap_table_kernel(int* table, long long entries, const __grid_constant__ IntPairs<N> p) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= entries) return;
  const int id = table[i];
  int lo = 0, hi = p.n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.src[mid] < id) lo = mid + 1;
    else hi = mid;
  }
  if (lo < p.n && p.src[lo] == id) table[i] = p.dst[lo];
}

// f(list) with the shorter of the two arguments that holds n entries.
template <typename F>
int with_pairs(const int* src, const int* dst, int n, F f) {
  auto fill = [&](auto& p) {
    p.n = n;
    for (int i = 0; i < n; ++i) {
      p.src[i] = src ? src[i] : 0;
      p.dst[i] = dst[i];
    }
    f(p);
    return (int)cudaGetLastError();
  };
  if (n <= kFewPairs) {
    IntPairs<kFewPairs> p;
    return fill(p);
  }
  IntPairs<kMostPairs> p;
  return fill(p);
}

}  // namespace

int launch_kv8_fork_tail(const Geom& g, uint16_t* tail, int src, const int* dst, int n, int n_rows, void* stream) {
  const dim3 grid((n_rows * g.D / 8 + 255) / 256, g.Hkv * 2, g.L);
  return with_pairs(nullptr, dst, n, [&](const auto& p) {
    fork_tail_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(g, tail, src, p, n_rows);
  });
}

int launch_copy_pages(uint8_t* pool, int layers, int num_pages, size_t page_bytes, const int* src, const int* dst, int n,
                      void* stream) {
  const size_t vecs = page_bytes / 16;
  const int x = (int)(vecs / 1024 < 1 ? 1 : vecs / 1024 > 64 ? 64 : vecs / 1024);
  return with_pairs(src, dst, n, [&](const auto& p) {
    copy_pages_kernel<<<dim3(x, n, layers), 256, 0, static_cast<cudaStream_t>(stream)>>>(reinterpret_cast<uint4*>(pool), num_pages,
                                                                                         vecs, p);
  });
}

int launch_remap_table(int* table, int rows, int cols, const int* src, const int* dst, int n, void* stream) {
  const long long entries = (long long)rows * cols;
  return with_pairs(src, dst, n, [&](const auto& p) {
    remap_table_kernel<<<(unsigned)((entries + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(table, entries, p);
  });
}

}  // namespace oscar
