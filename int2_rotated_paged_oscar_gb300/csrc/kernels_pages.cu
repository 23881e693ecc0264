// Page management on the device: tail rows of a fork, page moves, block-table rewriting.
#include "common.cuh"
#include "kv8_internal.h"

namespace oscar {
namespace {

__global__ void __launch_bounds__(256) fork_tail_kernel(Geom g, uint16_t* tail, int src, const __grid_constant__ ForkSlots dst,
                                                        int n_rows) {
  const int layer = blockIdx.z, hk = blockIdx.y;  // hk: kv head * 2 + (K|V)
  const int vecs = n_rows * g.D / 8;
  const size_t req = kv8_tail_req_elems(g) / 8, sect = (size_t)hk * g.P * g.D / 8;
  uint4* base = reinterpret_cast<uint4*>(tail) + (size_t)layer * g.max_req * req + sect;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < vecs; i += gridDim.x * blockDim.x) {
    const uint4 x = base[src * req + i];
    for (int k = 0; k < dst.n; ++k) base[dst.dst[k] * req + i] = x;
  }
}

__global__ void __launch_bounds__(256) copy_pages_kernel(uint4* pool, int num_pages, size_t vecs, const __grid_constant__ PagePairs p) {
  const size_t layer = (size_t)blockIdx.z * num_pages;
  const uint4* src = pool + (layer + p.src[blockIdx.y]) * vecs;
  uint4* dst = pool + (layer + p.dst[blockIdx.y]) * vecs;
  for (size_t i = blockIdx.x * blockDim.x + threadIdx.x; i < vecs; i += (size_t)gridDim.x * blockDim.x) dst[i] = src[i];
}

__global__ void __launch_bounds__(256) remap_table_kernel(int* table, int rows, int cols, int stride, const __grid_constant__ PagePairs p) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long long)rows * cols) return;
  int* e = table + (i / cols) * stride + i % cols;
  const int id = *e;
  int lo = 0, hi = p.n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (p.src[mid] < id) lo = mid + 1;
    else hi = mid;
  }
  if (lo < p.n && p.src[lo] == id) *e = p.dst[lo];
}

}  // namespace

int launch_kv8_fork_tail(const Geom& g, uint16_t* tail, int src, const ForkSlots& dst, int n_rows, void* stream) {
  const int vecs = n_rows * g.D / 8;
  fork_tail_kernel<<<dim3((vecs + 255) / 256, g.Hkv * 2, g.L), 256, 0, static_cast<cudaStream_t>(stream)>>>(g, tail, src, dst, n_rows);
  return (int)cudaGetLastError();
}

int launch_copy_pages(uint8_t* pool, int layers, int num_pages, size_t page_bytes, const PagePairs& p, void* stream) {
  const size_t vecs = page_bytes / 16;
  const int x = (int)(vecs / 1024 < 1 ? 1 : vecs / 1024 > 64 ? 64 : vecs / 1024);
  copy_pages_kernel<<<dim3(x, p.n, layers), 256, 0, static_cast<cudaStream_t>(stream)>>>(reinterpret_cast<uint4*>(pool), num_pages,
                                                                                         vecs, p);
  return (int)cudaGetLastError();
}

int launch_remap_table(int* table, int rows, int cols, int stride, const PagePairs& p, void* stream) {
  const long long n = (long long)rows * cols;
  remap_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream)>>>(table, rows, cols, stride, p);
  return (int)cudaGetLastError();
}

}  // namespace oscar
