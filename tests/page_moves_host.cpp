// Page moves with launches that fail: kv8_abi.cpp over fakes of its launchers and of the CUDA runtime, all in host memory.
// Prints one line per failed case; the exit status is their number.
#include <cstdio>
#include <cstring>
#include <vector>

#include "../int2_rotated_paged_oscar_gb300/csrc/kv8_internal.h"
#include "../int2_rotated_paged_oscar_gb300/csrc/oscar_ctx.h"

namespace {

int launches = 0, fails_at = -1;   // the launch that returns an error, counted from 0
bool launch_fails() { return launches++ == fails_at; }
bool capturing = false;
int failed = 0;
void expect(bool ok, const char* what, int at) {
  if (!ok) std::printf("launch %d fails: %s\n", at, what), ++failed;
}

}  // namespace

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaMalloc(void**, size_t) { return cudaErrorMemoryAllocation; }
cudaError_t cudaFree(void*) { return cudaSuccess; }
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaEventRecordWithFlags(cudaEvent_t, cudaStream_t, unsigned) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = capturing ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
}

namespace oscar {
oscar_status fail(oscar_status code, const char*, ...) { return code; }
oscar_status cuda_fail(int, const char*) { return OSCAR_ERR_CUDA; }
oscar_status validate(const oscar_config*, Geom*) { return OSCAR_ERR_INVALID; }
oscar_status check_layer(const oscar_ctx*, int32_t) { return OSCAR_OK; }
oscar_status check_workspace(const void*) { return OSCAR_OK; }
cudaEvent_t take_event(oscar_ctx*) { return nullptr; }
Kv8DecodeWs kv8_plan(const Geom&, int, long long) { return {}; }
size_t kv8_select_ws_bytes(const Geom&, int, int) { return 0; }
int launch_kv8_write(const Kv8WriteArgs&, void*, bool) { return 1; }
int launch_kv8_decode(const Kv8DecodeArgs&, void*, bool) { return 1; }
int launch_kv8_combine(const Kv8DecodeArgs&, void*, bool) { return 1; }
int launch_kv8_select(const Kv8SelectArgs&, void*, bool) { return 1; }
int launch_kv8_fork_tail(const Geom&, uint16_t*, int, const int*, int, int, void*) { return launch_fails(); }
int launch_copy_pages(uint8_t* pool, int layers, int num_pages, size_t bytes, const int* src, const int* dst, int n, void*) {
  if (launch_fails()) return 1;
  for (int l = 0; l < layers; ++l)
    for (int i = 0; i < n; ++i)
      std::memcpy(pool + ((size_t)l * num_pages + dst[i]) * bytes, pool + ((size_t)l * num_pages + src[i]) * bytes, bytes);
  return 0;
}
int launch_remap_table(int* table, int rows, int cols, const int* src, const int* dst, int n, void*) {
  if (launch_fails()) return 1;
  for (int i = 1; i < n; ++i) expect(src[i - 1] < src[i], "the list is not ascending", fails_at);
  for (int e = 0; e < rows * cols; ++e)
    for (int lo = 0, hi = n; lo < hi;) {
      const int mid = (lo + hi) / 2;
      if (src[mid] == table[e]) {
        table[e] = dst[mid];
        break;
      }
      if (src[mid] < table[e]) lo = mid + 1;
      else hi = mid;
    }
  return 0;
}
}  // namespace oscar

int main() {
  constexpr int kPages = 5000, kLive = 2300;
  oscar_ctx ctx;
  ctx.g.L = 2, ctx.g.Hq = ctx.g.Hkv = 1, ctx.g.D = 64, ctx.g.P = 16, ctx.g.max_req = 4;
  ctx.g.max_pages_per_req = kPages, ctx.g.num_pages = kPages;
  const size_t bytes = oscar::kv8_geom(ctx.g).page_bytes();
  std::vector<uint8_t> pool(2 * kPages * bytes);
  std::vector<uint16_t> tail(1);
  ctx.kv8_pool = pool.data();
  ctx.kv8_tail = tail.data();
  // the live pages: every second one of the upper 4600, 1350 of them at ids from 2300 on, which move; each holds its own id
  ctx.refcount.assign(kPages, 0);
  std::vector<int> table;
  for (int i = 0; i < kPages; ++i) {
    if (i >= kPages - 2 * kLive && i % 2) {
      ctx.refcount[i] = 1 + i % 3;
      table.push_back(i);
      for (int l = 0; l < 2; ++l) std::memcpy(&pool[((size_t)l * kPages + i) * bytes], &i, sizeof i);
    } else {
      ctx.free_stack.push_back(i);
    }
  }
  table.push_back(-1);
  const std::vector<int> table0 = table, refs0 = ctx.refcount, free0 = ctx.free_stack;
  std::vector<int32_t> map(kPages, -7);
  int32_t live = -7;
  auto compact = [&] {
    launches = 0;
    return oscar_compact_pages(&ctx, table.data(), 1, (int)table.size(), map.data(), &live, nullptr);
  };
  auto holds = [&](const std::vector<int>& t) {   // every entry's page holds what the first table's page held
    for (size_t e = 0; e + 1 < t.size(); ++e)
      for (int l = 0; l < 2; ++l)
        if (std::memcmp(&pool[((size_t)l * kPages + t[e]) * bytes], &table0[e], sizeof(int))) return false;
    return t.back() == -1;
  };
  constexpr int kLists = 2;   // of at most 1000 pages each, copied and rewritten
  for (fails_at = 0; fails_at < 2 * kLists; ++fails_at) {
    expect(compact() == OSCAR_ERR_CUDA, "no error", fails_at);
    expect(table == table0, "the table has changed", fails_at);
    expect(ctx.refcount == refs0 && ctx.free_stack == free0, "the allocator has changed", fails_at);
    expect(holds(table), "a page is lost", fails_at);
  }
  fails_at = -1;
  // a stream that is being captured: refused, before anything changes
  const int32_t dst[2] = {1, 3};
  std::vector<int32_t> rows(2 * kPages);
  capturing = true;
  expect(compact() == OSCAR_ERR_INVALID && launches == 0 && table == table0, "a captured compaction", -1);
  for (int n : {2 * 16, 2 * 16 + 5})
    expect(oscar_kv8_fork(&ctx, table.data(), n, 0, dst, 2, rows.data(), nullptr) == OSCAR_ERR_INVALID && launches == 0, "a captured fork", -1);
  expect(ctx.refcount == refs0 && ctx.free_stack == free0, "the allocator after captures", -1);
  capturing = false;
  expect(compact() == OSCAR_OK && live == kLive && launches == 2 * kLists, "the call after the failures", -1);
  bool right = (int)ctx.free_stack.size() == kPages - kLive;
  for (size_t e = 0; e + 1 < table0.size(); ++e)
    right = right && table[e] == map[table0[e]] && table[e] < kLive && ctx.refcount[table[e]] == refs0[table0[e]];
  expect(right && holds(table), "the table after the call", -1);
  // a fork whose copy fails leaves the refcounts as they were
  const std::vector<int> refs = ctx.refcount;
  launches = fails_at = 0;
  expect(oscar_kv8_fork(&ctx, table.data(), 16 * 20 + 5, 0, dst, 2, rows.data(), nullptr) == OSCAR_ERR_CUDA, "no error of the fork", 0);
  expect(ctx.refcount == refs, "the fork's refcounts", 0);
  return failed;
}
