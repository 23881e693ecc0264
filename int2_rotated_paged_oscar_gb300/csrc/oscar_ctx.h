// The context behind the C ABI and the helpers its translation units share
// (oscar_abi.cpp defines them).
#pragma once
#include <cuda_runtime.h>

#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

#include "../../include/oscar.h"
#include "oscar_internal.h"

struct oscar_timing {
  std::vector<std::pair<cudaEvent_t, cudaEvent_t>> pending;
  double ms = 0.0;
  int launches = 0;
};

struct oscar_ctx {
  oscar::Geom g{};
  uint8_t* pool = nullptr;
  uint16_t* slab = nullptr;
  int* d_status = nullptr;
  int* d_tickets = nullptr;  // one-launch decode counters [max_requests][n_kv_heads], zero between launches
  std::mutex mu;
  std::vector<int32_t> refcount;
  std::vector<int32_t> free_stack;  // top = back
  long long alloc_fail_after = -1;  // fault injection (OSCAR_FAULT_ALLOC_FAIL_AFTER)
  long long allocs_done = 0;
  bool timing = false;
  std::map<std::string, oscar_timing> timers;
  std::vector<cudaEvent_t> event_pool;
  long long launches = 0;
  // per layer: operand exponents of the history's scales and zeros in the
  // decode MMAs (kNoOperandExp until a clip threshold is known for the layer)
  std::vector<int> opexp_K, opexp_V;
  int decode_form = OSCAR_DECODE_AUTO;
  // 8-bit cache (oscar_kv8_bind): null until bound
  uint8_t* kv8_pool = nullptr;
  uint16_t* kv8_tail = nullptr;
  int kv8_format = 0;
  int device = 0;  // the device that was current when the device buffers were handed over
};

namespace oscar {

// Record a message for oscar_last_error and return the code.
oscar_status fail(oscar_status code, const char* fmt, ...);
oscar_status cuda_fail(int err, const char* what);
oscar_status validate(const oscar_config* c, Geom* out);
oscar_status check_layer(const oscar_ctx* ctx, int32_t layer);
oscar_status check_workspace(const void* workspace);
cudaEvent_t take_event(oscar_ctx* ctx);

// Counts a launch and, with timing on, brackets it with events on its stream.
struct LaunchScope {
  oscar_ctx* ctx;
  const char* name;
  cudaStream_t s;
  cudaEvent_t a = nullptr, b = nullptr;
  // Inside stream capture the two records become external event-record nodes
  // of the graph, so one replay of the graph times the kernel on the device.
  unsigned flags = cudaEventRecordDefault;
  LaunchScope(oscar_ctx* c, const char* n, void* stream) : ctx(c), name(n), s(static_cast<cudaStream_t>(stream)) {
    if (ctx->timing) {
      cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
      if (cudaStreamIsCapturing(s, &cs) == cudaSuccess && cs == cudaStreamCaptureStatusActive)
        flags = cudaEventRecordExternal;
      a = take_event(ctx);
      b = take_event(ctx);
      if (a) cudaEventRecordWithFlags(a, s, flags);
    }
  }
  void done(int err) {
    if (err == 0) ctx->launches++;
    if (ctx->timing && a && b) {
      cudaEventRecordWithFlags(b, s, flags);
      ctx->timers[name].pending.push_back({a, b});
    }
  }
};

}  // namespace oscar
