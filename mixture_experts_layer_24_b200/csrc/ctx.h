// ctx.h -- the context behind moe_ctx_t and what every entry point does with
// it: launch counting, NVTX names and kernel timing (host code only).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <mutex>
#include <string>
#include <unordered_map>
#include <vector>

#include "../../include/moe.h"

// In a file with a fail(status, text) that records the text for moe_last_error.
#define MOE_CUDA(call)                                                                              \
  do {                                                                                              \
    cudaError_t err_ = (call);                                                                      \
    if (err_ != cudaSuccess)                                                                        \
      return fail(MOE_ERR_CUDA, std::string(#call) + ": " + cudaGetErrorString(err_));             \
  } while (0)

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kRouteCounters = 4096;

struct moe_ctx {
  moe_config_t cfg;
  int device = 0;
  int* d_status = nullptr;
  int num_sms = 148;
  bool chain = true;  // programmatic dependent launch between this library's kernels
  unsigned int* d_counters = nullptr;  // [kRouteCounters] arrival counters of the decode router (self-resetting)
  std::mutex counters_mu;
  int counters_taken = 0;
  std::unordered_map<unsigned long long, int> counter_of_stream;
  int host_status = 0;
  EncodeTiledFn encode = nullptr;
  std::atomic<int64_t> launches{0};
  // kernel timing (moe_profile_*)
  bool prof_on = false;
  struct Rec {
    int kind;
    cudaEvent_t a, b;
  };
  std::vector<Rec> prof_pending;
  std::vector<cudaEvent_t> ev_pool;
  double prof_ms[MOE_PROF_KINDS] = {};
  int64_t prof_n[MOE_PROF_KINDS] = {};
  std::mutex prof_mu;

  // The arrival counter of a decode router launch on s, shared with no launch that may run beside it: launches on one
  // stream follow each other and take the stream's; a captured launch keeps one for good, since its graph may be
  // replayed beside anything (but not beside itself). NULL when all are taken.
  unsigned int* route_counter(cudaStream_t s) {
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamIsCapturing(s, &capture) != cudaSuccess ||
        (capture == cudaStreamCaptureStatusNone && cudaStreamGetId(s, &id) != cudaSuccess)) {
      cudaGetLastError();
      return nullptr;
    }
    std::lock_guard<std::mutex> g(counters_mu);
    if (capture == cudaStreamCaptureStatusNone) {
      const auto it = counter_of_stream.find(id);
      if (it != counter_of_stream.end()) return d_counters + it->second;
    }
    if (counters_taken == kRouteCounters) return nullptr;
    if (capture == cudaStreamCaptureStatusNone) counter_of_stream[id] = counters_taken;
    return d_counters + counters_taken++;
  }

  // cuTensorMapEncodeTiled on the current device. It is a driver call and needs that device's context current on this
  // thread; a thread whose first CUDA call this is has none yet (cudaGetDevice binds nothing, cudaSetDevice does).
  template <typename... Args>
  CUresult encode_tiled(Args... args) const {
    CUresult r = encode(args...);
    int current = 0;
    if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&current) == cudaSuccess &&
        cudaSetDevice(current) == cudaSuccess)
      r = encode(args...);
    return r;
  }

  cudaEvent_t take_event() {
    if (!ev_pool.empty()) {
      cudaEvent_t e = ev_pool.back();
      ev_pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    cudaEventCreate(&e);
    return e;
  }
};

namespace {
// Step names of the MOE_PROF_* kinds, for the NVTX ranges below.
static const char* const kStepNames[MOE_PROF_KINDS] = {"moe.router",  "moe.topk", "moe.permute",
                                                       "moe.gather",  "moe.gate_up", "moe.down",
                                                       "moe.quant",   "moe.combine", "moe.ffn_fused",
                                                       "moe.rows",    "moe.swiglu",  "moe.route_bwd",
                                                       "moe.product"};

// Counts one kernel launch, names it with an NVTX range on the host timeline
// (free unless a profiler is attached), and, when timing is on, brackets it
// with events on the launching stream.
struct Prof {
  moe_ctx* c;
  int kind;
  cudaStream_t s;
  cudaEvent_t a = nullptr;
  Prof(moe_ctx* c_, int kind_, cudaStream_t s_) : c(c_), kind(kind_), s(s_) {
    nvtxRangePushA(kStepNames[kind]);
    if (c->prof_on) {
      std::lock_guard<std::mutex> g(c->prof_mu);
      a = c->take_event();
      cudaEventRecord(a, s);
    }
  }
  ~Prof() {
    nvtxRangePop();
    c->launches.fetch_add(1, std::memory_order_relaxed);
    if (a) {
      std::lock_guard<std::mutex> g(c->prof_mu);
      cudaEvent_t b = c->take_event();
      cudaEventRecord(b, s);
      c->prof_pending.push_back({kind, a, b});
    }
  }
};
}  // namespace
