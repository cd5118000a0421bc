// Host helpers shared by the files behind the C ABI: buffer carving, the device
// check and the launch tracer.
#pragma once
#include <hip/hip_runtime.h>
#include <string.h>

#include <mutex>
#include <vector>

#include "../../include/mok.h"

namespace mok {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// gfx950 check and compute-unit count, once per device (device properties
// only; no device memory is touched).
inline int g_cus[64] = {0};
inline int g_wclk_khz[64] = {0};   // rate of the device's 64-bit real-time counter

inline mok_status check_device(int* cus = nullptr, int* wclk_khz = nullptr) {
  static std::mutex mu;
  static int state[64] = {0};   // 0 unknown, 1 ok, 2 bad
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MOK_ERR_DEVICE;
  std::lock_guard<std::mutex> g(mu);
  if (state[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOK_ERR_DEVICE;
    state[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_cus[dev] = prop.multiProcessorCount;
    int khz = 0;
    if (hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev) != hipSuccess || khz <= 0)
      khz = 100000;
    g_wclk_khz[dev] = khz;
  }
  if (cus) *cus = g_cus[dev];
  if (wclk_khz) *wclk_khz = g_wclk_khz[dev];
  return state[dev] == 1 ? MOK_OK : MOK_ERR_DEVICE;
}

inline mok_status launched(hipError_t e) { return e == hipSuccess ? MOK_OK : MOK_ERR_DEVICE; }

// Launch tracing: when on, each launch is bracketed by two events recorded on
// its stream; within one API call, consecutive launches on one stream share
// the event between them (the end of one is the start of the next), since
// nothing else is enqueued there in between. Events come from a pool that is
// reused across collections.
struct Tracer {
  std::mutex mu;
  bool on = false;
  struct Rec {
    const char* name;
    hipEvent_t a, b;
    bool shared_a;         // a is the previous record's b
  };
  std::vector<Rec> recs;
  std::vector<hipEvent_t> pool;
  hipEvent_t chain = nullptr;   // end event of the last launch of the current API call
  hipStream_t chain_st = nullptr;
  hipEvent_t get() {
    hipEvent_t e = nullptr;
    if (!pool.empty()) {
      e = pool.back();
      pool.pop_back();
    } else if (hipEventCreateWithFlags(&e, hipEventDisableSystemFence) != hipSuccess) {
      // timing-only events: no system-scope cache writeback and invalidation
      // between the traced kernels (mok_trace_collect synchronises the device)
      e = nullptr;
    }
    return e;
  }
};
inline Tracer g_tr;

// One per API call that launches work: no event chain crosses its boundary
// (the caller may enqueue its own work between calls).
struct TraceCall {
  TraceCall() { reset(); }
  ~TraceCall() { reset(); }
  static void reset() {
    if (!g_tr.on && !g_tr.chain) return;
    std::lock_guard<std::mutex> g(g_tr.mu);
    g_tr.chain = nullptr;
    g_tr.chain_st = nullptr;
  }
};

struct TraceScope {
  const char* name;
  hipStream_t st;
  hipEvent_t a = nullptr;
  bool shared = false;
  TraceScope(const char* n, hipStream_t s) : name(n), st(s) {
    if (!g_tr.on) return;
    std::lock_guard<std::mutex> g(g_tr.mu);
    if (g_tr.chain && g_tr.chain_st == st) {
      a = g_tr.chain;
      shared = true;
    } else {
      a = g_tr.get();
      if (a) (void)hipEventRecord(a, st);
    }
  }
  ~TraceScope() {
    if (!a) return;
    std::lock_guard<std::mutex> g(g_tr.mu);
    hipEvent_t b = g_tr.get();
    if (!b) {
      if (!shared) g_tr.pool.push_back(a);
      g_tr.chain = nullptr;
      return;
    }
    (void)hipEventRecord(b, st);
    g_tr.recs.push_back({name, a, b, shared});
    g_tr.chain = b;
    g_tr.chain_st = st;
  }
};

#define MOK_TRY(expr)                               \
  do {                                              \
    const mok_status _s = launched(expr);           \
    if (_s != MOK_OK) return _s;                    \
  } while (0)

// Launch `expr` (which enqueues one kernel on `st`) under the tracer.
#define MOK_RUN(name, expr)                         \
  do {                                              \
    TraceScope _ts(name, st);                       \
    MOK_TRY(expr);                                  \
  } while (0)

}  // namespace mok
