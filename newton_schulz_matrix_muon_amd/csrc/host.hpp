// Host-side helpers shared by the library's translation units: the calling thread's last HIP
// error, launch timing with HIP events, and small argument checks.
#pragma once

#include "muon_ns.h"

#include <hip/hip_runtime.h>

#include <mutex>
#include <utility>
#include <vector>

#include "common.hpp"

namespace mns {

// The hipError_t of the calling thread's last HIP failure (mns_last_hip_error).
inline thread_local int g_last_hip = 0;

// ------------------------------------------------------------------ launch timing
enum Kind { K_PREP = 0, K_FINALIZE, K_SYRK, K_SYMPROD, K_RECT, K_CAST, K_SQUARE, K_ADAMW,
            K_LAYER_NORM, K_ROUTE, K_EXPERT_GEMM, NKINDS };
inline const char* const kKindNames[NKINDS] = {"prep_norm", "finalize_norm", "gemm_syrk", "gemm_symprod",
                                        "gemm_rect", "cast", "gemm_square", "adamw",
                                        "layer_norm", "expert_rows", "expert_gemm"};

struct Timing {
  std::mutex mu;
  bool on = false;
  std::vector<std::pair<hipEvent_t, hipEvent_t>> ev[NKINDS];
  std::vector<hipEvent_t> pool;
};
inline Timing& timing() {
  static Timing* t = new Timing();  // never destroyed: events may outlive static teardown
  return *t;
}

inline hipEvent_t take_event(Timing& t) {
  if (!t.pool.empty()) {
    hipEvent_t e = t.pool.back();
    t.pool.pop_back();
    return e;
  }
  hipEvent_t e = nullptr;
  if (hipEventCreate(&e) != hipSuccess) return nullptr;
  return e;
}

// Launch `f` (which enqueues exactly one kernel on `s`), with events around it when
// timing is on. Returns MNS_OK or MNS_ERR_HIP.
template <class F>
int launch(int kind, hipStream_t s, F&& f) {
  Timing& t = timing();
  hipEvent_t e0 = nullptr, e1 = nullptr;
  bool rec = false;
  {
    std::lock_guard<std::mutex> lk(t.mu);
    if (t.on) {
      e0 = take_event(t);
      e1 = take_event(t);
      rec = e0 && e1;
    }
  }
  if (rec) (void)hipEventRecord(e0, s);
  f();
  hipError_t err = hipGetLastError();
  if (rec) {
    (void)hipEventRecord(e1, s);
    std::lock_guard<std::mutex> lk(t.mu);
    t.ev[kind].emplace_back(e0, e1);
  }
  if (err != hipSuccess) {
    g_last_hip = (int)err;
    return MNS_ERR_HIP;
  }
  return MNS_OK;
}

// ------------------------------------------------------------------ validation helpers
inline bool valid_dtype(int dt) { return dt == F32 || dt == BF16 || dt == F16; }

inline int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Compute units of the current device, looked up once per device.
inline int device_cus() {
  static int cached[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (!cached[dev]) {
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    cached[dev] = cus;
  }
  return cached[dev];
}

}  // namespace mns
