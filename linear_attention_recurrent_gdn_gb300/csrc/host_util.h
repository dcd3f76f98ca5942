// Host-side helpers of the mixer and attention operators' C entry points: error text,
// alignment, launch status, the device's multiprocessors (internal).
#pragma once
#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "../../include/deltalog.h"

namespace dl {

struct ErrOut {
  char* buf;
  int32_t len;
  ErrOut(char* b, int32_t n) : buf(b), len(n) {
    if (buf && len > 0) buf[0] = 0;
  }
  dl_status operator()(dl_status s, const char* fmt, ...) const {
    if (buf && len > 0) {
      va_list ap;
      va_start(ap, fmt);
      vsnprintf(buf, (size_t)len, fmt, ap);
      va_end(ap);
    }
    return s;
  }
};

inline int64_t elem(int64_t dtype) { return dtype == DL_F32 ? 4 : 2; }
inline bool al(const void* p, int64_t b) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(b - 1)) == 0; }
inline bool bad_type(int64_t t) { return t < DL_F32 || t > DL_F16; }

// After a launch: CUDA's sticky state is left clean for the caller's next call.
inline dl_status done(const ErrOut& fail, cudaError_t e) {
  if (e == cudaSuccess) return DL_OK;
  (void)cudaGetLastError();
  return fail(DL_ECUDA, "launch failed: %s", cudaGetErrorString(e));
}

// Multiprocessors of the current device (a GB300's where there is none to ask).
inline int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 152;
  }
  n = known[dev].load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return 152;
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace dl
