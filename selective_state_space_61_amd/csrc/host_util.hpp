// host_util.hpp -- what the entry points of the C ABI share on the host: the thread's error text,
// argument checks and the launch check.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/ssm.h"

namespace ssm_host {

inline thread_local char g_err[512] = "";

inline ssm_status_t fail(ssm_status_t s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

struct Range {
  const void* p;
  int64_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Arg {
  const void* p;
  int64_t align;
  const char* name;
};

// first non-NULL argument not aligned to its element size, or NULL
inline const Arg* misaligned(const Arg* args, size_t n) {
  for (size_t i = 0; i < n; ++i)
    if (args[i].p && !aligned(args[i].p, static_cast<uintptr_t>(args[i].align))) return &args[i];
  return nullptr;
}

// compute units of the current device, cached per device
inline int device_cus() {
  static int cache[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int cus = __atomic_load_n(&cache[dev], __ATOMIC_RELAXED);
  if (cus == 0) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    __atomic_store_n(&cache[dev], cus, __ATOMIC_RELAXED);
  }
  return cus;
}

inline ssm_status_t check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(SSM_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return SSM_OK;
}

}  // namespace ssm_host
