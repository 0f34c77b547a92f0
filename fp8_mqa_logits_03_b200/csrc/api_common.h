// api_common.h -- what the files of the C ABI share: error reporting, argument
// helpers and the process-wide settings.  Host code only.
#pragma once
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/fp8idx.h"

namespace fp8idx {

inline thread_local std::string t_last_error;  // message of the last non-OK return on this thread
inline unsigned long long g_wait_limit_ns = 2000000000ull;
inline int g_debug_withhold = 0;

inline int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return code;
}

inline int ok() {
  t_last_error.clear();
  return FP8IDX_OK;
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(FP8IDX_ECUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

inline int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

#define FP8IDX_TRY(x)          \
  do {                         \
    int _rc = (x);             \
    if (_rc != FP8IDX_OK) return _rc; \
  } while (0)

}  // namespace fp8idx
