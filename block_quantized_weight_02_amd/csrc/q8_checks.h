// q8_checks.h -- argument checks of the host sides that came after q8_api.cpp
// (q8_w4_api.cpp, q8_logits_api.cpp): each returns Q8_OK, or the status with the
// message set.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/q8gemv.h"
#include "q8_internal.h"

namespace q8 {

// Workspace bytes of the arrival counters: the products' counter region, so that
// one zeroed workspace serves every call.
constexpr size_t kCounterBytes = (size_t)4 << 20;
constexpr int64_t kMaxInt = 0x7fffffff;

inline int ok() {
  report_error(Q8_OK, "%s", "");
  return Q8_OK;
}

inline int check_ptr(const void *p, const char *name) {
  if (!p) return report_error(Q8_ERR_NULL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return report_error(Q8_ERR_ALIGN, "%s = %p is not 16-byte aligned", name, p);
  return Q8_OK;
}

inline int check_opt(const void *p, const char *name) {
  return p ? check_ptr(p, name) : (int)Q8_OK;
}

inline int check_range(int64_t v, int64_t lo, int64_t hi, const char *name) {
  if (v < lo || v > hi)
    return report_error(Q8_ERR_SHAPE, "%s = %lld out of range: need %lld <= %s <= %lld", name,
                        (long long)v, (long long)lo, name, (long long)hi);
  return Q8_OK;
}

inline int check_workspace(const void *ws, size_t bytes, size_t need) {
  if (need == 0) return Q8_OK;
  if (!ws || bytes < need)
    return report_error(Q8_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed",
                        ws ? bytes : (size_t)0, need);
  return check_ptr(ws, "workspace");
}

inline int done(hipError_t e, const char *what) {
  if (e == hipSuccess) return ok();
  (void)hipGetLastError();   // do not leave the failure for the caller's next HIP call
  return report_error(Q8_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

}  // namespace q8
