// mxq_host.h - argument checks and the optional guards shared by the files of
// the extern "C" boundary.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "mxq.h"
#include "mxq_internal.h"

namespace mxq {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool log_enabled() {
  static const int on = [] {
    const char* v = getenv("MXQ_LOG");
    return (v != nullptr && v[0] != '\0' && v[0] != '0') ? 1 : 0;
  }();
  return on != 0;
}

inline int check_mk(int64_t rows, int64_t K, int64_t ld) {
  if (rows < 0 || K <= 0 || ld < 0) return MXQ_ERR_SHAPE;
  if (K % 32 != 0 || ld < K) return MXQ_ERR_SHAPE;
  if (rows >= kMaxDim || K >= kMaxDim || ld >= kMaxDim) return MXQ_ERR_SHAPE;
  return MXQ_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MXQ_OK : MXQ_ERR_HIP; }

// The guard's status for a scan's result.
inline int guard_status(int scan_error, bool bad, const char* what, int64_t rows, int64_t cols) {
  if (scan_error != 0) return MXQ_ERR_HIP;
  if (!bad) return MXQ_OK;
  if (log_enabled()) fprintf(stderr, "[mxq] non-finite value in %s [%lld x %lld]\n", what, (long long)rows,
                             (long long)cols);
  return MXQ_ERR_NONFINITE;
}

// MXQ_CHECK_FINITE: scan a bf16 [rows][ld] input (or output) for infinities and
// NaNs; MXQ_OK when the guard is off.
inline int finite_guard(const char* what, const void* x, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
  if (!check_finite_enabled()) return MXQ_OK;
  bool bad = false;
  const int err = scan_nonfinite_bf16(x, rows, cols, ld, stream, &bad);
  return guard_status(err, bad, what, rows, cols);
}

// The same of a float32 [rows][ld] operand.
inline int finite_guard_f32(const char* what, const void* x, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream) {
  if (!check_finite_enabled()) return MXQ_OK;
  bool bad = false;
  const int err = scan_nonfinite_f32(x, rows, cols, ld, stream, &bad);
  return guard_status(err, bad, what, rows, cols);
}

// The same of the scales of an MXFP4 output: blocks quantized from an infinity or a NaN.
inline int finite_guard_mx(const char* what, const void* scales, int64_t rows, int64_t cols, hipStream_t stream) {
  if (!check_finite_enabled()) return MXQ_OK;
  bool bad = false;
  const int err = scan_nonfinite_mx(scales, rows, cols, stream, &bad);
  return guard_status(err, bad, what, rows, cols);
}

// a launch's status, then the guard on its bf16 output
inline int output_guard(hipError_t e, const char* what, const void* y, int64_t rows, int64_t cols, hipStream_t stream) {
  if (e != hipSuccess) return MXQ_ERR_HIP;
  return finite_guard(what, y, rows, cols, cols, stream);
}

}  // namespace mxq
