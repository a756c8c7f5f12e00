// Host-side checks shared by the C ABI layers (nvfp4_api.hip, int4_api.hip).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool mul_ok(int64_t a, int64_t b) { return a >= 0 && b >= 0 && (a == 0 || b <= INT64_MAX / a); }

// Clear a stale error from earlier unrelated work so that a launch failure
// is attributed to this call.
inline void clear_error() { (void)hipGetLastError(); }

inline int launch_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH; }

// Calls are not graph-capture safe: refuse a stream that is being captured
// (before anything is enqueued on it).
inline int stream_status(hipStream_t s) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(s, &cs) != hipSuccess) return NVFP4_ERR_LAUNCH;
  return cs == hipStreamCaptureStatusNone ? NVFP4_OK : NVFP4_ERR_CAPTURE;
}

}  // namespace nvfp4
