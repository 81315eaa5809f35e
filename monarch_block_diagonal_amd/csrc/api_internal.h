// Shared by the C-ABI translation units (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "plan.h"

namespace monarch {

// Records a HIP error for monarch_status_string(MONARCH_ERR_HIP) on the
// calling thread; returns MONARCH_OK or MONARCH_ERR_HIP.
int record_hip(hipError_t e);

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Records the caller's events (if any) on the stream, one per mark().
struct Tracer {
  void* const* ev;
  int n;
  int idx = 0;
  hipStream_t s;
  hipError_t mark() {
    hipError_t e = hipSuccess;
    if (ev && idx < n && ev[idx]) e = hipEventRecord(static_cast<hipEvent_t>(ev[idx]), s);
    ++idx;
    return e;
  }
};

// Writes n kernel names separated by ';' into buf (truncated); returns n.
int write_names(const char* const* names, int n, char* buf, size_t buf_len);

// Null and alignment checks of the backward's pointers (not the workspace);
// no HIP call. Returns a monarch_status.
int bwd_check(const Problem& pr, const void* dy, const void* x, const void* w1, const void* w2,
              const void* z, const void* y, const void* dx, const void* dw1, const void* dw2,
              const void* dbias);

// bwd_check, the workspace checks, then the backward plan's launches on `stream`
// (ws: ws_bytes of device memory, at least workspace_bytes(pr)).
int bwd_impl(const Problem& pr, const void* dy, const void* x, const void* w1, const void* w2,
             const void* z, const void* y, void* dx, void* dw1, void* dw2, void* dbias, void* ws,
             size_t ws_bytes, void* stream, void* const* events, int n_events);

}  // namespace monarch
