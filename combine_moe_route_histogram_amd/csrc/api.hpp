// What the C entry points share: argument checks, error records, stream and
// workspace helpers (defined in moe_api.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {

// Records the message that moe_last_error() gives on this thread; returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_status(hipError_t e, const char* what);
int check_dims(const moe_dims* d);
int check_ptr(const void* p, const char* name);   // non-null, 16-byte aligned

constexpr size_t kAlign = 256;   // of workspaces and their sections
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

#define MOE_TRY(expr)            \
  do {                           \
    const int _s = (expr);       \
    if (_s != MOE_OK) return _s; \
  } while (0)

}  // namespace moe
