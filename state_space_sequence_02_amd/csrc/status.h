// Error reporting and argument checks shared by the C ABI's source files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m2 {

// Records the calling thread's last-error text and returns `status`.
int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// The calling thread's last-error text ("" if none).
const char* last_error();
// Clears the last-error text and returns MAMBA2_OK.
int ok();
// A required pointer: non-NULL and 16-byte aligned.
int need(const void* p, const char* name);
// An optional pointer: NULL or 16-byte aligned.
int maybe(const void* p, const char* name);
int hip_status(hipError_t e, const char* where);
// A workspace of at least `needed` bytes, 256-byte aligned.
int need_workspace(const void* p, size_t bytes, size_t needed);

inline size_t round256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace m2

#define CHECK(expr)               \
  do {                            \
    const int rc_ = (expr);       \
    if (rc_ != MAMBA2_OK) return rc_; \
  } while (0)
