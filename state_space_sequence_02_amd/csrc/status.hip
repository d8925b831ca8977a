// The calling thread's last-error text and the argument checks that every
// C ABI source file uses.
#include "status.h"

#include <stdarg.h>
#include <stdio.h>

#include "mamba2_ssd.h"

namespace m2 {

namespace {

thread_local char g_last_error[512] = "";

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

const char* last_error() { return g_last_error; }

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return status;
}

int ok() {
  g_last_error[0] = '\0';
  return MAMBA2_OK;
}

int need(const void* p, const char* name) {
  if (!p) return fail(MAMBA2_ERR_NULL, "%s is NULL", name);
  if (!aligned16(p)) return fail(MAMBA2_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return MAMBA2_OK;
}

int maybe(const void* p, const char* name) {
  if (p && !aligned16(p)) return fail(MAMBA2_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return MAMBA2_OK;
}

int hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return ok();
  return fail(MAMBA2_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

int need_workspace(const void* p, size_t bytes, size_t needed) {
  if (!p) return fail(MAMBA2_ERR_WORKSPACE, "workspace is NULL");
  if (((uintptr_t)p & 255u) != 0)
    return fail(MAMBA2_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (bytes < needed)
    return fail(MAMBA2_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, needed);
  return MAMBA2_OK;
}

}  // namespace m2
