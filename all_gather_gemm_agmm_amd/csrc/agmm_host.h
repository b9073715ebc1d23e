// Status and plan bookkeeping shared by the host sources of the C ABI
// (agmm_api.cpp, agmm_ops.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "agmm.h"

namespace agmm {

// Status and message of this thread's most recent call into the library.
inline thread_local int g_status = AGMM_OK;
inline thread_local std::string g_msg;

inline int set_err(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_status = status;
  g_msg = buf;
  return status;
}

inline int ok() {
  g_status = AGMM_OK;
  g_msg.clear();
  return AGMM_OK;
}

inline int hip_err(hipError_t e, const char* what) {
  return set_err(AGMM_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

}  // namespace agmm
