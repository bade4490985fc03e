// sb_host.h -- what the host files of the library share: error reporting,
// device properties and argument checks.
#pragma once

#include <stdint.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/seam_blend.h"

extern "C" int sb_fail_message(int code, const char *msg); // abi.cpp
extern "C" int sb_cu_count(void);                          // abi.cpp

namespace sb {

inline int failf(int code, const char *fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return sb_fail_message(code, buf);
}

inline bool aligned(const void *p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
inline int elem_bytes(int dtype) { return dtype == SB_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) { return dtype == SB_F32 || dtype == SB_F16 || dtype == SB_BF16; }

} // namespace sb
