// What the C entry points share: the calling thread's error message and the device check (ple_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ple {

int fail(int code, const char* fmt, ...);
int ok();
int hip_fail(hipError_t e, const char* what);
int check_device();  // the current device must be gfx950 (checked once per device)

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace ple
