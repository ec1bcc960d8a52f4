// Host-side helpers that the sources of the C ABI share.
#pragma once

#include <stdint.h>

namespace mega_moe {

// Sets the calling thread's message (mega_moe_last_error) and returns code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the calling thread's message and returns MEGA_MOE_OK.
int ok();

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace mega_moe
