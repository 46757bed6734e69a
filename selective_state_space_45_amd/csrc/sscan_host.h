// Host-side helpers shared by the C entry points: errors, buffer checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sscan {

// The calling thread's error message and the status code that goes with it.  The
// message lives in a fixed array: nothing here allocates, so nothing throws.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();
int hip_fail(hipError_t e, const char* what);

inline bool overlaps(const void* a, size_t abytes, const void* b, size_t bbytes) {
  if (!a || !b || abytes == 0 || bbytes == 0) return false;
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  return pa < pb + bbytes && pb < pa + abytes;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

struct Buf {
  const void* p;
  size_t n;
};

}  // namespace sscan
