// abi.h -- what the C entry points share: pointer checks, the status of a HIP
// call, and the guard that keeps C++ exceptions inside the library.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/w4a16.h"

namespace w4a16 {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline int check_ptrs(std::initializer_list<const void*> required) {
  for (const void* p : required) {
    if (!p) return W4A16_ERR_INVALID_ARG;
  }
  for (const void* p : required) {
    if (!aligned16(p)) return W4A16_ERR_MISALIGNED;
  }
  return W4A16_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

// The launchers report hipGetLastError() after their launches; an error an
// earlier runtime call of the caller left pending is cleared (consumed) first
// so that it is not reported as this call's failure.
inline void clear_pending_error() { (void)hipGetLastError(); }

// Runs an entry point's body so that no C++ exception crosses the C ABI: a
// failed host allocation (std::bad_alloc) or any other exception becomes
// W4A16_ERR_HOST.
template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return W4A16_ERR_HOST;
  }
}

inline int validate_dtype(int32_t dtype) {
  return (dtype == W4A16_F16 || dtype == W4A16_BF16) ? W4A16_OK : W4A16_ERR_INVALID_ARG;
}

// Bytes rounded up to the parts a workspace is divided in.
inline int64_t pad256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// HIP takes grids of less than 2^32 work-items.
inline bool too_large(int64_t workgroups, int64_t threads) {
  return workgroups > (((int64_t)1 << 32) - 1) / threads;
}

}  // namespace w4a16
