// What the files of the C ABI share: the calling thread's error text, and
// small helpers for workspaces and pointers (internal to libmoe.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// Sets the calling thread's error text and returns st.
moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it and returns MOE_OK.
moe_status ok();
moe_status hip_fail(hipError_t e, const char* what);

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

#define MOE_CHECK_LAUNCH(expr, what)                      \
  do {                                                    \
    hipError_t e_ = (expr);                               \
    if (e_ != hipSuccess) return moe::hip_fail(e_, what); \
  } while (0)

}  // namespace moe
