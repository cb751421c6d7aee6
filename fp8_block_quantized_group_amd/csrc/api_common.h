// Status, message and argument helpers shared by the C ABI's sources.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/moe_fp8.h"

namespace moe {

// sets the thread's message and returns `code`
moe_status_t fail(moe_status_t code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// clears the message
moe_status_t ok();
moe_status_t launch_status(hipError_t err, const char* what);
moe_status_t check_ptr(const void* ptr, const char* name, size_t align);

constexpr size_t kAlign = 256;
inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace moe

#define CHECK(expr)                         \
  do {                                      \
    const moe_status_t _s = (expr);         \
    if (_s != MOE_OK) return _s;            \
  } while (0)
