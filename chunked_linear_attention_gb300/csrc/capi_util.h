// What the files of the C boundary share (defined in capi.cu).
#pragma once

#include <cstdint>

namespace ttt {

// Device address of the status word for the current device, or NULL.
int* capi_status_ptr();
// The bounded-wait limit set by ttt_set_wait_limit_ns.
unsigned long long capi_wait_limit_ns();

inline bool capi_aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace ttt
