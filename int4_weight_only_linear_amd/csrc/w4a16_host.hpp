// What the host translation units of libw4a16 share: status and message of a
// failing call, pointer checks, and the per-device property cache.
#pragma once

#include "w4a16.h"

#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

// sets the thread's message and returns st; ok() clears it
w4a16_status fail(w4a16_status st, const char* fmt, ...);
w4a16_status ok();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// [a, a + na) and [b, b + nb) overlap
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + nb && pb < pa + na;
}

inline size_t act_bytes(int64_t n) { return (size_t)n * 2; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// ---- per-device properties, filled once per device ------------------------
struct DeviceInfo {
  bool ready = false;
  int err = 0;  // a hipError_t
  bool gfx950 = false;
  int cu_count = 0;
  char arch[64] = {0};
  // this device's copy of `scratch` (w4a16_linear_noalloc), set up on the
  // entry point's first call on the device
  bool scratch_ready = false;
  void* scratch_ptr = nullptr;
};

// the current device's, refusing devices that are not gfx950
w4a16_status device_info(const DeviceInfo** out);
// the CU count that plans are made for: the current device's, or MI355X's
// where none is visible (clears the thread's message)
int planning_cus();

}  // namespace w4a16
