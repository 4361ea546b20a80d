// Host helpers shared by the C ABI's source files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "moelora.h"

namespace moelora {

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// MOELORA_OK when the current device is a gfx950 (looked up once per device).
inline int check_device() {
  static int known[64];  // 0 unknown, 1 gfx950, -1 other
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MOELORA_EHIP;
  if (dev < 0 || dev >= 64) return MOELORA_EDEVICE;
  if (known[dev] == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MOELORA_EHIP;
    known[dev] = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
  }
  return known[dev] == 1 ? MOELORA_OK : MOELORA_EDEVICE;
}

}  // namespace moelora
