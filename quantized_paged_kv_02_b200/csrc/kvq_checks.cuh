// Host-side checks of arguments that the entry points around the cache share (rotary positions, rows
// read back, accepted paths).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace kvq {

// Do n bytes at a and m bytes at b overlap?
inline bool bytes_overlap(const void* a, size_t n, const void* b, size_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return n > 0 && m > 0 && x < y + m && y < x + n;
}

}  // namespace kvq
