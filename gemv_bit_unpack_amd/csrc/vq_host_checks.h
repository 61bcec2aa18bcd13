// What the host sides of the operators share: checks of types and alignment, pieces of a workspace.
#pragma once

#include <cstddef>
#include <cstdint>

#include "vq_internal.h"

namespace vqi {

inline bool valid_dtype(vq_dtype t) { return t == VQ_F16 || t == VQ_BF16 || t == VQ_F32; }
inline size_t size_of(vq_dtype t) { return t == VQ_F32 ? 4 : 2; }
inline size_t padded(size_t n) { return (n + 255) / 256 * 256; }
inline bool misaligned(const void* p, size_t a) { return p && !aligned(p, a); }

// Consecutive 256-byte aligned pieces of a workspace.
struct Pieces {
  uint8_t* base;
  size_t at = 0;
  void* take(size_t n) {
    void* p = base ? base + at : nullptr;
    at += padded(n);
    return p;
  }
};

}  // namespace vqi
