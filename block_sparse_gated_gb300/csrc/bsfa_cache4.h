// bsfa_cache4.h -- internal: argument checks shared by the 4-bit cache's
// entry points.
#pragma once
#include <cstdint>

#include "bsfa.h"

namespace bsfa {

constexpr int CACHE4_MAX_BATCH = 4096;  // sequences per call
constexpr int CACHE4_MAX_HEADS = 4096;  // KV heads

// Sizes (no pointer is looked at), then pointers and strides.
bsfa_status validate_cache4(const bsfa_cache4* c);
bsfa_status validate_cache4_pointers(const bsfa_cache4* c);

// 16-bit rows: a base on 16 bytes, and strides that keep every row there (a
// dimension of extent 1 has no stride to speak of).
inline bool rows_aligned(const void* base, const int64_t (&stride)[3], const int64_t (&extent)[3]) {
  if (reinterpret_cast<uintptr_t>(base) & 15u) return false;
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1 && (stride[i] <= 0 || stride[i] % 8)) return false;
  return true;
}

}  // namespace bsfa
