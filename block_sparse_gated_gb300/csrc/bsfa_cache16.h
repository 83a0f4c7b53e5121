// bsfa_cache16.h -- internal: argument checks shared by the 16-bit cache's
// entry points.
#pragma once
#include <cstdint>

#include "bsfa.h"

namespace bsfa {

// Sizes (no pointer is looked at), then pointers and strides.
bsfa_status validate_cache16(const bsfa_cache16* c);
bsfa_status validate_cache16_pointers(const bsfa_cache16* c);

}  // namespace bsfa
