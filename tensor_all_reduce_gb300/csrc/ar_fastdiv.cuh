// Division by an invariant on the device (see FastDiv).
#pragma once

#include "ar_serve.h"

namespace ar {

__device__ __forceinline__ int operator/(int n, const FastDiv& f) { return (int)((__umulhi((uint32_t)n, f.m) + (uint32_t)n) >> f.s); }

}  // namespace ar
