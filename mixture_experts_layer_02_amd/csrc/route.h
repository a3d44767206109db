// Logits as unsigned keys of the same order, for the top-k of route.hip's kernels and of the decode step.
#pragma once

#include "common.h"

namespace moe {

// Order-preserving unsigned key of a float (larger float, larger key), with
// -0.0 made equal to +0.0; 0 is below every finite float's key and marks an
// absent element.  key_float inverts it (+0.0 for the key of zero).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0.0 + 0.0 = +0.0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

}  // namespace moe
