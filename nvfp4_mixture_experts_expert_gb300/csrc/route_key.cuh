// Order-preserving key of a (logit, expert) pair, shared by the routing kernels.
#pragma once
#include <cstdint>

namespace nvfp4 {

// Order-preserving key of a (logit, expert) pair: larger logit first, equal
// logits -> lower expert first.  Lanes with no expert get key 0, below every
// real key (also below -inf logits).
__device__ __forceinline__ uint64_t route_key(float v, int e) {
  uint32_t u = __float_as_uint(v);
  if (u == 0x80000000u) u = 0u;  // -0 ranks equal to +0
  const uint32_t ord = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)ord << 32) | (uint32_t)(0xFFFFFFFFu - (uint32_t)e);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t ord = (uint32_t)(key >> 32);
  return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7FFFFFFFu) : ~ord);
}
__device__ __forceinline__ int key_expert(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

}  // namespace nvfp4
