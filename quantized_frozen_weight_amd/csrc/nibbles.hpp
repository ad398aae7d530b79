// 4-bit codes widened for the integer products.
#pragma once
#include "common.hpp"

namespace qlora {

// Sixteen consecutive 4-bit codes (8 bytes, the even k in each low nibble)
// as sixteen int8 values in k order.
__device__ __forceinline__ i32x4 widen_nibbles(u32x2 w) {
  i32x4 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t lo = w[h] & 0x0F0F0F0Fu;             // k = 0, 2, 4, 6 of this dword
    uint32_t hi = (w[h] >> 4) & 0x0F0F0F0Fu;      // k = 1, 3, 5, 7
    lo |= (lo & 0x08080808u) * 30u;               // sign-extend each nibble
    hi |= (hi & 0x08080808u) * 30u;
    out[2 * h] = (int)__builtin_amdgcn_perm(hi, lo, 0x05010400u);      // k 0..3
    out[2 * h + 1] = (int)__builtin_amdgcn_perm(hi, lo, 0x07030602u);  // k 4..7
  }
  return out;
}

// The same codes times 16: a code in the upper half of a byte is 16 q with its
// sign in place.
__device__ __forceinline__ i32x4 widen_nibbles16(u32x2 w) {
  i32x4 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = (w[h] << 4) & 0xF0F0F0F0u, hi = w[h] & 0xF0F0F0F0u;   // even k, odd k
    out[2 * h] = (int)__builtin_amdgcn_perm(hi, lo, 0x05010400u);
    out[2 * h + 1] = (int)__builtin_amdgcn_perm(hi, lo, 0x07030602u);
  }
  return out;
}

}  // namespace qlora
