// qpn_kv_order.h -- FP16 numbers as integers in their order, and keys that put tokens
// in the order of their logits.  (constexpr: for the kernels and for host code alike.)
#pragma once

#include <stdint.h>

namespace qpn {

// Ascending in the value: the bits of an FP16 number (-0 as 0).  From 1 on whatever the bits are:
// 0 stands for "none" where values are counted, so that a NaN, which has no place in the order,
// must not be one either (0xFFFF, of which a buffer of bytes 0xFF consists, would be).
constexpr uint32_t ordered_bits(uint32_t b) {
  b = b == 0x8000u ? 0u : b;
  const uint32_t o = b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u;
  return o ? o : 1u;
}
// And back to bits.
constexpr uint32_t bits_of_ordered(uint32_t o) { return o & 0x8000u ? o ^ 0x8000u : o ^ 0xFFFFu; }

// Descending in the value, then ascending in the index (below 2^24).
constexpr uint64_t key_of(uint32_t order, uint32_t index) {
  return (uint64_t)order << 32 | (0xFFFFFFFFu - index);
}
constexpr int index_of(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

}  // namespace qpn
