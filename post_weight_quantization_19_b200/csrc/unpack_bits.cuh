// Unpacking of 32 codes from BITS int32 words (the LSB-first stream of
// pack_bits.cuh).
#pragma once

#include <stdint.h>

namespace gptq {

// Code j (a compile-time constant after unrolling) of a 32-code chunk.
template <int BITS>
__device__ __forceinline__ uint32_t code_at(const uint32_t (&w)[BITS], int j) {
  constexpr uint32_t mask = (1u << BITS) - 1u;
  const int pos = j * BITS, wi = pos >> 5, off = pos & 31;
  uint32_t v = w[wi] >> off;
  if (off + BITS > 32) v |= w[wi + 1] << (32 - off);
  return v & mask;
}

}  // namespace gptq
