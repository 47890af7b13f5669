// Unpacking of 4-bit codes, eight to a word, and packed bf16 arithmetic.
#pragma once

#include "common.cuh"

namespace ple {

// Codes i and i + 4 of a word (i = 0..3) where they stand: read as f16 pair,
// c 2^-24 for even i and c 2^-20 for odd i; read as bf16, c 2^-133 and c 2^-129.
__device__ __forceinline__ uint32_t code_bits(uint32_t word, int i) {
  return (i < 2 ? word : word >> 8) & (i % 2 == 0 ? 0x000F000Fu : 0x00F000F0u);
}

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t bf2_mad(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
  return y;
}

}  // namespace ple
