// 8-bit tensors: e4m3 codes with a power of two for each 32 columns of a row.
//
// A row's block of 32 columns has one byte b, 2^(b - 127): the least power
// with which the block's largest value stays within e4m3's 448, so nothing is
// ever cut off; 255 (NaN) where a value is NaN or infinite. Both the products
// and ple_mx8_read take code * 2^(b - 127).
//
// The bytes lie as the tensor cores' scale operands do: for each 128 rows and
// 128 columns a piece of 512 bytes, [row % 32][row % 128 / 32][block % 4], the
// pieces of a row block one after the other. A product's stage thus fetches
// its scales in one piece and hands them to tensor memory in one copy.
#pragma once

#include "common.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace ple {

constexpr int kMxBlock = 32;     // columns that share a scale
constexpr int kMxTile = 128;     // rows and columns of a piece of scales
constexpr int kMxPiece = 512;    // bytes of it

// Byte of row r's block of columns j.
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t r, int j, int columns) {
  return ((r >> 7) * (columns >> 7) + (j >> 2)) * kMxPiece + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (j & 3);
}

// Scale byte of a block whose largest magnitude has these float32 bits: with
// top = m 2^q, m in [1, 2), the exponent is q - 8, or q - 7 where m > 1.75
// (448 = 1.75 * 2^8): the carry of the added bits says which.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255;
  const int b = static_cast<int>((top + 0x1FFFFFu) >> 23) - 8;
  return b > 0 ? b : 0;
}

// 2^(b - 127), b < 255; 2^-127 is a subnormal. NaN for 255.
__device__ __forceinline__ float mx_power(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}
// 2^(127 - b): what values are multiplied by before they become codes. Scale
// bytes are 247 at most, or 255: its codes do not matter, they read as NaN.
__device__ __forceinline__ float mx_inverse(uint32_t b) { return __uint_as_float(b == 255 ? 0u : (254 - b) << 23); }

// Codes of two and four scaled values, the first in the lowest byte.
__device__ __forceinline__ uint32_t mx_codes2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d) {
  return mx_codes2(a, b) | mx_codes2(c, d) << 16;
}

// Values of two codes, unscaled.
__device__ __forceinline__ float2 mx_values2(uint32_t codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes), __NV_E4M3)));
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// 32 bytes in one store, where the address is a multiple of 32 (a whole sector
// at a time), or two.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4* const p = static_cast<uint4*>(to);
    p[0] = make_uint4(v[0], v[1], v[2], v[3]);
    p[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Larger magnitude of three values, NaN if one is.
__device__ __forceinline__ float abs_max(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Bytes of a tensor's scales, or -1 for sizes that have none.
inline int64_t mx_scale_size(int64_t rows, int64_t columns) {
  if (rows < 0 || rows > INT32_MAX || columns < kMxTile || columns % kMxTile != 0 || columns > INT32_MAX) return -1;
  return (rows + kMxTile - 1) / kMxTile * (columns / kMxTile) * kMxPiece;
}

}  // namespace ple
