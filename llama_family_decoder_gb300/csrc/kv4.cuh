// Row format of the 4-bit KV cache (see kv4.cu), and helpers to take codes out of words.
#pragma once

#include <stdint.h>

namespace blk {

constexpr int kKv4Codes = 64;   // code bytes of a row
constexpr int kKv4Scales = 16;  // 4 bf16 scales, then 4 bf16 offsets

// The channel in the low nibble of code byte b; the high nibble holds the one 8 further.
// Byte b = 16 t + 4 j + 2 u + e: block 2 j + e of 16 channels, element 2 t + u of its lower 8.
__host__ __device__ constexpr int kv4_byte_channel(int b) {
  return 16 * (2 * ((b >> 2) & 3) + (b & 1)) + 2 * (b >> 4) + ((b >> 1) & 1);
}

// (w & mask) | bits in one instruction: the mask in a register (see kept_constant), as an
// instruction has room for one constant only.
template <uint32_t BITS>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "n"(BITS));
  return r;
}
// A constant that the compiler keeps in a register instead of folding it.
__device__ __forceinline__ uint32_t kept_constant(uint32_t c) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(c));
  return r;
}

}  // namespace blk
