// mnw_int4_row.cuh -- a cached head row in 4 bits.
//
// A row of d elements is four groups of d / 4.  The row's record is a float32
// scale S and a multiplier m (1 .. 255, 8 bits) for each group; an element is
// code * m * S with codes of -7 .. 7, held as code + 8.  Of eight elements,
// element e lies at bits 4 (e / 2) + 16 (e % 2) of a 32-bit word, so a shift and
// a mask leave two neighbours in the halves of a register.
//
// Two levels, because keys have channels much larger than the rest, which one
// scale a row would leave no codes for the others, and because code * m, an
// integer of at most 11 bits, is exact in FP16: the tensor cores take it as it
// is, and the scale multiplies FP32 scores and probabilities.
#pragma once
#include <cstdint>

#include "mnw_convert.cuh"

namespace mnw {
namespace int4row {

constexpr int kRecord = 8;  // bytes of a row's record
// Operands hold code * m * 2^-24: a nibble under an exponent of zero is that multiple of FP16's smallest value.
constexpr float kUnit = 16777216.f;

// A group's multipliers as FP16 pairs: m, m / 16 (for nibbles that lie four bits up) and -8 m 2^-24.
struct Mul {
  uint32_t m, m16, off;
};
// t: the two multipliers in bytes 0 and 2 (the others hold anything)
__device__ __forceinline__ Mul multipliers(uint32_t t) {
  Mul x;
  uint32_t h;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(h) : "r"(t), "r"(0x00FF00FFu), "r"(0x64006400u));  // (t & mask) | 1024
  x.m = f16x2_sub(h, 0x64006400u);
  x.m16 = f16x2_mul(x.m, 0x2C002C00u);
  x.off = f16x2_mul(x.m, 0x80088008u);
  return x;
}
// Pair j of a word (elements 2 j, 2 j + 1 of its eight): (code m) 2^-24, exact.
template <int J>
__device__ __forceinline__ uint32_t pair(uint32_t w, const Mul& x) {
  const uint32_t y = J < 2 ? w : w >> 8;
  return f16x2_fma(y & ((J & 1) ? 0x00F000F0u : 0x000F000Fu), (J & 1) ? x.m16 : x.m, x.off);
}

}  // namespace int4row
}  // namespace mnw
