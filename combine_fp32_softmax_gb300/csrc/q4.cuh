// The 4-bit weight format: W[r, c] = s[c / G, r] * (q[r, c] - 8), q in 0..15,
// one bf16 scale per group of G columns of a row.
//
// Eight columns 8j..8j+7 of a row share one 32-bit word: columns 0, 2, 4, 6
// in nibbles 0..3, columns 1, 3, 5, 7 in nibbles 4..7.  So word >> 4i masked
// with 0x000F000F holds columns 2i and 2i+1 in its two halves: one shift and
// one mask-and-or make a pair of neighbouring bf16 values.
#pragma once
#include <cuda_bf16.h>

#include <cstddef>
#include <cstdint>

namespace moe {

// Scales are stored [cols / G][rows rounded up to 8]: a row of scales (one
// group, all matrix rows) then starts on a 16-byte boundary whatever the
// row count, as TMA needs.
__host__ __device__ constexpr size_t q4_scale_pitch(size_t rows) { return (rows + 7) / 8 * 8; }

#ifdef __CUDACC__
// bf16x2 bits 0x4300 | n are 128 + n exactly (n < 128: the step of bf16 in
// [128, 256) is 1), and subtracting 136 is exact too, so the result is q - 8
// without rounding.  One shift, one mask-and-or, one fused multiply-add: the
// integer instructions issue at half rate, so the C++ form, which compiles to
// one more of them, took 1.45 times as long.
__device__ __forceinline__ uint32_t q4_pair(uint32_t word, int i) {
  uint32_t biased, v;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(biased) : "r"(word >> (4 * i)));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(biased), "r"(0x3F803F80u), "r"(0xC308C308u));
  return v;
}
// The four pairs of a word as (q - 8) / 64, exact in bf16, with two integer
// instructions less.  bf16 bit patterns below 256 are equidistant numbers,
// pattern b being b 2^-133 (the subnormals and the first binade share their
// step), so a nibble in bits 0-3 or 4-7 of a half is the number q or 16 q
// times 2^-133 as it stands, and one exact fused multiply-add by 2^127 or
// 2^123 brings it to its place.
constexpr float kQ4Unit = 64.f;  // what the pairs have to be multiplied by
__device__ __forceinline__ void q4_pairs(uint32_t word, uint32_t (&v)[4]) {
  const uint32_t up = word >> 8;
  const uint32_t m = 0x000F000Fu, bias = 0xBE00BE00u;  // -8 / 64
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[0]) : "r"(word & m), "r"(0x7F007F00u), "r"(bias));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[1]) : "r"(word & (m << 4)), "r"(0x7D007D00u), "r"(bias));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[2]) : "r"(up & m), "r"(0x7F007F00u), "r"(bias));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[3]) : "r"(up & (m << 4)), "r"(0x7D007D00u), "r"(bias));
}
#endif

}  // namespace moe
