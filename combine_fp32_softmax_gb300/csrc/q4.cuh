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
#endif

}  // namespace moe
