// The steps' coefficients and the fp16 scales of their matrices, shared by the
// products of ortho.cu and the one-launch form of ortho_small.cu.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace moe {
namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
// The polynomial is kept as B + 2.5 I, and the step is (a - 2.5) X + (B + 2.5 I) X:
// where X nears orthogonality the diagonal of B nears b + c = -2.74, and its
// rounding to fp16 would be as large as all others together.
constexpr float kNsShift = 2.5f;
constexpr float kNsEps = 1e-7f;
// |X| <= 1 in the Frobenius norm at first and its singular values stay below
// 1.3, so entries of X, A, B are below 1.3, 1.7, 14: times 2^10, 2^12, 2^11 they
// stay below fp16's 65504, and entries 2^-24, 2^-26, 2^-25 are still normal.
constexpr float kSX = 1024.f, kSA = 4096.f, kSB = 2048.f;
constexpr int kSXLog2 = 10;
// Below this norm of X the cubic term of a step is under 2^-19 of the linear one
// for five steps on: the result is a^steps X.
constexpr float kTiny = 0x1p-17f;

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

}  // namespace
}  // namespace moe
