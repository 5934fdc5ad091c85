// The steps' coefficients and the fp16 scales of their matrices, shared by the
// products of ortho.cu and the one-launch form of ortho_small.cu.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace moe {
namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
// In the last two steps the polynomial is kept as B + 2.5 I, and the step is
// (a - 2.5) X + (B + 2.5 I) X: where X nears orthogonality the diagonal of B nears
// b + c = -2.74, and its rounding to fp16 would be as large as all others together.
// Before, X's own part stays out of the product (see kLo).
constexpr float kNsShift = 2.5f;
constexpr int kShiftSteps = 2;
// What rounding to fp16 leaves of X is kept too, times 2^9 in e4m3 (four bits more),
// for the a X of every step but the last.  The steps raise a small singular value 485-fold, and the
// roundings of X have parts in every direction, also where G has nothing: without
// these bits a 704 x 1024 matrix of rank 100 comes out 1.7e-2 of its norm off, with
// them 2.6e-3 (rank 20: 4.2e-2 and 2.9e-3; full rank 1.9e-3 and 1.8e-3).
constexpr float kLo = 512.f;
constexpr float kNsEps = 1e-7f;
// |X| <= 1 in the Frobenius norm at first and its singular values stay below
// 1.3, so entries of X, A, B are below 1.3, 1.7, 14: times 2^10, 2^12, 2^11 they
// stay below fp16's 65504, and entries 2^-24, 2^-26, 2^-25 are still normal.
constexpr float kSX = 1024.f, kSA = 4096.f, kSB = 2048.f;
constexpr int kSXLog2 = 10;
// X of step i is step_scale(...) times what is stored.  A matrix whose norm is small
// beside eps grows by kNsA a step at first and is stored in units that grow with it,
// so it loses nothing to fp16's range.
__device__ __forceinline__ float step_scale(float scal, float grown) { return fminf(1.f / kSX, scal * grown); }
// Below this norm of X the steps are linear for all of the most there may be (kNsA^16
// is 2^28.6): the result is a^steps X.
constexpr float kTiny = 0x1p-80f;
// The norm from the whole sum of squares: infinite past fp32's range.  A part of the sum
// may leave that range only where the whole does, so what counts as infinite does not
// depend on how the parts are shared out.
__device__ __forceinline__ float norm_of(double squares) {
  return squares > 0x1.fffffep127 ? INFINITY : static_cast<float>(sqrt(squares));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Two fp32 values to e4m3 (lo in the lower byte), and two back.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return unpack_f16(h);
}
// What x lost when it was rounded to the fp16 pair `hi`, in e4m3.
__device__ __forceinline__ uint32_t rest_e4m3(float x0, float x1, uint32_t hi) {
  const float2 h = unpack_f16(hi);
  return pack_e4m3(kLo * (x0 - h.x), kLo * (x1 - h.y));
}

}  // namespace
}  // namespace moe
