// bf16 matrices to 4-bit codes with group scales, and back (format: q4.cuh).
//
// Both directions move every byte once.  66 x 1408 x 2048, G=64: dequantise 73
// us, 6570 GB/s, HBM-bound; quantise 93 us, 5170 GB/s, bound by instructions
// (104 us with one fp32 value to an instruction).  One block takes 32 rows x 256 columns, a
// warp one row of it at a time: 16 bytes of bf16 and 4 of codes per thread, so
// a warp's accesses are whole 512- and 128-byte stretches.  A group's maximum
// is a shuffle reduction over its G / 8 threads.  The scales of the tile go
// through shared memory, because consecutive scales in memory belong to
// consecutive rows.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"
#include "trace.h"

namespace moe {

namespace {

constexpr int kQ4Rows = 32, kQ4Cols = 256, kQ4Warps = 8;
constexpr int kQ4RowsPerWarp = kQ4Rows / kQ4Warps;

struct Q4Tile {
  int mat, row0, col0;
};

// Tiles fit 32 bits: 2^31 of them are 35 TB of weights.
__device__ __forceinline__ Q4Tile q4_tile(unsigned i, unsigned row_tiles, unsigned col_tiles) {
  Q4Tile t;
  const unsigned r = i / col_tiles;
  t.col0 = static_cast<int>(i - r * col_tiles) * kQ4Cols;
  t.mat = static_cast<int>(r / row_tiles);
  t.row0 = static_cast<int>(r - t.mat * row_tiles) * kQ4Rows;
  return t;
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

// Two fp32 values to an instruction.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

// The codes 8 + rint(x / s) of eight bf16 values |x| <= 7.1 s, s bf16 and
// normal, r within 1 ulp of 1 / s.  x r and one Newton step give a quotient
// that is exact where x / s is halfway between two integers and otherwise on
// the right side of it (over all significands of x and s; x / s is at least
// 2^-14 of itself away from halfway where it is not halfway).  Adding
// 1.5 * 2^23 then rounds it to an integer, ties to even.  The codes of the even
// columns and of the odd ones are put together as numbers (below 2^16: exact),
// which end up in the low halves of 2^23 + them.
__device__ __forceinline__ uint32_t q4_word(const uint32_t (&w)[4], float s, float r) {
  constexpr float kRound = 12582912.f;
  const uint64_t rr = pair_of(r, r), ss = pair_of(-s, -s);
  uint64_t word = 0;
#pragma unroll
  for (int p = 3; p >= 0; --p) {
    const uint64_t x = pair_of(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xFFFF0000u));
    const uint64_t y = mul2(x, rr), q = fma2(fma2(y, ss, x), rr, y);
    const uint64_t code = add2(add2(q, pair_of(kRound + 8.f, kRound + 8.f)), pair_of(-kRound, -kRound));
    word = p == 3 ? code : fma2(word, pair_of(16.f, 16.f), code);
  }
  word = add2(word, pair_of(8388608.f, 8388608.f));
  return __byte_perm(static_cast<uint32_t>(word), static_cast<uint32_t>(word >> 32), 0x5410);
}
__device__ __forceinline__ float rcp_approx(float s) {  // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}
// The same by division, for subnormal scales (whose rounding can leave x / s
// beyond the range, too) and those with a subnormal reciprocal.
__device__ __noinline__ uint32_t q4_code_exact(float x, float s) {
  return min(max(__float2int_rn(x / s), -8), 7) + 8;
}

// The scales of a tile between memory, [group][row], and the threads.
template <int G, typename F>
__device__ __forceinline__ void q4_tile_scales(const Q4Tile& t, int cols, const F& each) {
  constexpr int GROUPS = kQ4Cols / G;
  const int groups = cols / G, g0 = t.col0 / G;
#pragma unroll
  for (int e0 = 0; e0 < GROUPS * kQ4Rows; e0 += kQ4Warps * 32) {
    const int e = e0 + static_cast<int>(threadIdx.x), g = e / kQ4Rows, rr = e % kQ4Rows;
    if (e < GROUPS * kQ4Rows && g0 + g < groups)
      each(g, rr, static_cast<size_t>(t.mat) * groups + g0 + g);
  }
}

template <int G>
__global__ void __launch_bounds__(kQ4Warps * 32)
    q4_quantize_kernel(const uint16_t* __restrict__ W, uint8_t* __restrict__ codes, uint16_t* __restrict__ scales,
                       int rows, int cols, unsigned row_tiles, unsigned col_tiles, unsigned tiles) {
  __shared__ uint16_t s_scale[kQ4Cols / G][kQ4Rows];
  constexpr int LANES = G / 8;  // threads of a group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t pitch = q4_scale_pitch(rows);
  for (unsigned i = blockIdx.x; i < tiles; i += gridDim.x) {
    const Q4Tile t = q4_tile(i, row_tiles, col_tiles);
    const int col = t.col0 + lane * 8;
    const bool in = col < cols;  // cols is a multiple of the group: a group is wholly in or out
    const size_t first = (static_cast<size_t>(t.mat) * rows + t.row0 + warp) * cols + col;
    const size_t step = static_cast<size_t>(kQ4Warps) * cols;
    uint4 v[kQ4RowsPerWarp];
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (in && t.row0 + j * kQ4Warps + warp < rows) v[j] = *reinterpret_cast<const uint4*>(W + first + j * step);
    }
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int rr = j * kQ4Warps + warp;
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      // bf16 magnitudes order like their bits; Inf and NaN come out on top,
      // so a group that holds one gets a non-finite scale
      uint32_t top2 = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                               __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
#pragma unroll
      for (int off = 1; off < LANES; off <<= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, off));
      const float top = bf16_value(max(top2 & 0xFFFFu, top2 >> 16));
      // rounded to bf16 the product is the quotient by 7 for every significand
      __nv_bfloat16 sb = __float2bfloat16_rn(top * (1.f / 7.f));
      float s = __bfloat162float(sb);
      const uint32_t exponent = __float_as_uint(s) >> 23;  // s >= 0
      uint32_t word;
      if (exponent > 1 && exponent < 253) {  // s and 1 / s well inside the normal range
        word = q4_word(w, s, rcp_approx(s));
      } else {
        sb = __float2bfloat16_rn(top / 7.f);
        s = __bfloat162float(sb);
        const bool some = s > 0.f && isfinite(s);
        word = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) {  // even columns in the lower half, odd ones in the upper
          word |= (some ? q4_code_exact(__uint_as_float(w[p] << 16), s) : 8) << (4 * p);
          word |= (some ? q4_code_exact(__uint_as_float(w[p] & 0xFFFF0000u), s) : 8) << (4 * p + 16);
        }
      }
      const bool row_in = t.row0 + rr < rows;
      if (in && row_in) *reinterpret_cast<uint32_t*>(codes + (first + j * step) / 2) = word;
      if (lane % LANES == 0) s_scale[lane / LANES][rr] = row_in ? __bfloat16_as_ushort(sb) : 0;
    }
    __syncthreads();
    q4_tile_scales<G>(t, cols, [&](int g, int rr, size_t row) {
      if (static_cast<size_t>(t.row0 + rr) < pitch) scales[row * pitch + t.row0 + rr] = s_scale[g][rr];
    });
    __syncthreads();  // the next tile rewrites s_scale
  }
}

template <int G>
__global__ void __launch_bounds__(kQ4Warps * 32)
    q4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                         uint16_t* __restrict__ W, int rows, int cols, unsigned row_tiles, unsigned col_tiles,
                         unsigned tiles) {
  __shared__ uint16_t s_scale[kQ4Cols / G][kQ4Rows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t pitch = q4_scale_pitch(rows);
  for (unsigned i = blockIdx.x; i < tiles; i += gridDim.x) {
    const Q4Tile t = q4_tile(i, row_tiles, col_tiles);
    const int col = t.col0 + lane * 8;
    const bool in = col < cols;
    const size_t first = (static_cast<size_t>(t.mat) * rows + t.row0 + warp) * cols + col;
    const size_t step = static_cast<size_t>(kQ4Warps) * cols;
    uint32_t word[kQ4RowsPerWarp];
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      word[j] = 0;
      if (in && t.row0 + j * kQ4Warps + warp < rows)
        word[j] = *reinterpret_cast<const uint32_t*>(codes + (first + j * step) / 2);
    }
    q4_tile_scales<G>(t, cols, [&](int g, int rr, size_t row) {
      if (t.row0 + rr < rows) s_scale[g][rr] = scales[row * pitch + t.row0 + rr];
    });
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int rr = j * kQ4Warps + warp;
      if (!in || t.row0 + rr >= rows) continue;
      const __nv_bfloat162 s = __bfloat162bfloat162(__ushort_as_bfloat16(s_scale[lane / (G / 8)][rr]));
      uint32_t out[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t pair = q4_pair(word[j], p);
        const __nv_bfloat162 o = __hmul2(s, *reinterpret_cast<const __nv_bfloat162*>(&pair));  // one rounding
        out[p] = *reinterpret_cast<const uint32_t*>(&o);
      }
      *reinterpret_cast<uint4*>(W + first + j * step) = make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
  }
}

// One block a tile, up to what a grid holds with room to spare.
unsigned q4_grid(long long tiles) { return static_cast<unsigned>(std::min<long long>(tiles, 1 << 30)); }

}  // namespace

cudaError_t launch_q4_quantize(const uint16_t* W, uint8_t* codes, uint16_t* scales, int mats, int rows, int cols,
                               int group, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_Q4, s);
  const int rt = ceil_div(static_cast<long long>(q4_scale_pitch(rows)), kQ4Rows), ct = ceil_div(cols, kQ4Cols);
  const long long tiles = static_cast<long long>(mats) * rt * ct;
  auto* kernel = group == 32 ? q4_quantize_kernel<32> : group == 64 ? q4_quantize_kernel<64> : q4_quantize_kernel<128>;
  kernel<<<q4_grid(tiles), kQ4Warps * 32, 0, s>>>(W, codes, scales, rows, cols, rt, ct, static_cast<unsigned>(tiles));
  return cudaGetLastError();
}

cudaError_t launch_q4_dequantize(const uint8_t* codes, const uint16_t* scales, uint16_t* W, int mats, int rows,
                                 int cols, int group, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_Q4, s);
  const int rt = ceil_div(rows, kQ4Rows), ct = ceil_div(cols, kQ4Cols);
  const long long tiles = static_cast<long long>(mats) * rt * ct;
  auto* kernel =
      group == 32 ? q4_dequantize_kernel<32> : group == 64 ? q4_dequantize_kernel<64> : q4_dequantize_kernel<128>;
  kernel<<<q4_grid(tiles), kQ4Warps * 32, 0, s>>>(codes, scales, W, rows, cols, rt, ct, static_cast<unsigned>(tiles));
  return cudaGetLastError();
}

}  // namespace moe
