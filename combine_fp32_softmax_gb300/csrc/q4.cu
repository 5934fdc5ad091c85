// bf16 matrices to 4-bit codes with group scales, and back (format: q4.cuh).
//
// Both directions move every byte once: HBM-bound.  One block takes 32 rows
// x 256 columns, a warp one row of it at a time: 16 bytes of bf16 and 4 of
// codes per thread, so a warp's accesses are whole 512- and 128-byte
// stretches.  A group's maximum is a shuffle reduction over its G / 8
// threads.  The scales of the tile go through shared memory, because
// consecutive scales in memory belong to consecutive rows.
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
constexpr int kQ4MaxGroups = kQ4Cols / 32;  // groups of a tile, G >= 32

struct Q4Tile {
  long long mat;
  int row0, col0;
};

__device__ __forceinline__ Q4Tile q4_tile(long long i, int row_tiles, int col_tiles) {
  Q4Tile t;
  t.col0 = static_cast<int>(i % col_tiles) * kQ4Cols;
  i /= col_tiles;
  t.row0 = static_cast<int>(i % row_tiles) * kQ4Rows;
  t.mat = i / row_tiles;
  return t;
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }

__global__ void __launch_bounds__(kQ4Warps * 32)
    q4_quantize_kernel(const uint16_t* __restrict__ W, uint8_t* __restrict__ codes, uint16_t* __restrict__ scales,
                       int rows, int cols, int group, int row_tiles, int col_tiles, long long tiles) {
  __shared__ uint16_t s_scale[kQ4MaxGroups][kQ4Rows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = group / 8;  // threads of a group
  const size_t pitch = q4_scale_pitch(rows);
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const Q4Tile t = q4_tile(i, row_tiles, col_tiles);
    const int col = t.col0 + lane * 8;
    const bool in = col < cols;  // cols is a multiple of the group: a group is wholly in or out
    uint4 v[kQ4RowsPerWarp];
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int row = t.row0 + j * kQ4Warps + warp;
      v[j] = make_uint4(0, 0, 0, 0);
      if (in && row < rows)
        v[j] = *reinterpret_cast<const uint4*>(W + (static_cast<size_t>(t.mat) * rows + row) * cols + col);
    }
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int rr = j * kQ4Warps + warp, row = t.row0 + rr;
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      // bf16 magnitudes order like their bits; Inf and NaN come out on top,
      // so a group that holds one gets a non-finite scale
      uint32_t top = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p) top = max(top, max(w[p] & 0x7FFFu, (w[p] >> 16) & 0x7FFFu));
      for (int off = 1; off < lanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      const __nv_bfloat16 sb = __float2bfloat16_rn(bf16_value(top) / 7.f);
      const float s = __bfloat162float(sb);
      uint32_t word = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = bf16_value((w[c >> 1] >> (16 * (c & 1))) & 0xFFFFu);
        int q = 0;
        if (s > 0.f && isfinite(s)) q = min(max(__float2int_rn(x / s), -8), 7);
        word |= static_cast<uint32_t>(q + 8) << (4 * (c >> 1) + 16 * (c & 1));
      }
      if (in && row < rows)
        *reinterpret_cast<uint32_t*>(codes + ((static_cast<size_t>(t.mat) * rows + row) * cols + col) / 2) = word;
      if (lane % lanes == 0) s_scale[lane / lanes][rr] = row < rows ? __bfloat16_as_ushort(sb) : 0;
    }
    __syncthreads();
    const int groups = cols / group, g0 = t.col0 / group;
    for (int e = threadIdx.x; e < (kQ4Cols / group) * kQ4Rows; e += blockDim.x) {
      const int g = e / kQ4Rows, rr = e % kQ4Rows;
      if (g0 + g < groups && static_cast<size_t>(t.row0 + rr) < pitch)
        scales[(static_cast<size_t>(t.mat) * groups + g0 + g) * pitch + t.row0 + rr] = s_scale[g][rr];
    }
    __syncthreads();  // the next tile rewrites s_scale
  }
}

__global__ void __launch_bounds__(kQ4Warps * 32)
    q4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                         uint16_t* __restrict__ W, int rows, int cols, int group, int row_tiles, int col_tiles,
                         long long tiles) {
  __shared__ uint16_t s_scale[kQ4MaxGroups][kQ4Rows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lanes = group / 8;
  const size_t pitch = q4_scale_pitch(rows);
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const Q4Tile t = q4_tile(i, row_tiles, col_tiles);
    const int col = t.col0 + lane * 8;
    const bool in = col < cols;
    uint32_t word[kQ4RowsPerWarp];
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int row = t.row0 + j * kQ4Warps + warp;
      word[j] = 0;
      if (in && row < rows)
        word[j] = *reinterpret_cast<const uint32_t*>(codes + ((static_cast<size_t>(t.mat) * rows + row) * cols + col) / 2);
    }
    const int groups = cols / group, g0 = t.col0 / group;
    for (int e = threadIdx.x; e < (kQ4Cols / group) * kQ4Rows; e += blockDim.x) {
      const int g = e / kQ4Rows, rr = e % kQ4Rows;
      if (g0 + g < groups && t.row0 + rr < rows)
        s_scale[g][rr] = scales[(static_cast<size_t>(t.mat) * groups + g0 + g) * pitch + t.row0 + rr];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQ4RowsPerWarp; ++j) {
      const int rr = j * kQ4Warps + warp, row = t.row0 + rr;
      if (!in || row >= rows) continue;
      const float s = bf16_value(s_scale[lane / lanes][rr]);
      uint32_t out[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t pair = q4_pair(word[j], p);
        // one rounding: 4-bit times 8-bit significands is exact in fp32
        const __nv_bfloat162 o = __floats2bfloat162_rn(s * bf16_value(pair & 0xFFFFu), s * bf16_value(pair >> 16));
        out[p] = *reinterpret_cast<const uint32_t*>(&o);
      }
      *reinterpret_cast<uint4*>(W + (static_cast<size_t>(t.mat) * rows + row) * cols + col) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
  }
}

// Blocks: every tile one, up to what a grid holds with room to spare.
unsigned q4_grid(long long tiles) { return static_cast<unsigned>(std::min<long long>(tiles, 1 << 20)); }

}  // namespace

cudaError_t launch_q4_quantize(const uint16_t* W, uint8_t* codes, uint16_t* scales, int mats, int rows, int cols,
                               int group, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_Q4, s);
  const int rt = ceil_div(static_cast<long long>(q4_scale_pitch(rows)), kQ4Rows), ct = ceil_div(cols, kQ4Cols);
  const long long tiles = static_cast<long long>(mats) * rt * ct;
  q4_quantize_kernel<<<q4_grid(tiles), kQ4Warps * 32, 0, s>>>(W, codes, scales, rows, cols, group, rt, ct, tiles);
  return cudaGetLastError();
}

cudaError_t launch_q4_dequantize(const uint8_t* codes, const uint16_t* scales, uint16_t* W, int mats, int rows,
                                 int cols, int group, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_Q4, s);
  const int rt = ceil_div(rows, kQ4Rows), ct = ceil_div(cols, kQ4Cols);
  const long long tiles = static_cast<long long>(mats) * rt * ct;
  q4_dequantize_kernel<<<q4_grid(tiles), kQ4Warps * 32, 0, s>>>(codes, scales, W, rows, cols, group, rt, ct, tiles);
  return cudaGetLastError();
}

}  // namespace moe
