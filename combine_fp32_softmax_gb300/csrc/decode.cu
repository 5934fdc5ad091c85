// The layer for a few tokens (T <= 64) and its linear form, y = x W^T, with
// bf16 or 4-bit weights.
//
// One warp computes one output element: a dot product of a weight row with
// an activation row, 8 columns a lane and step, in fp32.  The router is the
// library's (launch_route).
//   hidden  h[r, i] = w_r * silu(x_t . W1_e[i]) * (x_t . W3_e[i])   fp32
//   out     y[t, c] = sum over the token's rows r, slots first, of h[r] . W2_e[c]
#include <cuda_runtime.h>

#include "decode.h"
#include "kernels.h"
#include "q4.cuh"
#include "trace.h"

namespace moe {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Eight consecutive weights of row `row` of matrix `mat` ([rows, K] each).
template <bool Q4>
__device__ __forceinline__ void load8(const DecodeWeight& W, size_t mat, int row, int rows, int K, int group, int col,
                                      float (&v)[8]) {
  const size_t at = (mat * rows + row) * K + col;
  if constexpr (Q4) {
    const uint32_t word = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(W.w) + at / 2);
    const float s = bf16_lo(W.scales[(mat * (K / group) + col / group) * q4_scale_pitch(rows) + row]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = q4_pair(word, i);
      v[2 * i] = s * bf16_lo(p);
      v[2 * i + 1] = s * bf16_hi(p);
    }
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W.w) + at);
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(p[i]);
      v[2 * i + 1] = bf16_hi(p[i]);
    }
  }
}
__device__ __forceinline__ void load8(const uint16_t* x, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(x);
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(p[i]);
    v[2 * i + 1] = bf16_hi(p[i]);
  }
}
__device__ __forceinline__ void load8(const float* x, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(x), b = *reinterpret_cast<const float4*>(x + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Dot product of a weight row with `x`; every lane gets the sum.
template <bool Q4, typename X>
__device__ __forceinline__ float dot_row(const DecodeWeight& W, size_t mat, int row, int rows, int K, int group,
                                         const X* x) {
  float acc = 0.f;
  for (int col = (threadIdx.x & 31) * 8; col < K; col += 256) {
    float w[8], v[8];
    load8<Q4>(W, mat, row, rows, K, group, col, w);
    load8(x + col, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(w[i], v[i], acc);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
  return acc;
}

__device__ __forceinline__ void store_y(void* y, int y_type, size_t at, float v) {
  if (y_type == MOE_Y_BF16)
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(y)[at] = v;
}

template <bool Q4>
__global__ void __launch_bounds__(kWarps * 32) decode_hidden_kernel(DecodeArgs a, float* __restrict__ h) {
  const moe_cfg& c = a.c;
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5), r = blockIdx.y, R = c.T * c.k;
  if (i >= c.d_ff) return;
  const int t = r < R ? r / c.k : (r - R) % c.T;
  const int e = r < R ? a.topk_idx[r] : c.E + (r - R) / c.T;
  const float w = r < R ? a.topk_w[r] : 1.f;
  const uint16_t* x = a.x + static_cast<size_t>(t) * c.d_model;
  const float g = dot_row<Q4>(a.W1, e, i, c.d_ff, c.d_model, a.group, x);
  const float u = dot_row<Q4>(a.W3, e, i, c.d_ff, c.d_model, a.group, x);
  if ((threadIdx.x & 31) == 0) h[static_cast<size_t>(r) * c.d_ff + i] = w * (g / (1.f + expf(-g)) * u);
}

template <bool Q4>
__global__ void __launch_bounds__(kWarps * 32) decode_out_kernel(DecodeArgs a, const float* __restrict__ h) {
  const moe_cfg& c = a.c;
  const int col = blockIdx.x * kWarps + (threadIdx.x >> 5), t = blockIdx.y, R = c.T * c.k;
  if (col >= c.d_model) return;
  float y = 0.f;
  for (int j = 0; j < c.k + c.n_shared; ++j) {
    const int r = j < c.k ? t * c.k + j : R + (j - c.k) * c.T + t;
    const int e = j < c.k ? a.topk_idx[r] : c.E + j - c.k;
    y += dot_row<Q4>(a.W2, e, col, c.d_model, c.d_ff, a.group, h + static_cast<size_t>(r) * c.d_ff);
  }
  if ((threadIdx.x & 31) == 0) store_y(a.y, a.y_type, static_cast<size_t>(t) * c.d_model + col, y);
}

template <bool Q4>
__global__ void __launch_bounds__(kWarps * 32) linear_kernel(LinearArgs a) {
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5), t = blockIdx.y;
  if (i >= a.n) return;
  const float y = dot_row<Q4>(a.W, 0, i, a.n, a.K, a.group, a.x + static_cast<size_t>(t) * a.K);
  if ((threadIdx.x & 31) == 0) store_y(a.y, a.y_type, static_cast<size_t>(t) * a.n + i, y);
}

}  // namespace

size_t decode_workspace_bytes(const moe_cfg& c) {
  const size_t Rs = static_cast<size_t>(c.T) * (c.k + c.n_shared);
  return kErrRegionBytes + align_up(sizeof(float) * Rs * c.d_ff, 256);
}
size_t linear_workspace_bytes(int, int, int) { return kErrRegionBytes; }

int decode_ws_init(void* ws, cudaStream_t s) {
  return cudaMemsetAsync(ws, 0, kErrRegionBytes, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_decode(const DecodeArgs& a, cudaStream_t s) {
  const moe_cfg& c = a.c;
  int* err = static_cast<int*>(a.ws);
  float* h = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + kErrRegionBytes);
  const int nb = ceil_div(c.T, kRouteTokensPerBlock);
  if (launch_route(a.logits, c.T, c.E, c.k, c.renorm, a.topk_idx, a.topk_w, nullptr, nb, err, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  TraceScope trace_scope(MOE_K_DECODE, s);
  const dim3 gh(ceil_div(c.d_ff, kWarps), c.T * (c.k + c.n_shared)), go(ceil_div(c.d_model, kWarps), c.T);
  if (a.group) {
    decode_hidden_kernel<true><<<gh, kWarps * 32, 0, s>>>(a, h);
    decode_out_kernel<true><<<go, kWarps * 32, 0, s>>>(a, h);
  } else {
    decode_hidden_kernel<false><<<gh, kWarps * 32, 0, s>>>(a, h);
    decode_out_kernel<false><<<go, kWarps * 32, 0, s>>>(a, h);
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_linear(const LinearArgs& a, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_LINEAR, s);
  const dim3 grid(ceil_div(a.n, kWarps), a.T);
  if (a.group)
    linear_kernel<true><<<grid, kWarps * 32, 0, s>>>(a);
  else
    linear_kernel<false><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
