// How evenly the router spreads tokens: counts, mean probabilities, the balance
// loss and the mean square of log(sum(exp(logits))), for each of B sequences of
// L = T / B tokens, and their gradient for the logits.
//
//   c_e = picks of expert e, P_e = mean_t p_te, both over the n tokens that count
//   loss  = E / (k n) sum_e c_e P_e,   zloss = mean_t lse_t^2
//   dz_te = p_te (a_e - sum_j a_j p_tj) + (2 h / n) lse_t p_te,  a_e = g E c_e / (k n^2)
//
// One warp takes a token, as in the router, with the router's own softmax
// (RowSoftmax), so p has its bits.  Both directions are bound by memory: the
// forward reads the logits and the picks, the backward the logits and the
// gradient to add to, and writes one.
//
// A sequence's sums are taken by as many blocks as its tokens give work to; each
// keeps the sums of its tokens in registers (one expert a lane), and a second
// launch adds the blocks' sums, in fp64 and in a fixed order.  A sequence that
// one block takes is finished in the first launch.
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "route.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kUnits = 152 * 4;  // blocks to spread the tokens over; fixed, so the sums' order is

// Blocks of a sequence: at least 32 tokens each, so that all blocks' sums fit in
// the E ceil(T / 32) words of the histogram regions of the workspace.
int seq_parts(int T, int B) {
  const int L = T / B;
  const long long each = std::max<long long>(32, ceil_div(T, kUnits));
  return static_cast<int>(std::max(1ll, L / each));
}

struct BalanceOut {
  int32_t* counts;
  float* mean_p;
  float* loss;
  float* zloss;
};

// Sequence b from its sums: count and sum of p of expert e on thread e.  Every
// thread of the block calls it.
__device__ __forceinline__ void finish_sequence(const BalanceOut& o, int b, int E, int k, int count, double psum, double zsum,
                                                int n, double* red) {
  const int e = threadIdx.x;
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double term = 0.0;
  if (e < E) {
    o.counts[static_cast<size_t>(b) * E + e] = count;
    o.mean_p[static_cast<size_t>(b) * E + e] = static_cast<float>(psum * inv);
    term = count * (psum * inv);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) term += __shfl_xor_sync(kFull, term, off);
  if ((e & 31) == 0 && e < 32 * kWarps) red[e >> 5] = term;  // the first 256 threads hold all experts
  __syncthreads();
  if (e == 0) {
    double s = 0.0;
    for (int i = 0; i < kWarps; ++i) s += red[i];
    o.loss[b] = static_cast<float>(s * E / k * inv);
    o.zloss[b] = static_cast<float>(zsum * inv);
  }
}

template <int EPL>
__global__ void __launch_bounds__(32 * kWarps)
    balance_sums_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                        const uint8_t* __restrict__ mask, int L, int B, int parts, int E, int k, int32_t* __restrict__ counts,
                        float* __restrict__ psums, float2* __restrict__ zn, BalanceOut out, int* err) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int hist[256];
  __shared__ float ps[kWarps][256];
  __shared__ double red[kWarps];
  __shared__ float zw[kWarps];
  __shared__ int nw[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (L + parts - 1) / parts;
  for (int u = blockIdx.x; u < B * parts; u += gridDim.x) {
    const int b = u / parts, c = u - b * parts;
    hist[threadIdx.x] = 0;
    __syncthreads();
    const int t1 = b * L + min(L, (c + 1) * per);
    float p[EPL] = {};
    float z = 0.f;
    int n = 0;
    for (int t = b * L + c * per + warp; t < t1; t += kWarps) {
      if (mask && !mask[t]) continue;  // whatever it holds
      ++n;
      RowSoftmax<EPL> r;
      if (lane < k) {
        const int e = topk_idx[static_cast<size_t>(t) * k + lane];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
          atomicAdd(&hist[e], 1);
        else
          record_error(err, MOE_ERR_ARG, t);
      }
      if (!row_softmax<EPL>(logits + static_cast<size_t>(t) * E, E, lane, r)) {
        if (lane == 0) record_error(err, MOE_ERR_NONFINITE_CODE, t);
        continue;
      }
      const float inv = 1.f / r.s;
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[i] += r.ex[i] * inv;
      const float lse = r.m + logf(r.s);
      z = fmaf(lse, lse, z);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) ps[warp][lane + 32 * i] = p[i];
    if (lane == 0) {
      zw[warp] = z;
      nw[warp] = n;
    }
    __syncthreads();
    const int e = threadIdx.x;
    double psum = 0.0, zsum = 0.0;
    int total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (e < E) psum += ps[w][e];
      zsum += zw[w];
      total += nw[w];
    }
    if (parts == 1) {
      finish_sequence(out, b, E, k, hist[e], psum, zsum, total, red);
    } else {
      if (e < E) {
        counts[static_cast<size_t>(u) * E + e] = hist[e];
        psums[static_cast<size_t>(u) * E + e] = static_cast<float>(psum);
      }
      if (e == 0) zn[u] = make_float2(static_cast<float>(zsum), static_cast<float>(total));
    }
    __syncthreads();
  }
}

// One block a sequence: the experts of a part side by side, groups of threads on
// every (1024 / width)-th part, then the groups in their order.
__global__ void __launch_bounds__(1024)
    balance_join_kernel(const int32_t* __restrict__ counts, const float* __restrict__ psums, const float2* __restrict__ zn,
                        int B, int parts, int E, int k, BalanceOut out) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ double sp[1024];
  __shared__ int sc[1024];
  __shared__ double red[kWarps], zred[32];
  __shared__ int nred[32];
  const int width = E <= 32 ? 32 : E <= 64 ? 64 : E <= 128 ? 128 : 256;
  const int groups = 1024 / width, g = threadIdx.x / width, e = threadIdx.x - g * width;
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    double s = 0.0, z = 0.0;
    int c = 0, n = 0;
    const size_t at = static_cast<size_t>(b) * parts;
    if (e < E) {
#pragma unroll 4
      for (int i = g; i < parts; i += groups) {
        s += psums[(at + i) * E + e];
        c += counts[(at + i) * E + e];
      }
    }
    for (int i = threadIdx.x; i < parts; i += 1024) {
      const float2 v = zn[at + i];
      z += v.x;
      n += static_cast<int>(v.y);  // tokens of a part: far below 2^24
    }
    sp[threadIdx.x] = s;
    sc[threadIdx.x] = c;
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      z += __shfl_xor_sync(kFull, z, off);
      n += __shfl_xor_sync(kFull, n, off);
    }
    if ((threadIdx.x & 31) == 0) {
      zred[threadIdx.x >> 5] = z;
      nred[threadIdx.x >> 5] = n;
    }
    __syncthreads();
    z = 0.0;
    n = 0;
    for (int i = 0; i < 32; ++i) {
      z += zred[i];
      n += nred[i];
    }
    if (threadIdx.x < 256) {
      s = 0.0;
      c = 0;
      if (threadIdx.x < E)
        for (int i = 0; i < groups; ++i) {
          s += sp[i * width + threadIdx.x];
          c += sc[i * width + threadIdx.x];
        }
    }
    finish_sequence(out, b, E, k, c, s, z, n, red);
    __syncthreads();
  }
}

// dlogits = add + gradient; add may be dlogits itself or null.
template <int EPL>
__global__ void __launch_bounds__(32 * kWarps)
    balance_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ counts, const uint8_t* __restrict__ mask,
                       const float* __restrict__ dloss, const float* __restrict__ dz, int T, int L, int E, int k,
                       const float* add, float* dlogits) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int nwarps = gridDim.x * kWarps;
  const int per = (T + nwarps - 1) / nwarps;  // consecutive tokens: few change of sequence
  const int t0 = min(T, (blockIdx.x * kWarps + (threadIdx.x >> 5)) * per), t1 = min(T, t0 + per);
  int cur = -1;
  float a[EPL], hz = 0.f;
  for (int t = t0; t < t1; ++t) {
    const size_t at = static_cast<size_t>(t) * E;
    float in[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      in[i] = add && e < E ? add[at + e] : 0.f;
    }
    RowSoftmax<EPL> r;
    const bool live = !mask || mask[t];
    if (live && row_softmax<EPL>(logits + at, E, lane, r)) {
      const int b = t / L;
      if (b != cur) {
        cur = b;
        int c[EPL], sum = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane + 32 * i;
          c[i] = e < E ? counts[static_cast<size_t>(b) * E + e] : 0;
          sum += c[i];
        }
        const float n = static_cast<float>(__reduce_add_sync(kFull, sum) / k);  // every token that counts has k picks
        const float f = dloss[b] * (static_cast<float>(E) / k) / n / n;
#pragma unroll
        for (int i = 0; i < EPL; ++i) a[i] = f * c[i];
        hz = 2.f * dz[b] / n;
      }
      const float inv = 1.f / r.s;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) dot = fmaf(a[i], r.ex[i] * inv, dot);
#pragma unroll
      for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(kFull, dot, off);
      const float shift = hz * (r.m + logf(r.s)) - dot;
#pragma unroll
      for (int i = 0; i < EPL; ++i) in[i] = fmaf(r.ex[i] * inv, a[i] + shift, in[i]);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E) dlogits[at + e] = in[i];
    }
  }
}

template <typename F>
cudaError_t with_epl(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

}  // namespace

cudaError_t launch_balance(const float* logits, const int32_t* topk_idx, const uint8_t* mask, int T, int B, int E, int k,
                           int32_t* counts, float* mean_p, float* loss, float* zloss, int32_t* part_counts, float* part_p,
                           float* part_zn, int* err, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE, s);
  const int parts = seq_parts(T, B);
  const BalanceOut out{counts, mean_p, loss, zloss};
  const int units = static_cast<int>(std::min<long long>(static_cast<long long>(B) * parts, num_sms() * 8));
  float2* zn = reinterpret_cast<float2*>(part_zn);
  cudaError_t e = with_epl(E, [&](auto epl) {
    return launch_pdl(balance_sums_kernel<epl.value>, dim3(units), dim3(32 * kWarps), 0, s, logits, topk_idx, mask, T / B, B,
                      parts, E, k, part_counts, part_p, zn, out, err);
  });
  if (e == cudaSuccess && parts > 1)
    e = launch_pdl(balance_join_kernel, dim3(std::min(B, 65535)), dim3(1024), 0, s, part_counts, part_p, zn, B, parts, E, k,
                   out);
  return e;
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* counts, const uint8_t* mask, const float* dloss,
                               const float* dz, int T, int B, int E, int k, const float* add, float* dlogits,
                               cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE_BWD, s);
  const int blocks = std::min(ceil_div(T, kWarps), num_sms() * 8);
  return with_epl(E, [&](auto epl) {
    return launch_pdl(balance_bwd_kernel<epl.value>, dim3(blocks), dim3(32 * kWarps), 0, s, logits, counts, mask, dloss, dz, T,
                      T / B, E, k, add, dlogits);
  });
}

}  // namespace moe
