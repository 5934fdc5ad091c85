// How evenly the router spreads tokens: counts, mean probabilities, the balance
// loss and the mean square of log(sum(exp(logits))), for each of B sequences of
// L = T / B tokens, and their gradient for the logits.
//
//   c_e = picks of expert e, P_e = mean_t p_te, both over the n tokens that count
//   loss  = E / (k n) sum_e c_e P_e,   zloss = mean_t lse_t^2
//   dz_te = p_te (a_e - sum_j a_j p_tj) + (2 h / n) lse_t p_te,  a_e = g E c_e / (k n^2)
//
// Both directions are bound by memory: the forward reads the logits and the
// picks, the backward the logits and the gradient to add to, and writes one.  A
// row lies on as few lanes as its 16-byte pieces need (two for 8 experts, 16 for
// 64), so that a warp has several rows and their chains of shuffles in flight,
// and the next rows are loaded while these are worked on.
//
// A sequence's sums are taken by as many blocks as its tokens give work to; each
// keeps the sums of its tokens in registers, in fp32, and a second launch adds the
// blocks' sums in a fixed order, with the roundings kept.  A sequence that one
// block takes is finished in the first launch.  (fp64 sums took longer than all
// the rest: the part has two such additions a clock and SM.)
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "route.cuh"
#include "trace.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kUnits = 152 * 3;  // blocks to spread the tokens over; fixed, so the sums' order is

// Blocks of a sequence: at least 32 tokens each, so that all blocks' sums fit in
// the E ceil(T / 32) words of the histogram regions of the workspace.
int seq_parts(int T, int B) {
  const int L = T / B;
  const long long each = std::max<long long>(32, ceil_div(T, kUnits));
  return static_cast<int>(std::max(1ll, L / each));
}

// How a row of E logits lies on lanes: LANES lanes (a power of two) of V values
// each, lane l holding experts V (l + LANES i) .. + V - 1 for i < N; V = 4 where
// rows are whole 16-byte pieces.  A warp takes 32 / LANES rows at one time.
template <int V_, int LANES_, int N_>
struct Lay {
  static constexpr int V = V_, LANES = LANES_, E = V_ * N_;  // E: values of a lane
  static __device__ __forceinline__ int expert(int l, int i) { return V * (l + LANES * (i / V)) + i % V; }
};
template <class Y>
__device__ __forceinline__ void load_values(const float* row, int E, int l, float (&v)[Y::E], float none) {
#pragma unroll
  for (int i = 0; i < Y::E; i += Y::V) {
    const int e = Y::expert(l, i);
    if constexpr (Y::V == 4) {
      const float4 w = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(none, none, none, none);
      v[i] = w.x;
      v[i + 1] = w.y;
      v[i + 2] = w.z;
      v[i + 3] = w.w;
    } else {
      v[i] = e < E ? row[e] : none;
    }
  }
}
template <class Y, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F f) {
#pragma unroll
  for (int off = Y::LANES / 2; off; off >>= 1) v = f(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
// p and lse of the row in v (in place); false where a logit is not finite.
template <class Y>
__device__ __forceinline__ bool softmax_values(float (&v)[Y::E], int E, int l, float& lse) {
  float m = -INFINITY, bad = 0.f;
#pragma unroll
  for (int i = 0; i < Y::E; ++i) {
    m = fmaxf(m, v[i]);
    if (Y::expert(l, i) < E) bad = fmaf(0.f, v[i], bad);  // NaN where v is not finite
  }
  m = lanes_reduce<Y>(m, [](float a, float b) { return fmaxf(a, b); });
  float s = bad;
#pragma unroll
  for (int i = 0; i < Y::E; ++i) {
    v[i] = expf(v[i] - m);  // 0 beyond E
    s += v[i];
  }
  s = lanes_reduce<Y>(s, [](float a, float b) { return a + b; });
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < Y::E; ++i) v[i] *= inv;
  lse = m + logf(s);
  return s == s;
}

// Sum with what its roundings left (the exact error of each addition kept).
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = hi + v, b = t - hi;
    lo += (hi - (t - b)) + (v - b);
    hi = t;
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

struct BalanceOut {
  int32_t* counts;
  float* mean_p;
  float* loss;
  float* zloss;
};

// Sequence b from its sums: count and sum of p of expert e on thread e.  Every
// thread of the block calls it; red has 8 places.
__device__ __forceinline__ void finish_sequence(const BalanceOut& o, int b, int E, int k, int count, float psum, float zsum,
                                                int n, float* red) {
  const int e = threadIdx.x;
  const float inv = n > 0 ? 1.f / n : 0.f;
  float term = 0.f;
  if (e < E) {
    const float P = psum * inv;
    o.counts[static_cast<size_t>(b) * E + e] = count;
    o.mean_p[static_cast<size_t>(b) * E + e] = P;
    term = (count * inv) * P;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) term += __shfl_xor_sync(kFull, term, off);
  if ((e & 31) == 0 && e < 256) red[e >> 5] = term;  // the first 256 threads hold all experts
  __syncthreads();
  if (e == 0) {
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += red[i];
    o.loss[b] = s * (static_cast<float>(E) / k);
    o.zloss[b] = zsum * inv;
  }
}

template <class Y>
__global__ void __launch_bounds__(kThreads, 3)
    balance_sums_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                        const uint8_t* __restrict__ mask, int L, int B, int parts, int E, int k, int32_t* __restrict__ counts,
                        float* __restrict__ psums, float2* __restrict__ zn, BalanceOut out, int* err) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int ROWS = 32 / Y::LANES, WARPS = kThreads / 32;
  __shared__ int hist[256];
  __shared__ float ps[WARPS][256];
  __shared__ float red[8], zw[WARPS];
  __shared__ int nw[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / Y::LANES, l = lane % Y::LANES;
  const int per = (L + parts - 1) / parts;
  for (int u = blockIdx.x; u < B * parts; u += gridDim.x) {
    const int b = u / parts, c = u - b * parts;
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    const int t0 = b * L + min(L, c * per), t1 = b * L + min(L, (c + 1) * per);
    auto live = [&](int t) { return t < t1 && (!mask || mask[t]); };
    int t = t0 + warp * ROWS + sub;
    bool on = live(t);
    float v[Y::E];
    load_values<Y>(logits + static_cast<size_t>(t) * E, on ? E : 0, l, v, -INFINITY);
    for (int i = threadIdx.x; i < (t1 - t0) * k; i += kThreads) {
      const int ti = t0 + i / k;
      if (mask && !mask[ti]) continue;  // whatever it holds
      const int e = topk_idx[static_cast<size_t>(t0) * k + i];
      if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
        atomicAdd(&hist[e], 1);
      else
        record_error(err, MOE_ERR_ARG, ti);
    }
    float p[Y::E] = {};
    float z = 0.f;
    int n = 0;
    for (int tw = t0 + warp * ROWS; tw < t1; tw += WARPS * ROWS) {  // the same rounds for all lanes of the warp
      // the next row is on its way while this one is worked on
      const int tn = t + WARPS * ROWS;
      const bool on_n = live(tn);
      float w[Y::E];
      load_values<Y>(logits + static_cast<size_t>(tn) * E, on_n ? E : 0, l, w, -INFINITY);
      float lse;
      const bool ok = softmax_values<Y>(v, on ? E : 0, l, lse);
      if (on) {
        ++n;
        if (ok) {
#pragma unroll
          for (int i = 0; i < Y::E; ++i) p[i] += v[i];
          z = fmaf(lse, lse, z);
        } else if (l == 0) {
          record_error(err, MOE_ERR_NONFINITE_CODE, t);
        }
      }
#pragma unroll
      for (int i = 0; i < Y::E; ++i) v[i] = w[i];
      t = tn;
      on = on_n;
    }
    // the rows of a warp, then the warps
#pragma unroll
    for (int off = Y::LANES; off < 32; off <<= 1) {
#pragma unroll
      for (int i = 0; i < Y::E; ++i) p[i] += __shfl_xor_sync(kFull, p[i], off);
      z += __shfl_xor_sync(kFull, z, off);
      n += __shfl_xor_sync(kFull, n, off);
    }
    if (sub == 0)
#pragma unroll
      for (int i = 0; i < Y::E; ++i)
        if (Y::expert(l, i) < E) ps[warp][Y::expert(l, i)] = p[i];
    if (lane == 0) {
      zw[warp] = z;
      nw[warp] = n;
    }
    __syncthreads();
    const int e = threadIdx.x;
    float psum = 0.f, zsum = 0.f;
    int total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (e < E) psum += ps[w][e];
      zsum += zw[w];
      total += nw[w];
    }
    if (parts == 1) {
      finish_sequence(out, b, E, k, e < E ? hist[e] : 0, psum, zsum, total, red);
    } else {
      if (e < E) {
        counts[static_cast<size_t>(u) * E + e] = hist[e];
        psums[static_cast<size_t>(u) * E + e] = psum;
      }
      if (e == 0) zn[u] = make_float2(zsum, static_cast<float>(total));
    }
    __syncthreads();
  }
}

// One block a sequence: a thread takes V experts (a 16-byte piece where rows are
// whole ones) of every group-th part; then the groups of a warp, and the warps, are
// added in a fixed order.
constexpr int kJoin = 512;
template <int V>
__global__ void __launch_bounds__(kJoin)
    balance_join_kernel(const int32_t* __restrict__ counts, const float* __restrict__ psums, const float2* __restrict__ zn,
                        int B, int parts, int E, int k, BalanceOut out) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int WARPS = kJoin / 32;
  __shared__ float sp[WARPS][256];
  __shared__ int sc[WARPS][256];
  __shared__ float red[8], zred[WARPS];
  __shared__ int nred[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int shift = 0;  // of the groups' width, a power of two of at least E / V
  while ((V << shift) < E) ++shift;
  const int groups = kJoin >> shift, g = tid >> shift, e = V * (tid & ((1 << shift) - 1));
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    Sum2 s[V], z;
    int c[V] = {}, n = 0;
    const size_t at = static_cast<size_t>(b) * parts;
    if (e < E) {
#pragma unroll 4
      for (int i = g; i < parts; i += groups) {
        const size_t from = (at + i) * E + e;
        if constexpr (V == 4) {
          const float4 p = *reinterpret_cast<const float4*>(psums + from);
          const int4 q = *reinterpret_cast<const int4*>(counts + from);
          s[0].add(p.x);
          s[1].add(p.y);
          s[2].add(p.z);
          s[3].add(p.w);
          c[0] += q.x;
          c[1] += q.y;
          c[2] += q.z;
          c[3] += q.w;
        } else {
          s[0].add(psums[from]);
          c[0] += counts[from];
        }
      }
    }
    for (int i = tid; i < parts; i += kJoin) {
      const float2 v = zn[at + i];
      z.add(v.x);
      n += static_cast<int>(v.y);  // tokens of a part: far below 2^24
    }
    float zs = z.value();
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      zs += __shfl_xor_sync(kFull, zs, off);
      n += __shfl_xor_sync(kFull, n, off);
    }
    if (lane == 0) {
      zred[warp] = zs;
      nred[warp] = n;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = s[j].value();
      int q = c[j];
      for (int off = 1 << shift; off < 32; off <<= 1) {
        v += __shfl_xor_sync(kFull, v, off);
        q += __shfl_xor_sync(kFull, q, off);
      }
      // groups wider than a warp: the warps of one group hold different experts
      if (e < E && (shift >= 5 || (lane >> shift) == 0)) {
        sp[shift > 5 ? g : warp][e + j] = v;
        sc[shift > 5 ? g : warp][e + j] = q;
      }
    }
    __syncthreads();
    float ps = 0.f;
    int count = 0;
    zs = 0.f;
    n = 0;
    const int rows = shift > 5 ? groups : WARPS;
    for (int i = 0; i < rows; ++i) {
      if (tid < E) {
        ps += sp[i][tid];
        count += sc[i][tid];
      }
    }
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      zs += zred[i];
      n += nred[i];
    }
    finish_sequence(out, b, E, k, count, ps, zs, n, red);
    __syncthreads();
  }
}

// dlogits = add + gradient; add may be dlogits itself or null.
template <class Y>
__global__ void __launch_bounds__(kThreads, 2)
    balance_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ counts, const uint8_t* __restrict__ mask,
                       const float* __restrict__ dloss, const float* __restrict__ dz, int T, int L, int E, int k,
                       const float* add, float* dlogits) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int ROWS = 32 / Y::LANES;
  const int lane = threadIdx.x & 31;
  const int sub = lane / Y::LANES, l = lane % Y::LANES;
  const int rounds = (T + ROWS - 1) / ROWS;
  const int nwarps = gridDim.x * (kThreads / 32), w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  // consecutive rows to a warp: the sequence rarely changes
  const int per = (rounds + nwarps - 1) / nwarps;
  const int r0 = min(rounds, w * per), r1 = min(rounds, r0 + per);
  int cur = -1;
  float a[Y::E] = {}, hz = 0.f;
  auto read = [&](int r, float (&v)[Y::E], float (&in)[Y::E], bool& on) {
    const int t = r * ROWS + sub;
    const bool here = r < r1 && t < T;
    on = here && (!mask || mask[t]);
    load_values<Y>(logits + static_cast<size_t>(t) * E, on ? E : 0, l, v, -INFINITY);
    load_values<Y>(add + static_cast<size_t>(t) * E, here && add ? E : 0, l, in, 0.f);
  };
  float v[Y::E], in[Y::E];
  bool on;
  read(r0, v, in, on);
  for (int r = r0; r < r1; ++r) {
    float vn[Y::E], inn[Y::E];
    bool on_n;
    read(r + 1, vn, inn, on_n);
    const int t = r * ROWS + sub, b = min(t, T - 1) / L;
    if (__any_sync(kFull, b != cur)) {
      cur = b;
      int c[Y::E], sum = 0;
#pragma unroll
      for (int i = 0; i < Y::E; ++i) {
        const int e = Y::expert(l, i);
        c[i] = e < E ? counts[static_cast<size_t>(b) * E + e] : 0;
        sum += c[i];
      }
#pragma unroll
      for (int off = Y::LANES / 2; off; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
      const float n = static_cast<float>(sum / k);  // every token that counts has k picks
      const float f = n > 0.f ? dloss[b] * (static_cast<float>(E) / k) / n / n : 0.f;
#pragma unroll
      for (int i = 0; i < Y::E; ++i) a[i] = f * c[i];
      hz = n > 0.f ? 2.f * dz[b] / n : 0.f;
    }
    float lse;
    const bool ok = softmax_values<Y>(v, on ? E : 0, l, lse);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < Y::E; ++i) dot = fmaf(a[i], v[i], dot);
    dot = lanes_reduce<Y>(dot, [](float x, float y) { return x + y; });
    if (on && ok) {
      const float shift = hz * lse - dot;
#pragma unroll
      for (int i = 0; i < Y::E; ++i) in[i] = fmaf(v[i], a[i] + shift, in[i]);
    }
    if (t < T) {
      float* to = dlogits + static_cast<size_t>(t) * E;
#pragma unroll
      for (int i = 0; i < Y::E; i += Y::V) {
        const int e = Y::expert(l, i);
        if (e < E) {
          if constexpr (Y::V == 4)
            *reinterpret_cast<float4*>(to + e) = make_float4(in[i], in[i + 1], in[i + 2], in[i + 3]);
          else
            to[e] = in[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < Y::E; ++i) {
      v[i] = vn[i];
      in[i] = inn[i];
    }
    on = on_n;
  }
}

template <typename F>
cudaError_t with_layout(int E, F f) {
  if (E % 4 == 0) {  // whole 16-byte pieces
    if (E <= 8) return f(Lay<4, 2, 1>{});
    if (E <= 16) return f(Lay<4, 4, 1>{});
    if (E <= 32) return f(Lay<4, 8, 1>{});
    if (E <= 64) return f(Lay<4, 16, 1>{});
    if (E <= 128) return f(Lay<4, 32, 1>{});
    return f(Lay<4, 32, 2>{});
  }
  if (E <= 8) return f(Lay<1, 8, 1>{});
  if (E <= 32) return f(Lay<1, 32, 1>{});
  if (E <= 128) return f(Lay<1, 32, 4>{});
  return f(Lay<1, 32, 8>{});
}

}  // namespace

cudaError_t launch_balance(const float* logits, const int32_t* topk_idx, const uint8_t* mask, int T, int B, int E, int k,
                           int32_t* counts, float* mean_p, float* loss, float* zloss, int32_t* part_counts, float* part_p,
                           float* part_zn, int* err, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE, s);
  const int parts = seq_parts(T, B);
  const BalanceOut out{counts, mean_p, loss, zloss};
  const int units = static_cast<int>(std::min<long long>(static_cast<long long>(B) * parts, num_sms() * 3));
  float2* zn = reinterpret_cast<float2*>(part_zn);
  cudaError_t e = with_layout(E, [&](auto y) {
    return launch_pdl(balance_sums_kernel<decltype(y)>, dim3(units), dim3(kThreads), 0, s, logits, topk_idx, mask, T / B, B,
                      parts, E, k, part_counts, part_p, zn, out, err);
  });
  if (e == cudaSuccess && parts > 1)
    e = launch_pdl(E % 4 ? balance_join_kernel<1> : balance_join_kernel<4>, dim3(std::min(B, 65535)), dim3(kJoin), 0, s,
                   part_counts, part_p, zn, B, parts, E, k, out);
  return e;
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* counts, const uint8_t* mask, const float* dloss,
                               const float* dz, int T, int B, int E, int k, const float* add, float* dlogits,
                               cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE_BWD, s);
  return with_layout(E, [&](auto y) {
    const long long warps = ceil_div(T, 32 / decltype(y)::LANES);
    const int blocks = static_cast<int>(std::min<long long>(ceil_div(warps, kThreads / 32), num_sms() * 2));
    return launch_pdl(balance_bwd_kernel<decltype(y)>, dim3(blocks), dim3(kThreads), 0, s, logits, counts, mask, dloss, dz, T,
                      T / B, E, k, add, dlogits);
  });
}

}  // namespace moe
