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
// row lies on few lanes, two 16-byte pieces each (one lane for 8 experts, eight for
// 64): a warp has several rows at one time, which share the instructions of its
// shuffles, logarithm and addresses (with one piece a lane these were most of 85
// instructions a token at 64 experts), and the next rows are loaded meanwhile.
//
// A sequence's sums are taken by as many blocks as its tokens give work to; each
// keeps the sums of its tokens in registers, in fp32, and the last of them to end
// (a second launch where there are more sequences than counters) adds the blocks'
// sums in a fixed order, with the roundings kept.  (fp64 sums took longer than all
// the rest: the part has two such additions a clock and SM.)
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "route.cuh"
#include "trace.h"

namespace moe {
namespace {

// Threads of a block of the sums and of the backward.  Blocks to spread the tokens
// over: two a SM; fixed, so the sums' order is.  (131,072 tokens of 64 experts, both
// directions: 31 us with 2, 35 with 3 and 40 with 4 blocks of 512 threads a SM, 47
// with 6 of 256: each block's own sums and their join cost more than the rows gain.)
constexpr int kThreads = 512, kBwdThreads = 256;
constexpr int kUnits = 152 * 2;

// Blocks of a sequence: at least 32 tokens each, so that all blocks' sums fit in
// the E ceil(T / 32) words of the histogram regions of the workspace, and below 8192
// (4096 as a rule), so that fp32 sums stay short.
int seq_parts(int T, int B) {
  const int L = T / B;
  const long long each = std::clamp<long long>(ceil_div(T, kUnits), 32, 4096);
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
// The row's values, `none` beyond E; zeros where the row is not wanted.
template <class Y>
__device__ __forceinline__ void load_values(const float* row, bool on, int E, int l, float (&v)[Y::E], float none) {
  none = on ? none : 0.f;
#pragma unroll
  for (int i = 0; i < Y::E; i += Y::V) {
    const int e = Y::expert(l, i);
    if constexpr (Y::V == 4) {
      const float4 w = on && e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(none, none, none, none);
      v[i] = w.x;
      v[i + 1] = w.y;
      v[i + 2] = w.z;
      v[i + 3] = w.w;
    } else {
      v[i] = on && e < E ? row[e] : none;
    }
  }
}
template <class Y, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F f) {
#pragma unroll
  for (int off = Y::LANES / 2; off; off >>= 1) v = f(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
// exp(v - max) of the row in v, in place, 1 / their sum and lse; false where a
// logit is not finite.  The instructions are most of a token's time here, so exp and
// log are the short forms.  In units of 2^-22 of itself p is off by |z - max| + 1 for its
// exponential (with the rounding of z - max), in the sum by log E + 1 (|z_j - max| weighted
// by p_j is at most log E) and 4 for its up to 16 additions, by 1 for the quotient and less
// for the product: |z - max| 2^-22 + 2^-18 for up to 256 experts.
template <class Y>
__device__ __forceinline__ bool softmax_values(float (&v)[Y::E], int E, int l, float& inv, float& lse) {
  float m = v[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < Y::E; ++i) {
    if (i) m = fmaxf(m, v[i]);
    if (Y::expert(l, i) < E) bad = fmaf(0.f, v[i], bad);  // NaN where v is not finite
  }
  m = lanes_reduce<Y>(m, [](float a, float b) { return fmaxf(a, b); });
  float s = bad;
#pragma unroll
  for (int i = 0; i < Y::E; ++i) {
    v[i] = exp_short(v[i] - m);  // 0 beyond E
    s += v[i];
  }
  s = lanes_reduce<Y>(s, [](float a, float b) { return a + b; });
  inv = __fdividef(1.f, s);
  lse = m + __logf(s);
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

// Sums of sequence b from those of its parts, by one block: a thread takes V experts
// (a 16-byte piece where rows are whole ones) of every group-th part; then the
// groups of a warp, and the warps, are added in a fixed order.
struct JoinShared {
  float sp[kThreads / 32][256];
  int sc[kThreads / 32][256];
  float red[8], z[kThreads / 32];
  int n[kThreads / 32];
};
template <int V>
__device__ __forceinline__ void join_sequence(const int32_t* counts, const float* psums, const float2* zn, int b, int parts,
                                              int E, int k, const BalanceOut& out, JoinShared& sh) {
  constexpr int WARPS = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int shift = 0;  // of the groups' width, a power of two of at least E / V
  while ((V << shift) < E) ++shift;
  const int groups = kThreads >> shift, g = tid >> shift, e = V * (tid & ((1 << shift) - 1));
  Sum2 s[V], z;
  int c[V] = {}, n = 0;
  const size_t at = static_cast<size_t>(b) * parts;
  // the parts were written by other blocks of this launch: read past L1
  if (e < E) {
#pragma unroll 4
    for (int i = g; i < parts; i += groups) {
      const size_t from = (at + i) * E + e;
      if constexpr (V == 4) {
        const float4 p = __ldcg(reinterpret_cast<const float4*>(psums + from));
        const int4 q = __ldcg(reinterpret_cast<const int4*>(counts + from));
        s[0].add(p.x);
        s[1].add(p.y);
        s[2].add(p.z);
        s[3].add(p.w);
        c[0] += q.x;
        c[1] += q.y;
        c[2] += q.z;
        c[3] += q.w;
      } else {
        s[0].add(__ldcg(psums + from));
        c[0] += __ldcg(counts + from);
      }
    }
  }
  for (int i = tid; i < parts; i += kThreads) {
    const float2 v = __ldcg(zn + at + i);
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
    sh.z[warp] = zs;
    sh.n[warp] = n;
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
      sh.sp[shift > 5 ? g : warp][e + j] = v;
      sh.sc[shift > 5 ? g : warp][e + j] = q;
    }
  }
  __syncthreads();
  float ps = 0.f;
  int count = 0;
  zs = 0.f;
  n = 0;
  const int rows = shift > 5 ? groups : WARPS;
  if (tid < E)
    for (int i = 0; i < rows; ++i) {
      ps += sh.sp[i][tid];
      count += sh.sc[i][tid];
    }
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    zs += sh.z[i];
    n += sh.n[i];
  }
  finish_sequence(out, b, E, k, count, ps, zs, n, sh.red);
}

template <class Y>
__global__ void __launch_bounds__(kThreads, 2)
    balance_sums_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                        const uint8_t* __restrict__ mask, int L, int B, int parts, int E, int k, int32_t* __restrict__ counts,
                        float* __restrict__ psums, float2* __restrict__ zn, int* arrived, BalanceOut out, int* err) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int ROWS = 32 / Y::LANES, WARPS = kThreads / 32;
  constexpr int AHEAD = Y::E <= 4 ? 2 : 1;  // rows on their way while one is worked on
  constexpr int PICKS = 4;                  // picks of a thread that are asked for before the rows
  __shared__ int last_part;
  __shared__ int hist[256];
  __shared__ JoinShared join;
  auto& ps = join.sp;
  auto& zw = join.z;
  auto& nw = join.n;
  auto& red = join.red;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / Y::LANES, l = lane % Y::LANES;
  const int per = (L + parts - 1) / parts;
  for (int u = blockIdx.x; u < B * parts; u += gridDim.x) {
    const int b = u / parts, c = u - b * parts;
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    const int t0 = b * L + min(L, c * per), t1 = b * L + min(L, (c + 1) * per);
    const int32_t* picks = topk_idx + static_cast<size_t>(t0) * k;
    const int slots = (t1 - t0) * k;
    int first[PICKS];
#pragma unroll
    for (int i = 0; i < PICKS; ++i) {
      const int at = threadIdx.x + i * kThreads;
      first[i] = at < slots ? picks[at] : 0;
    }
    auto live = [&](int t) { return t < t1 && (!mask || mask[t]); };
    constexpr int STEP = WARPS * ROWS;
    const int tw0 = t0 + warp * ROWS;
    float v[AHEAD][Y::E];
    bool on[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int t = tw0 + sub + j * STEP;
      on[j] = live(t);
      load_values<Y>(logits + static_cast<size_t>(t) * E, on[j], E, l, v[j], -INFINITY);
    }
    __syncthreads();
    auto count = [&](int at, int e) {
      if (mask && !mask[t0 + at / k]) return;  // whatever it holds
      if (static_cast<unsigned>(e) < static_cast<unsigned>(E))
        atomicAdd(&hist[e], 1);
      else
        record_error(err, MOE_ERR_ARG, t0 + at / k);
    };
#pragma unroll
    for (int i = 0; i < PICKS; ++i)
      if (static_cast<int>(threadIdx.x) + i * kThreads < slots) count(threadIdx.x + i * kThreads, first[i]);
    for (int at = threadIdx.x + PICKS * kThreads; at < slots; at += kThreads) count(at, picks[at]);
    float p[Y::E] = {};
    float z = 0.f;
    int n = 0;
    for (int tw = tw0; tw < t1; tw += AHEAD * STEP) {  // the same rounds for all lanes of the warp
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int t = tw + sub + j * STEP, tn = t + AHEAD * STEP;
        float w[Y::E];
#pragma unroll
        for (int i = 0; i < Y::E; ++i) w[i] = v[j][i];
        const bool now = on[j];
        on[j] = live(tn);
        load_values<Y>(logits + static_cast<size_t>(tn) * E, on[j], E, l, v[j], -INFINITY);
        float inv, lse;
        const bool ok = softmax_values<Y>(w, E, l, inv, lse);
        const float use = now ? inv : 0.f;  // a row that is not there: zeros' exponentials, times 0
        n += now;
#pragma unroll
        for (int i = 0; i < Y::E; ++i) p[i] = fmaf(w[i], use, p[i]);
        z = fmaf(now ? lse : 0.f, lse, z);
        if (__any_sync(kFull, now && !ok) && now && !ok && l == 0) record_error(err, MOE_ERR_NONFINITE_CODE, t);
      }
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
    if (e < E)
#pragma unroll
      for (int w = 0; w < WARPS; ++w) psum += ps[w][e];
    if (parts == 1 || e == 0)
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
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
      if (arrived) {  // the last block of a sequence joins its parts
        __threadfence();
        __syncthreads();
        if (e == 0) {
          last_part = atomicAdd(arrived + b, 1) == parts - 1;
          if (last_part) arrived[b] = 0;  // for the next call
        }
        __syncthreads();
        if (last_part) {
          __threadfence();
          join_sequence<Y::V>(counts, psums, zn, b, parts, E, k, out, join);
        }
      }
    }
    __syncthreads();
  }
}

// The parts' sums of more sequences than there are counters for.
template <int V>
__global__ void __launch_bounds__(kThreads)
    balance_join_kernel(const int32_t* counts, const float* psums, const float2* zn, int B, int parts, int E, int k,
                        BalanceOut out) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ JoinShared join;
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    join_sequence<V>(counts, psums, zn, b, parts, E, k, out, join);
    __syncthreads();
  }
}

// dlogits = add + gradient; add may be dlogits itself or null.
template <class Y>
__global__ void __launch_bounds__(kBwdThreads, 4)
    balance_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ counts, const uint8_t* __restrict__ mask,
                       const float* __restrict__ dloss, const float* __restrict__ dz, int T, int L, int E, int k,
                       const float* add, float* dlogits) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int ROWS = 32 / Y::LANES;
  const int lane = threadIdx.x & 31;
  const int sub = lane / Y::LANES, l = lane % Y::LANES;
  const int rounds = (T + ROWS - 1) / ROWS;
  const int nwarps = gridDim.x * (kBwdThreads / 32), w = blockIdx.x * (kBwdThreads / 32) + (threadIdx.x >> 5);
  // consecutive rows to a warp: the sequence rarely changes
  const int per = (rounds + nwarps - 1) / nwarps;
  const int r0 = min(rounds, w * per), r1 = min(rounds, r0 + per);
  int next = 0;  // first token after the sequence in hand
  float a[Y::E] = {}, hz = 0.f;
  auto read = [&](int r, float (&v)[Y::E], float (&in)[Y::E], bool& on) {
    const int t = r * ROWS + sub;
    const bool here = r < r1 && t < T;
    on = here && (!mask || mask[t]);
    load_values<Y>(logits + static_cast<size_t>(t) * E, on, E, l, v, -INFINITY);
    load_values<Y>(add + static_cast<size_t>(t) * E, here && add, E, l, in, 0.f);
  };
  float v[Y::E], in[Y::E];
  bool on;
  read(r0, v, in, on);
  for (int r = r0; r < r1; ++r) {
    float vn[Y::E], inn[Y::E];
    bool on_n;
    read(r + 1, vn, inn, on_n);
    const int t = r * ROWS + sub;
    if (__any_sync(kFull, t >= next)) {
      const int b = min(t, T - 1) / L;
      next = (b + 1) * L;
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
    float inv, lse;
    const bool ok = softmax_values<Y>(v, E, l, inv, lse);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < Y::E; ++i) dot = fmaf(a[i], v[i], dot);
    dot = lanes_reduce<Y>(dot, [](float x, float y) { return x + y; });
    const float shift = fmaf(hz, lse, -dot * inv);
    if (ok && on)
#pragma unroll
      for (int i = 0; i < Y::E; ++i) in[i] = fmaf(v[i] * inv, a[i] + shift, in[i]);
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

// Blocks for so much work, as many as fit, or as the caller allows.
int blocks_of(long long work, int fit, int max_grid) {
  return static_cast<int>(std::min<long long>(work, max_grid > 0 ? std::min(fit, max_grid) : fit));
}

template <typename F>
cudaError_t with_layout(int E, F f) {
  if (E % 4 == 0) {  // whole 16-byte pieces
    if (E <= 8) return f(Lay<4, 1, 2>{});
    if (E <= 16) return f(Lay<4, 2, 2>{});
    if (E <= 32) return f(Lay<4, 4, 2>{});
    if (E <= 64) return f(Lay<4, 8, 2>{});
    if (E <= 128) return f(Lay<4, 16, 2>{});
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
                           float* part_zn, int* arrived, int* err, int max_grid, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE, s);
  const int parts = seq_parts(T, B);
  const BalanceOut out{counts, mean_p, loss, zloss};
  const int units = blocks_of(static_cast<long long>(B) * parts, num_sms() * 2, max_grid);
  float2* zn = reinterpret_cast<float2*>(part_zn);
  int* counters = B <= kBalanceCounters ? arrived : nullptr;
  cudaError_t e = with_layout(E, [&](auto y) {
    return launch_pdl(balance_sums_kernel<decltype(y)>, dim3(units), dim3(kThreads), 0, s, logits, topk_idx, mask, T / B, B,
                      parts, E, k, part_counts, part_p, zn, counters, out, err);
  });
  if (e == cudaSuccess && parts > 1 && !counters)
    e = launch_pdl(E % 4 ? balance_join_kernel<1> : balance_join_kernel<4>, dim3(blocks_of(B, 65535, max_grid)), dim3(kThreads), 0, s,
                   part_counts, part_p, zn, B, parts, E, k, out);
  return e;
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* counts, const uint8_t* mask, const float* dloss,
                               const float* dz, int T, int B, int E, int k, const float* add, float* dlogits,
                               int max_grid, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_BALANCE_BWD, s);
  return with_layout(E, [&](auto y) {
    const long long warps = ceil_div(T, 32 / decltype(y)::LANES);
    const int blocks = blocks_of(ceil_div(warps, kBwdThreads / 32), num_sms() * 4, max_grid);
    return launch_pdl(balance_bwd_kernel<decltype(y)>, dim3(blocks), dim3(kBwdThreads), 0, s, logits, counts, mask, dloss, dz, T,
                      T / B, E, k, add, dlogits);
  });
}

}  // namespace moe
