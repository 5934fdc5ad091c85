// Router of one token on one warp: softmax over the experts, top-k on the
// logits.  Shared by the routing kernels and the layer for a few tokens, so
// every path gives the same bits.
#pragma once
#include <math.h>

#include <cstdint>

#include "common.cuh"

namespace moe {

constexpr unsigned kFull = 0xffffffffu;

// Softmax statistics of one logit row held lane-strided by a warp
// (expert e = lane + 32 * i).  Router forward and backward both use this,
// so the backward's probabilities are bit-identical to the forward's.
template <int EPL>
struct RowSoftmax {
  float v[EPL];   // logits (-inf beyond E)
  float ex[EPL];  // expf(v - m) (0 beyond E)
  float m, s;     // max, sum of ex
};

// One logit row, lane-strided (-inf beyond E).
template <int EPL>
__device__ __forceinline__ void row_load(const float* __restrict__ row, int E, int lane, float (&v)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    v[i] = (e < E) ? row[e] : -INFINITY;
  }
}

// Order-preserving key of a finite float: a larger value has a larger
// unsigned key, -0.0 and +0.0 share one, and every finite value's key is
// above 0 (the key of "no entry").  Warp max/min over keys are single
// redux.sync instructions, where a float max needs a shuffle butterfly.
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// Softmax statistics of the row already in r.v; false if it holds a
// non-finite logit (the statistics are then unspecified).  key[i] is the
// order key of entry i (0 beyond E).
template <int EPL>
__device__ __forceinline__ bool row_stats(int E, int lane, RowSoftmax<EPL>& r, unsigned (&key)[EPL]) {
  bool bad = false;
  unsigned kmax = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (e < E && !isfinite(r.v[i])) bad = true;
    key[i] = e < E ? order_key(r.v[i]) : 0u;
    kmax = max(kmax, key[i]);
  }
  bad = __any_sync(kFull, bad);
  // The maximum is exact whichever way it is found; -0.0 and +0.0 give the
  // same exp(v - m) bits.
  const float m = key_value(__reduce_max_sync(kFull, kmax));
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    r.ex[i] = (e < E) ? expf(r.v[i] - m) : 0.f;
    s += r.ex[i];
  }
  // xor butterfly: every lane adds the same pairs, so all lanes end with
  // the same bits.
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
  r.m = m;
  r.s = s;
  return !bad;
}

template <int EPL>
__device__ __forceinline__ bool row_softmax(const float* __restrict__ row, int E, int lane, RowSoftmax<EPL>& r) {
  row_load<EPL>(row, E, lane, r.v);
  unsigned key[EPL];
  return row_stats<EPL>(E, lane, r, key);
}

// Routes token t on one warp (its logit row already in r.v): softmax
// statistics, then k rounds of warp argmax.  Lane j < k ends with slot j's
// expert and weight.  A row with a non-finite logit is reported and gets the
// placeholder routing slot j -> expert j with weight 0.
template <int EPL>
__device__ __forceinline__ void route_token(RowSoftmax<EPL>& r, int t, int E, int k, int renorm, int lane, int* err,
                                            int& my_idx, float& my_w) {
  my_idx = lane;
  my_w = 0.f;
  unsigned key[EPL];
  if (!row_stats<EPL>(E, lane, r, key)) {
    if (lane == 0) record_error(err, MOE_ERR_NONFINITE_CODE, t);
    return;
  }
  float my_ex = 0.f;
  for (int j = 0; j < k; ++j) {
    // Best remaining entry of this lane: strictly greater keeps the lower
    // index on ties (entries are visited in increasing expert index).
    unsigned bk = 0;
    unsigned be = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > bk) {
        bk = key[i];
        be = static_cast<unsigned>(lane + 32 * i);
      }
    // Winner under (value desc, index asc), a strict total order: the
    // largest key, then the lowest expert index holding it.  Every lane
    // gets the same winner.
    const unsigned kbest = __reduce_max_sync(kFull, bk);
    const int bi = static_cast<int>(__reduce_min_sync(kFull, bk == kbest ? be : 0xffffffffu));
    const int owner = bi & 31, which = bi >> 5;
    float ex = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i == which) {
        if (lane == owner) key[i] = 0u;  // taken
        ex = r.ex[i];
      }
    ex = __shfl_sync(kFull, ex, owner);
    if (lane == j) {
      my_idx = bi;
      my_ex = ex;
    }
  }
  // one division per slot, all slots at once, outside the serial picks
  const float my_p = my_ex / r.s;
  float psum = 0.f;
  if (renorm)
    for (int j = 0; j < k; ++j) psum += __shfl_sync(kFull, my_p, j);
  my_w = renorm ? my_p / psum : my_p;
}

}  // namespace moe
