// Softmax cross entropy of z = x W^T over a vocabulary of V rows, without
// keeping the logits.
//
//   forward   lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target(t)
//   backward  D_tv = (g_t + h_t) exp(z_tv - lse_t) - [v = target(t)] g_t,
//             dx = D W, dW = D^T x, g and h the gradients of loss and lse
//
// The forward is one product whose epilogue keeps, of each row's 128 logits of
// a tile half, their maximum m and sum of exp(z - m); a second kernel joins a
// row's pairs.  loss is formed as (m - z_target) + log(sum), so that a certain
// token's small loss does not come out of the difference of two large numbers.
//
// The backward takes the vocabulary in pieces: the product again, with an
// epilogue that turns logits into D (one to three bf16 values, see terms_of), then
// the two products that read D.  A piece's D takes 512 MB at most unless there are
// more than 32,768 tokens; what it costs in memory traffic hides behind the
// products.
#include <algorithm>
#include <cstring>

#include "dense.cuh"
#include "xent.h"

namespace moe {
namespace {

constexpr int kCodeXent = 0x11;  // + operation, in the error word of a wait that ran out

// K blocks of a run of sums of fp32 gradients.
constexpr int kExactRun = 8;
// And of bf16 ones at most, 131,072 terms: each 16 lose up to 2^-23 of the sum, always
// towards zero, so a run 2^-10 of its terms' magnitudes, a quarter of the result's own
// rounding.  (2^22 tokens alike in one run: dW short by 2.0e-2 of itself.)
constexpr int kRoundedRun = 2048;
// K blocks of a run of a logit's sums: as even runs as there are of 12 at most.  Taking
// out a run costs the epilogue 0.3 us, and at a tile's end two runs of the next one
// are all that the products have room for: with runs of 4, 8, 11 and 16 of the 32
// blocks of d = 2048, 2000 tokens of V = 32001 take 185, 149, 146 and 145 us forward
// and 205, 168, 157 and 152 us for D, and lose 2^-19, 2^-18, 2^-17.5 and 2^-17 of the
// terms' magnitudes at most.
// Few tokens' time is their weights' bytes: runs of one block, whose losses nearly
// vanish (loss off by 1e-7 of itself, as a plain fp32 product's; 1e-6 with 8), cost
// 3 % there (2.5 us of 37 tokens of d = 4096 and V = 50257).
int logit_run(int T, int d) {
  const int blocks = d / kBK;
  return T <= kBM ? 1 : ceil_div(blocks, ceil_div(blocks, 12));
}
// Bytes of D that a piece of the vocabulary takes at least, and its columns at least.
constexpr size_t kPieceBytes = size_t(512) << 20;
constexpr int kPieceCols = 8192;
// bf16 values that D is the sum of: three (24 bits) for an fp32 gradient; two for a
// bf16 one of up to 256 tokens, where bytes and latency count more than the
// products: a row of a gradient is then little more than its target's term, whose
// rounding would be as large again as the result's own (2.4e-3 of the norm against
// 1.7e-3); one for more tokens.  Where only one of the two gradients is bf16 then, the
// products of the other take three values, and its own take a fourth, D rounded in
// units as it is alone (the first of three is no such value: dx was off by 3.1e-3 to 4.1e-3
// of its norm).  That costs 2 bytes of D (2000 tokens of V = 32001, d = 2048, bf16 dx and
// fp32 dW: 1025 -> 1065 us), where a second value in the product would cost another
// 2 T V d operations.
constexpr int kTerms = 3;
int terms_of(int T, bool f32) { return f32 ? kTerms : T <= 256 ? 2 : 1; }

struct Target {
  const void* p;
  int wide;  // int64
};
// The target of row t, or -1 for none.
__device__ __forceinline__ int load_target(const Target& g, int t, int V) {
  const long long v = g.wide ? static_cast<const long long*>(g.p)[t] : static_cast<const int*>(g.p)[t];
  return v >= 0 && v < V ? static_cast<int>(v) : -1;
}

// Tiles whose rows change fastest: the row blocks that share a tile of W run at
// the same time, and x stays in L2.
template <int CG>
__device__ __forceinline__ DenseTile rows_first(const DenseParams& p, int i, int rank) {
  const int nb = i / p.mt, mb = i - nb * p.mt;
  return {0, mb * kBM * CG + rank * kBM, nb * p.tn, 0, p.nkb};
}

// ------------------------------------------------------------- forward
struct StatsOp {
  static constexpr bool A_MN = false, B_MN = false, F16 = false, ONE = true, FLIP_A = false, FLIP_B = false, CHUNKS = false;
  struct Params : DenseParams {
    Target target;
    // [T][2 nt]: of half a tile's logits the maximum m and the sum s of exp(z - m) less
    // 1, the largest term's: a certain token's loss, log1p(s - 1), is not what the
    // roundings of sums near 1 leave (it was off by up to 6 2^-24 of 1)
    float2* part;
    float* zt;     // [T] the target's logit
  };
  static __device__ __forceinline__ float flag(const Params&, int) { return 1.f; }
  template <int CG>
  static __device__ __forceinline__ DenseTile tile(const Params& p, int i, int rank) {
    return rows_first<CG>(p, i, rank);
  }
  static __device__ __forceinline__ void coords(const Params&, const DenseTile& t, int kb, int& ak, int& am, int& bk,
                                                int& bn) {
    ak = bk = kb * kBK;
    am = t.m0;
    bn = t.n0;
  }
  static __device__ __forceinline__ int pre(const Params& p, const DenseTile& t, const DenseEpi& e) {
    const int row = t.m0 + 32 * e.q + e.lane;
    return row < p.M ? load_target(p.target, row, p.N) : -1;
  }
  static __device__ __forceinline__ void epilogue(const Params& p, const DenseTile& t, DenseEpi& e, int target,
                                                  uint32_t (&acc)[4][32]) {
    const int row = t.m0 + 32 * e.q + e.lane;
    const int col = dense_col(p, t, e), n = dense_width(p, t, e);
    if (n < 128) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * c + j >= n) acc[c][j] = 0xff800000u;  // -inf: exp is 0
    }
    float m4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      m4[c] = __uint_as_float(acc[c][0]);
#pragma unroll
      for (int j = 1; j < 32; ++j) m4[c] = fmaxf(m4[c], __uint_as_float(acc[c][j]));
    }
    const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    const float base = m == -INFINITY ? 0.f : m;  // nothing but -inf: the sum is 0
    float s4[4] = {0.f, 0.f, 0.f, 0.f};
    int ones[4] = {-1, 0, 0, 0};  // terms that are 1, but for the largest
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float v = exp_short(__uint_as_float(acc[c][j]) - base);
        const bool one = v >= 1.f;  // not where v is NaN
        s4[j & 3] += one ? 0.f : v;
        ones[j & 3] += one;
      }
    if (row < p.M)
      p.part[static_cast<size_t>(row) * (2 * p.nt) + 2 * (t.n0 / p.tn) + e.part] =
          make_float2(m, ((s4[0] + s4[1]) + (s4[2] + s4[3])) + ((ones[0] + ones[1]) + (ones[2] + ones[3])));
    const int rel = target - col;
    const bool here = target >= 0 && rel >= 0 && rel < min(n, 128);
    if (__any_sync(0xffffffffu, here)) {
      uint32_t z = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (rel == 32 * c + j) z = acc[c][j];
      if (here) p.zt[row] = __uint_as_float(z);
    }
  }
};

// Joins the pairs of a row, WARPS warps a row (eight where there are few rows), the
// pairs in a fixed order.
// What the sum y + 1 of a pair with the maximum x adds to one with the maximum m.
// A pair without a finite logit (y = -1) adds nothing.
__device__ __forceinline__ float pair_adds(float2 a, float m) {
  const float s = 1.f + a.y;
  return s == 0.f ? 0.f : s * (a.x == m ? 1.f : expf(a.x - m));
}
__device__ __forceinline__ float2 join_pairs(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.x == m ? a.y + pair_adds(b, m) : b.y + pair_adds(a, m));
}
template <int WARPS>
__global__ void __launch_bounds__(256) xent_join_kernel(const float2* __restrict__ part, const float* __restrict__ zt,
                                                        Target target, int T, int V, int np, float* __restrict__ loss,
                                                        float* __restrict__ lse, int* err) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float2 sw[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = WARPS == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
  if (t >= T) return;
  const float2* row = part + static_cast<size_t>(t) * np;
  float2 v = make_float2(-INFINITY, -1.f);
  constexpr int STEP = 32 * WARPS;
  for (int i = WARPS == 1 ? lane : static_cast<int>(threadIdx.x); i < np; i += 4 * STEP) {
    float2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = i + j * STEP < np ? row[i + j * STEP] : make_float2(-INFINITY, -1.f);
    const float m = fmaxf(fmaxf(fmaxf(v.x, w[0].x), fmaxf(w[1].x, w[2].x)), w[3].x);
    bool less = v.x == m;  // the largest term's 1 is out
    float s = less ? v.y : pair_adds(v, m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool out = !less && w[j].x == m;
      s += out ? w[j].y : pair_adds(w[j], m);
      less |= out;
    }
    v = make_float2(m, s);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1)
    v = join_pairs(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off)));
  if constexpr (WARPS > 1) {
    if (lane == 0) sw[warp] = v;
    __syncthreads();
    if (warp) return;
    v = sw[lane & 7];
#pragma unroll
    for (int off = 4; off; off >>= 1)
      v = join_pairs(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, off), __shfl_xor_sync(0xffffffffu, v.y, off)));
  }
  if (lane == 0) {
    const float ls = log1pf(v.y);
    lse[t] = v.x + ls;
    const long long g = target.wide ? static_cast<const long long*>(target.p)[t] : static_cast<const int*>(target.p)[t];
    if (g >= V) record_error(err, MOE_ERR_ARG, t);
    loss[t] = g >= 0 && g < V ? (v.x - zt[t]) + ls : 0.f;
  }
}

// ------------------------------------------------------------ backward: D
// What the backward needs of a row.
//
// Where D enters a product in one bf16 value, a row of it is kept divided by its unit, that
// number which makes its target's entry, the largest as a rule, a bf16 value exactly.
// dx, whose rows are sums over a row of D, is multiplied by it again in fp32.  dW's
// sums have a part of every row: they are multiplied by the rows' mean unit
// (common_units).  All units are near one number, which takes the largest entry to
// the top of a binade, where the steps are small beside the values: the step at the
// bottom, which the same weight for all tokens can meet, is twice as large.  (dW of
// 1800 of 2000 tokens, V = 32001: off by 1.9e-3 of its norm, its own rounding being
// 1.7e-3; 2.9e-3 with units near 1 that dW is not multiplied by.)
struct RowGrads {
  Target target;
  const float* loss;
  const float* dloss;
  const float* dlse;  // or null
  int V;
  const float* units;  // what the units are near, and their mean; null: 1
  // D at the target: (g + h) p - g with p = exp(-loss), so that what is left of a
  // certain token's gradient is not the difference of two numbers near g.  One fma in
  // every kernel: a unit comes of rounding this to bf16, and where the kernels that divide
  // and multiply by it had another last bit, a row could be off by a step of bf16.
  static __device__ __forceinline__ float at_target(float loss, float g, float h) {
    return __fmaf_rn(h, expf(-loss), __fmul_rn(g, expm1f(-loss)));
  }
  static __device__ __forceinline__ float unit_near(float at, float near) {
    return at / bf16_lo(pack_bf16(at / near, 0.f));
  }
  // Of a row with the entry `at` at its target, or 0 without one.
  __device__ __forceinline__ float unit(float at) const {
    const float s = unit_near(at, units ? units[0] : 1.f);
    return s > 0.25f && s < 4.f ? s : units ? units[1] : 1.f;
  }
};

struct GradOp {
  static constexpr bool A_MN = false, B_MN = false, F16 = false, ONE = true, FLIP_A = false, FLIP_B = false, CHUNKS = false;
  struct Params : DenseParams {
    RowGrads rows;
    const float* lse;
    int v0;             // the piece is columns [v0, v0 + N) of V; columns from V on are zeros
    int terms;          // D is the sum of so many bf16 values, each N columns further
    int rounded;        // 1: another N columns with D in one bf16 value, divided by its unit
    uint16_t* D;        // [T, (terms + rounded) N]
  };
  struct Pre {
    float w, lse, at;  // of exp(z - lse); log of the sum; D at the target
    float by;          // 1 / unit
    int rel;           // the target's column among this thread's, or another number
  };
  static __device__ __forceinline__ float flag(const Params&, int) { return 1.f; }
  template <int CG>
  static __device__ __forceinline__ DenseTile tile(const Params& p, int i, int rank) {
    return rows_first<CG>(p, i, rank);
  }
  static __device__ __forceinline__ void coords(const Params& p, const DenseTile& t, int kb, int& ak, int& am, int& bk,
                                                int& bn) {
    ak = bk = kb * kBK;
    am = t.m0;
    bn = p.v0 + t.n0;
  }
  static __device__ __forceinline__ Pre pre(const Params& p, const DenseTile& t, const DenseEpi& e) {
    const int row = t.m0 + 32 * e.q + e.lane;
    Pre r{0.f, 0.f, 0.f, 1.f, -1};
    if (row < p.M) {
      const int target = load_target(p.rows.target, row, p.rows.V);
      const float g = target >= 0 ? p.rows.dloss[row] : 0.f, h = p.rows.dlse ? p.rows.dlse[row] : 0.f;
      r.w = g + h;
      r.lse = p.lse[row];
      if (g != 0.f) {
        r.at = p.rows.at_target(p.rows.loss[row], g, h);
        r.rel = target - (p.v0 + dense_col(p, t, e));
      }
      if (p.terms == 1) {
        const float s = p.rows.unit(r.at);
        r.w /= s;
        r.at /= s;
      } else if (p.rounded) {
        r.by = 1.f / p.rows.unit(r.at);
      }
    }
    return r;
  }
  static __device__ __forceinline__ void epilogue(const Params& p, const DenseTile& t, DenseEpi& e, const Pre& r,
                                                  uint32_t (&acc)[4][32]) {
    const int col = dense_col(p, t, e);  // of the piece
    const int n = p.rows.V - (p.v0 + col);  // columns that exist
    const int w = dense_width(p, t, e);  // a multiple of 32
    const int y = t.m0 + 32 * e.q;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= w) break;
      float f[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float v = r.w * exp_short(__uint_as_float(acc[c][j]) - r.lse);
        // a row that no gradient reaches adds nothing, whatever its logits are
        f[j] = (r.w != 0.f && 32 * c + j < n) ? v : 0.f;
        if (32 * c + j == r.rel) f[j] = r.at;
      }
      uint16_t* to = p.D + static_cast<size_t>(y + e.lane) * ((p.terms + p.rounded) * p.N) + col + 32 * c;
      auto put = [&](int k, const uint32_t* w) {
        if (y + e.lane < p.M) {
          st_32(to + k * p.N, w);
          st_32(to + k * p.N + 16, w + 8);
        }
      };
      if (p.rounded) {
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) w[u] = pack_bf16(r.by * f[2 * u], r.by * f[2 * u + 1]);
        put(p.terms, w);
      }
      for (int k = 0;; ++k) {
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) w[u] = pack_bf16(f[2 * u], f[2 * u + 1]);
        put(k, w);
        if (k + 1 == p.terms) break;
#pragma unroll
        for (int u = 0; u < 16; ++u) {  // what the value so far leaves, exactly
          f[2 * u] -= bf16_lo(w[u]);
          f[2 * u + 1] -= bf16_hi(w[u]);
        }
      }
    }
  }
};

// ----------------------------------------------- backward: products of D
// out (+)= A . B with 16-bit or fp32 results.  DX: A = D [T, terms N], B = rows
// [v0, ..) of W, K runs over the piece, once for each bf16 term of D.  DW: A =
// D^T, B = x, K runs over the tokens, likewise.  Either may take one of D's values alone.
template <bool DX>
struct ProdOp {
  static constexpr bool A_MN = !DX, B_MN = true, F16 = false, ONE = true, FLIP_A = false, FLIP_B = false, CHUNKS = false;
  struct Params : DenseParams {
    int v0;           // DX: the piece's first column of the vocabulary
    int once;         // K blocks of one of D's bf16 terms
    int cols;         // columns of the piece: from one term of D to the next
    int d0;           // first column in D of the first term
    int per_split;    // K blocks of a split; each has a matrix of its own in out
    RowGrads rows;    // DX; units also else
    int unit;         // the rows of D that it takes are divided by their units
    const float* prev;  // added to the products, laid out as out is in fp32
    void* out;        // [splits][M][N]
    int bf16;         // type of out
    int apart, prev_apart;  // 1: not on a 32-byte boundary
  };
  static __device__ __forceinline__ float flag(const Params&, int) { return 1.f; }
  template <int CG>
  static __device__ __forceinline__ DenseTile tile(const Params& p, int i, int rank) {
    // columns fastest: the tiles that run at one time are about as many row
    // blocks as column blocks
    const int per = p.mt * p.nt, split = i / per, j = i - split * per;
    const int mb = j / p.nt, nb = j - mb * p.nt;
    const int kb0 = min(p.nkb, split * p.per_split);
    return {split, mb * kBM * CG + rank * kBM, nb * p.tn, kb0, min(p.nkb, kb0 + p.per_split)};
  }
  static __device__ __forceinline__ void coords(const Params& p, const DenseTile& t, int kb, int& ak, int& am, int& bk,
                                                int& bn) {
    const int term = (kb >= p.once) + (kb >= 2 * p.once), k = (kb - term * p.once) * kBK;  // three terms at most
    if constexpr (DX) {
      ak = p.d0 + kb * kBK;  // the terms follow one another in a row of D
      am = t.m0;
      bk = p.v0 + k;
    } else {
      ak = bk = k;
      am = p.d0 + t.m0 + term * p.cols;
    }
    bn = t.n0;
  }
  static __device__ __forceinline__ float pre(const Params& p, const DenseTile& t, const DenseEpi& e) {
    if constexpr (!DX) return p.unit ? p.rows.units[1] : 1.f;
    const int row = t.m0 + 32 * e.q + e.lane;
    if (!p.unit || row >= p.M) return 1.f;
    const float g = load_target(p.rows.target, row, p.rows.V) >= 0 ? p.rows.dloss[row] : 0.f;
    const float h = p.rows.dlse ? p.rows.dlse[row] : 0.f;
    return p.rows.unit(g != 0.f ? p.rows.at_target(p.rows.loss[row], g, h) : 0.f);
  }
  static __device__ __forceinline__ void epilogue(const Params& p, const DenseTile& t, DenseEpi& e, float unit,
                                                  uint32_t (&acc)[4][32]) {
    const int x = dense_col(p, t, e), row = t.m0 + 32 * e.q + e.lane;
    const int w = dense_width(p, t, e);  // a multiple of 32
    if (row >= p.M) return;
    const size_t at = (static_cast<size_t>(t.mat) * p.M + row) * p.N + x;
    if (p.unit)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] = __float_as_uint(unit * __uint_as_float(acc[c][j]));
    if (p.prev) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (32 * c < w)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t v[8];
            const float* from = p.prev + at + 32 * c + 8 * j;
            if (p.prev_apart) {
              *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(from);
              *reinterpret_cast<uint4*>(v + 4) = *reinterpret_cast<const uint4*>(from + 4);
            } else {
              ld_32(from, v);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[c][8 * j + i] = __float_as_uint(__uint_as_float(acc[c][8 * j + i]) + __uint_as_float(v[i]));
          }
    }
    auto store = [&](void* to, const uint32_t* w) {
      if (p.apart)
        st_2x16(to, w);
      else
        st_32(to, w);
    };
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (32 * c >= w) break;
      if (p.bf16) {
        uint32_t b[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          b[u] = pack_bf16(__uint_as_float(acc[c][2 * u]), __uint_as_float(acc[c][2 * u + 1]));
        uint16_t* to = static_cast<uint16_t*>(p.out) + at + 32 * c;
        store(to, b);
        store(to + 16, b + 8);
      } else {
        float* to = static_cast<float*>(p.out) + at + 32 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) store(to + 8 * j, &acc[c][8 * j]);
      }
    }
  }
};

// What the units of D's rows are near, and their mean by the squares of the targets'
// entries, from up to 1024 tokens spread over all; by one block of 256.
__device__ __forceinline__ void common_units(const RowGrads& rows, int T, float* units) {
  __shared__ float ws[3][8];
  constexpr int EACH = 4;
  const int n = min(T, 256 * EACH), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float at[EACH], most = 0.f;
  float g[EACH], h[EACH], loss[EACH];  // all asked for before any is used
  int target[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int j = min(static_cast<int>(threadIdx.x) + 256 * i, n - 1);
    const int t = static_cast<int>(static_cast<long long>(j) * T / n);
    target[i] = load_target(rows.target, t, rows.V);
    g[i] = rows.dloss[t];
    h[i] = rows.dlse ? rows.dlse[t] : 0.f;
    loss[i] = rows.loss[t];
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const bool here = static_cast<int>(threadIdx.x) + 256 * i < n && target[i] >= 0 && g[i] != 0.f;
    const float v = RowGrads::at_target(loss[i], g[i], h[i]);
    at[i] = here && isfinite(v) ? v : 0.f;
    most = fmaxf(most, fabsf(at[i]));
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
  if (lane == 0) ws[0][warp] = most;
  __syncthreads();
  for (int w = 0; w < 8; ++w) most = fmaxf(most, ws[0][w]);
  int ex;
  const float near = most > 0.f ? frexpf(most, &ex) * (256.f / 255.f) : 1.f;  // 255 / 256: bf16's last value below 1
  float sum = 0.f, weight = 0.f;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const float s = RowGrads::unit_near(at[i], near) / near - 1.f;
    if (!(fabsf(s) < 0.01f)) continue;  // also 0 and what has no bf16 value
    sum = fmaf(at[i] * at[i], s, sum);
    weight = fmaf(at[i], at[i], weight);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    weight += __shfl_xor_sync(0xffffffffu, weight, off);
  }
  if (lane == 0) {
    ws[1][warp] = sum;
    ws[2][warp] = weight;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = weight = 0.f;
    for (int w = 0; w < 8; ++w) {
      sum += ws[1][w];
      weight += ws[2][w];
    }
    const float u = sum / weight;
    units[0] = near;
    units[1] = near * (fabsf(u) < 0.01f ? 1.f + u : 1.f);  // near itself where squares leave fp32's range
  }
}

// x with the rows that no gradient reaches cleared: what they hold (padding may
// hold anything) must not meet D's zeros in dW's sums.  units: of D, if wanted.
__global__ void __launch_bounds__(256) xent_rows_kernel(const uint4* __restrict__ x, RowGrads rows, int T, int pieces,
                                                        float* __restrict__ units, uint4* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  if (units && blockIdx.x == gridDim.x - 1) common_units(rows, T, units);
  const size_t total = static_cast<size_t>(T) * pieces;
  for (size_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
    const int t = static_cast<int>(i / pieces);
    const bool live = (load_target(rows.target, t, rows.V) >= 0 && rows.dloss[t] != 0.f) || (rows.dlse && rows.dlse[t] != 0.f);
    out[i] = live ? x[i] : make_uint4(0, 0, 0, 0);
  }
}

// Sum of the splits in their order.
__global__ void __launch_bounds__(256) xent_sum_kernel(const float4* __restrict__ part, int splits, size_t n4, int bf16,
                                                       void* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  for (size_t i = blockIdx.x * 256ull + threadIdx.x; i < n4; i += gridDim.x * 256ull) {
    float4 a = part[i];
    for (int s = 1; s < splits; ++s) {
      const float4 v = part[s * n4 + i];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    if (bf16)
      static_cast<uint2*>(out)[i] = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
    else
      static_cast<float4*>(out)[i] = a;
  }
}

// ------------------------------------------------------------------ host
constexpr int kMaxSplits = 64;

// How D enters the products: as so many bf16 values for dx and for dW, the first of so
// many; behind these (rounded) in one value for the gradient that takes one alone.
struct Terms {
  int dx, dW, first, rounded;
};
Terms terms_for(int T, bool want_dx, bool dx_f32, bool want_dW, bool dW_f32) {
  const int x = want_dx ? terms_of(T, dx_f32) : 1, w = want_dW ? terms_of(T, dW_f32) : 1;
  const int first = std::max(x, w), rounded = first > 1 && ((want_dx && x == 1) || (want_dW && w == 1));
  return {x, w, first, rounded};
}

struct Plan {
  int cols;    // most columns of a piece, a multiple of 256, counted in bf16 values of a row of D
  DenseShape dx, dW;
  size_t err, part, zt, D, acc, xz, units, total;
};

// Tiles of the logits [T, cols], tn a multiple of `unit`.  Where a row block or a few
// have all tokens, or all tiles run at one time, single CTAs take equal shares of
// the vocabulary: its rows' bytes, or latency, are what counts then.
void logit_tiles(DenseParams& p, int T, int cols, int unit) {
  const int mt = ceil_div(T, kBM);
  if (mt > 1 && static_cast<long long>(mt) * ceil_div(cols, kBN) > 152) {
    dense_shape(p, 2, kBN, 1, false);
    return;
  }
  const int each = std::max(1, 152 / mt), rounds = ceil_div(cols, static_cast<long long>(each) * kBN);
  const int tn = std::max(64, ceil_div(ceil_div(cols, static_cast<long long>(each) * rounds), unit) * unit);
  dense_shape(p, 1, std::min(kBN, tn), 1, false);
  p.a_bytes = std::min(kBM, ceil_div(T, 8) * 8) * 128;  // no more rows than there are
}
int logit_cg(const DenseParams& p, int T) { return p.mt == ceil_div(T, kBM) ? 1 : 2; }

Plan plan(int T, int V, int d, int backward, const Terms& h) {
  Plan p{};
  DenseParams tiles{};
  tiles.M = T;
  tiles.N = V;
  logit_tiles(tiles, T, V, 16);
  const int all = ceil_div(V, kBN) * kBN;
  const long long want = std::max<long long>(kPieceBytes / 2 / T / kBN * kBN, kPieceCols);
  // every value of D for the whole vocabulary at most
  p.cols = static_cast<int>(std::min<long long>(want, 1ll * (kTerms + 1) * all));
  if (backward) {
    const int width = std::min(V, p.cols / (h.first + h.rounded));
    p.dx = dense_pick(T, d, 1, (h.rounded ? h.dx : h.first) * ceil_div(width, kBK), false, kMaxSplits);
    p.dW = dense_pick(width, d, 1, (h.rounded ? h.dW : h.first) * ceil_div(T, kBK), false, width == V ? kMaxSplits : 1);
  }
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  p.err = take(kErrRegionBytes);
  const size_t begin = o;
  p.part = take(sizeof(float2) * 2 * tiles.nt * T);
  p.zt = take(sizeof(float) * T);
  size_t end = o;
  if (backward) {
    o = begin;  // the forward's scratch is free by then
    p.D = take(size_t(2) * T * p.cols);
    p.acc = take(sizeof(float) * std::max(size_t(p.dx.splits) * T, p.dW.splits > 1 ? size_t(p.dW.splits) * V : 0) * d);
    p.xz = take(size_t(2) * T * d);
    p.units = take(sizeof(float) * 2);
    end = std::max(end, o);
  }
  p.total = end;
  return p;
}

template <class Op>
int launch_logits(typename Op::Params& p, const XentArgs& a, int trace, cudaStream_t s) {
  return dense_launch<Op>(logit_cg(p, a.T), p, a.grid_limit, trace, s);
}

// out [n] = sum of `splits` fp32 arrays.
int launch_sum(const float* part, int splits, size_t n, bool bf16, void* out, cudaStream_t s) {
  TraceScope trace_scope(MOE_K_XENT_ROWS, s);
  const size_t n4 = n / 4;
  const int blocks = static_cast<int>(std::min<size_t>((n4 + 255) / 256, num_sms() * 8));
  return launch_pdl(xent_sum_kernel, dim3(blocks), dim3(256), 0, s, reinterpret_cast<const float4*>(part), splits, n4, bf16,
                    out) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

size_t xent_workspace_bytes(int T, int V, int d, int backward) {
  size_t most = 0;
  for (int types = 0; types < (backward ? 4 : 1); ++types)  // of dx and dW; one alone takes what both of its type do
    most = std::max(most, plan(T, V, d, backward, terms_for(T, true, types & 1, true, types & 2)).total);
  return most;
}

int launch_xent_fwd(const XentArgs& a, cudaStream_t s) {
  const Plan L = plan(a.T, a.V, a.d, 0, {});
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  int* err = reinterpret_cast<int*>(ws + L.err);
  StatsOp::Params p;
  std::memset(&p, 0, sizeof(p));
  p.M = a.T;
  p.N = a.V;
  logit_tiles(p, a.T, a.V, 16);
  if (!dense_map_k(&p.tmA, a.x, false, a.d, a.T, 1, a.d, p.a_bytes / 128) ||
      !dense_map_k(&p.tmB, a.W, false, a.d, a.V, 1, a.d, p.b_bytes / 128))
    return MOE_ERR_CUDA;
  p.nkb = a.d / kBK;
  p.run_kb = logit_run(a.T, a.d);
  p.code = kCodeXent;
  p.err = err;
  p.target = {a.target, a.target_type};
  p.part = reinterpret_cast<float2*>(ws + L.part);
  p.zt = reinterpret_cast<float*>(ws + L.zt);
  const int rc = launch_logits<StatsOp>(p, a, MOE_K_XENT, s);
  if (rc != MOE_OK) return rc;
  TraceScope trace_scope(MOE_K_XENT_JOIN, s);
  const bool few = a.T <= 4 * 152;  // a block a row as long as all rows run at one time
  return launch_pdl(few ? xent_join_kernel<8> : xent_join_kernel<1>, dim3(few ? a.T : ceil_div(a.T, 8)), dim3(256), 0, s,
                    p.part, p.zt, p.target, a.T, a.V, 2 * p.nt, a.loss, a.lse, err) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

int launch_xent_bwd(const XentArgs& a, cudaStream_t s) {
  const Terms h = terms_for(a.T, a.dx, a.dx_type == MOE_Y_F32, a.dW, a.dW_type == MOE_Y_F32);
  const int values = h.first + h.rounded;  // of D
  const Plan L = plan(a.T, a.V, a.d, 1, h);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  int* err = reinterpret_cast<int*>(ws + L.err);
  void* D = ws + L.D;
  float* accbuf = reinterpret_cast<float*>(ws + L.acc);
  uint16_t* xz = reinterpret_cast<uint16_t*>(ws + L.xz);
  float* units = a.dW && h.dW == 1 ? reinterpret_cast<float*>(ws + L.units) : nullptr;
  const Target target{a.target, a.target_type};
  const RowGrads rows{target, a.loss, a.dloss, a.dlse, a.V, units};
  // pieces of about equal size, whole tiles wide
  const int most = L.cols / values / kBN * kBN;
  const int pieces = ceil_div(a.V, most);
  const int width = ceil_div(ceil_div(a.V, pieces), kBN) * kBN;
  int rc;

  if (a.dW) {
    TraceScope trace_scope(MOE_K_XENT_ROWS, s);
    const long long n = static_cast<long long>(a.T) * (a.d / 8);
    const int blocks = static_cast<int>(std::min<long long>(ceil_div(n, 256), num_sms() * 8ll));
    if (launch_pdl(xent_rows_kernel, dim3(blocks), dim3(256), 0, s, reinterpret_cast<const uint4*>(a.x), rows, a.T, a.d / 8,
                   units, reinterpret_cast<uint4*>(xz)) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  for (int v0 = 0; v0 < a.V; v0 += width) {
    const int real = std::min(width, a.V - v0);
    const int cols = ceil_div(real, kBN) * kBN;
    {
      GradOp::Params p;
      std::memset(&p, 0, sizeof(p));
      p.M = a.T;
      p.N = cols;
      logit_tiles(p, a.T, cols, 32);
      if (!dense_map_k(&p.tmA, a.x, false, a.d, a.T, 1, a.d, p.a_bytes / 128) ||
          !dense_map_k(&p.tmB, a.W, false, a.d, a.V, 1, a.d, p.b_bytes / 128))
        return MOE_ERR_CUDA;
      p.D = static_cast<uint16_t*>(D);
      p.nkb = a.d / kBK;
      p.run_kb = logit_run(a.T, a.d);  // the forward's logits, bit for bit
      p.code = kCodeXent + 1;
      p.err = err;
      p.rows = rows;
      p.lse = a.lse;
      p.v0 = v0;
      p.terms = h.first;
      p.rounded = h.rounded;
      if ((rc = launch_logits<GradOp>(p, a, MOE_K_XENT_GRAD, s)) != MOE_OK) return rc;
    }
    if (a.dx) {
      ProdOp<true>::Params p;
      std::memset(&p, 0, sizeof(p));
      const bool f32 = a.dx_type == MOE_Y_F32;
      const int splits = L.dx.splits;
      p.M = a.T;
      p.N = a.d;
      p.once = cols / kBK;
      p.nkb = h.dx * p.once;
      p.run_kb = f32 ? kExactRun : kRoundedRun;
      p.rows = rows;
      p.unit = h.dx == 1;
      p.d0 = p.unit && h.rounded ? h.first * cols : 0;
      p.code = kCodeXent + 2;
      p.err = err;
      p.v0 = v0;
      p.cols = cols;
      p.per_split = ceil_div(p.nkb, splits);  // a split without K blocks keeps the sums so far
      dense_shape(p, L.dx.cg, L.dx.tn, splits, false);
      const bool last = v0 + width >= a.V;
      // fp32 sums of the pieces so far: in dx itself where it has that type
      float* sums = splits == 1 && f32 ? static_cast<float*>(a.dx) : accbuf;
      p.prev = v0 > 0 ? sums : nullptr;
      p.prev_apart = (reinterpret_cast<uintptr_t>(sums) & 31) != 0;
      p.out = splits == 1 && last ? a.dx : sums;
      p.bf16 = splits == 1 && last && !f32;
      p.apart = (reinterpret_cast<uintptr_t>(p.out) & 31) != 0;
      if (!dense_map_k(&p.tmA, D, false, size_t(cols) * values, a.T, 1, size_t(cols) * values, 128) ||
          !dense_map_mn(&p.tmB, a.W, false, a.d, a.V, 1, p.b_bytes / kBoxBytes))
        return MOE_ERR_CUDA;
      if ((rc = dense_launch<ProdOp<true>>(L.dx.cg, p, a.grid_limit, MOE_K_XENT_DX, s)) != MOE_OK) return rc;
      if (last && splits > 1 && (rc = launch_sum(accbuf, splits, size_t(a.T) * a.d, !f32, a.dx, s)) != MOE_OK) return rc;
    }
    if (a.dW) {
      ProdOp<false>::Params p;
      std::memset(&p, 0, sizeof(p));
      const bool f32 = a.dW_type == MOE_Y_F32;
      const int splits = pieces == 1 ? L.dW.splits : 1;  // accbuf holds dx's sums else
      p.M = real;
      p.N = a.d;
      p.once = ceil_div(a.T, kBK);
      p.nkb = h.dW * p.once;
      p.run_kb = f32 ? kExactRun : kRoundedRun;
      p.rows = rows;
      p.unit = h.dW == 1;
      p.d0 = p.unit && h.rounded ? h.first * cols : 0;
      p.code = kCodeXent + 3;
      p.err = err;
      p.cols = cols;
      p.per_split = ceil_div(p.nkb, splits);
      dense_shape(p, L.dW.cg, L.dW.tn, splits, false);
      p.bf16 = splits == 1 && !f32;
      p.out = splits > 1 ? static_cast<void*>(accbuf) : static_cast<uint8_t*>(a.dW) + size_t(v0) * a.d * (f32 ? 4 : 2);
      p.apart = (reinterpret_cast<uintptr_t>(p.out) & 31) != 0;
      if (!dense_map_mn(&p.tmA, D, false, size_t(cols) * values, a.T, 1, 2) ||
          !dense_map_mn(&p.tmB, xz, false, a.d, a.T, 1, p.b_bytes / kBoxBytes))
        return MOE_ERR_CUDA;
      if ((rc = dense_launch<ProdOp<false>>(L.dW.cg, p, a.grid_limit, MOE_K_XENT_DW, s)) != MOE_OK) return rc;
      if (splits > 1 && (rc = launch_sum(accbuf, splits, size_t(a.V) * a.d, !f32, a.dW, s)) != MOE_OK) return rc;
    }
  }
  return MOE_OK;
}

}  // namespace moe
