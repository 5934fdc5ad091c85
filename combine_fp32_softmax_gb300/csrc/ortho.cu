// Matrices to nearly orthogonal ones: X = G / (|G| + eps) in the Frobenius norm,
// then a number of steps of
//   A = X X^T,  B = b A + c A A,  X <- a X + B X
// with (a, b, c) = (3.4445, -4.7750, 2.0315), which bring every singular value of
// X near 1 (between 0.7 and 1.2 after five steps for those above 0.0016).  Where
// there are more rows than columns the products are X^T X and X B, so that A is
// always the smaller of the two and nothing is transposed in memory.
//
// X, A and B are kept in fp16 between the products, scaled by powers of two so
// that their whole range is normal numbers: a rounding is at most 2^-11 of a value,
// eight times finer than bf16's at the same tensor-core rate.  Beside X there are 8
// bits of what its rounding leaves, for the a X of a step, and B's diagonal is
// shifted in the last steps (ortho.cuh says why and what that measured): the result
// is then off by less than its own final rounding to bf16.  The norm itself enters
// as an fp32 factor of the first step, so a bf16 G is taken exactly.
//
// A and A A are symmetric: only the tiles on and above the diagonal are computed.
// Where the products run on CTA pairs only those are stored, and the products that
// read them take the others transposed (dense_flip); on single CTAs, whose tiles
// are smaller, the epilogue stores both halves.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_fp16.h>

#include "dense.cuh"
#include "ortho.cuh"
#include "ortho.h"

namespace moe {
namespace {

constexpr int kCodeOrtho = 0x19;
constexpr int kNormParts = 1024;  // partial sums of squares of a matrix, at most

// ------------------------------------------------------------- products
enum OrthoKind : int { kGramWide, kGramTall, kSquare, kUpdateWide, kUpdateTall };

template <int KIND>
struct OrthoOp {
  static constexpr bool SYM = KIND == kGramWide || KIND == kGramTall || KIND == kSquare;
  static constexpr bool A_MN = KIND == kGramTall;
  static constexpr bool B_MN = KIND == kGramTall || KIND == kUpdateWide;
  static constexpr bool F16 = true, ONE = false, CHUNKS = true;
  // which operands are symmetric matrices
  static constexpr bool FLIP_A = KIND == kSquare || KIND == kUpdateWide, FLIP_B = KIND == kSquare || KIND == kUpdateTall;
  struct Params : DenseParams {
    const float* scal;   // [mats]: X of the first step is scal times what is stored; 0: matrix needs no products
    int first;           // the first step
    float grown, grows;  // kNsA to the power of the step, and of the next (see step_scale)
    const __half* old;   // square: A; update: X, laid out as the result
    int pitch;           // of old
    uint8_t* lo;         // update: what rounding left of X, laid out as old; that of the result takes its place
    int lo_in, lo_out;   // whether it is there and wanted
    float shift;         // square, update: the polynomial is kept plus so many I
    void* out;           // [mats][M] rows
    int out_pitch;       // of out, a multiple of 16
    int bf16;            // last update: bf16 results
    int apart;           // 1: out is not on a 32-byte boundary
  };
  static __device__ __forceinline__ int tiles_each(const Params& p) { return SYM ? p.nt * (p.nt + 1) / 2 : p.mt * p.nt; }
  static __device__ __forceinline__ float flag(const Params& p, int i) { return p.scal[i / tiles_each(p)]; }
  template <int CG>
  static __device__ __forceinline__ DenseTile tile(const Params& p, int i, int rank) {
    const int per = tiles_each(p), mat = i / per;
    int j = i - mat * per, mb, nb;
    if constexpr (SYM) {  // row mb has the tiles mb, mb + 1, ... of its columns
      mb = 0;
      while (j >= p.nt - mb) j -= p.nt - mb++;
      nb = mb + j;
    } else {
      mb = j / p.nt;
      nb = j - mb * p.nt;
    }
    return {mat, mb * kBM * CG + rank * kBM, nb * p.tn, 0, p.nkb};
  }
  static __device__ __forceinline__ void coords(const Params&, const DenseTile& t, int kb, int& ak, int& am, int& bk,
                                                int& bn) {
    ak = bk = kb * kBK;
    am = t.m0;
    bn = t.n0;
  }
  // Read while the tile's products still run: the matrix's factor and, for
  // square and update, this thread's 128 values of the old matrix.
  struct Pre {
    float r;
    uint32_t old[SYM && KIND != kSquare ? 1 : 64];
    uint32_t lo[SYM ? 1 : 32];
  };
  static __device__ __forceinline__ Pre pre(const Params& p, const DenseTile& t, const DenseEpi& e) {
    Pre o;
    o.r = p.scal[t.mat];
    if constexpr (KIND == kSquare || !SYM) {
      const int x = dense_col(p, t, e), row = t.m0 + 32 * e.q + e.lane;
      const int w = dense_width(p, t, e);  // what it reads past the last column lies before the pitch
      const __half* from = p.old + (static_cast<size_t>(t.mat) * p.M + row) * p.pitch + x;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (row < p.M && 16 * u < w) {
          ld_32(from + 16 * u, &o.old[8 * u]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) o.old[8 * u + k] = 0u;
        }
      }
      if constexpr (!SYM) {
        const uint8_t* lo = p.lo + (static_cast<size_t>(t.mat) * p.M + row) * p.pitch + x;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (p.lo_in && row < p.M && 32 * c < w) {
            ld_32(lo + 32 * c, &o.lo[8 * c]);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) o.lo[8 * c + k] = 0u;
          }
        }
      }
    }
    return o;
  }
  static __device__ __forceinline__ void chunk(const Params& p, const DenseTile& t, const DenseEpi& e, const Pre& pre, int c,
                                               const uint32_t (&acc)[32]) {
    if (pre.r == 0.f) return;  // no products for this matrix
    const float r = p.first ? pre.r : step_scale(pre.r, p.grown);
    const float out = p.bf16 ? 1.f : 1.f / step_scale(pre.r, p.grows);  // update: of X' in what is stored
    const int x = dense_col(p, t, e) + 32 * c, y = t.m0 + 32 * e.q;
    // gram: A = r^2 sums; square: B + s I = b A + c sums + s I; update: X' =
    // (a - s) r X + r sums
    const float fs = KIND == kSquare                         ? kNsC * (kSB / (kSA * kSA))
                     : (KIND == kGramWide || KIND == kGramTall) ? r * r * kSA
                                                             : (r * out) / kSB;
    const float fo = KIND == kSquare ? kNsB * (kSB / kSA) : (kNsA - p.shift) * (r * out);
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = fs * __uint_as_float(acc[j]);
    if constexpr (KIND == kSquare || !SYM) {
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const float2 o = unpack_f16(pre.old[16 * c + u]);
        v[2 * u] = fmaf(fo, o.x, v[2 * u]);
        v[2 * u + 1] = fmaf(fo, o.y, v[2 * u + 1]);
      }
    }
    if constexpr (!SYM) {
      if (p.lo_in) {
        const float fl = fo * (1.f / kLo);
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const float2 o = unpack_e4m3(pre.lo[8 * c + u / 2] >> (16 * (u & 1)));
          v[2 * u] = fmaf(fl, o.x, v[2 * u]);
          v[2 * u + 1] = fmaf(fl, o.y, v[2 * u + 1]);
        }
      }
    }
    if (KIND == kSquare && x == y) {  // the chunk on the diagonal: column lane of a lane's row
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == e.lane) v[j] += p.shift * kSB;
    }
    uint32_t w[16];
#pragma unroll
    for (int u = 0; u < 16; ++u)
      w[u] = !SYM && p.bf16 ? pack_bf16(v[2 * u], v[2 * u + 1]) : pack_f16(v[2 * u], v[2 * u + 1]);
    uint16_t* mat = static_cast<uint16_t*>(p.out) + static_cast<size_t>(t.mat) * p.M * p.out_pitch;
    if (y + e.lane < p.M) {
      uint16_t* to = mat + static_cast<size_t>(y + e.lane) * p.out_pitch + x;
#pragma unroll
      for (int h = 0; h < 2; ++h)  // columns between the last and the pitch may hold anything
        if (x + 16 * h < p.out_pitch) {
          if (!SYM && p.apart)
            st_2x16(to + 16 * h, w + 8 * h);
          else
            st_32(to + 16 * h, w + 8 * h);
        }
      if constexpr (!SYM) {
        if (p.lo_out) {
          uint32_t l[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            l[u] = rest_e4m3(v[4 * u], v[4 * u + 1], w[2 * u]) | rest_e4m3(v[4 * u + 2], v[4 * u + 3], w[2 * u + 1]) << 16;
          st_32(p.lo + (static_cast<size_t>(t.mat) * p.M + y + e.lane) * p.pitch + x, l);
        }
      }
    }
    if constexpr (SYM) {
      if (!p.upper && t.n0 / p.tn > t.m0 / p.tn) {  // a tile off the diagonal: also to the other side
        // neighbouring lanes' rows side by side: even lanes take the even columns,
        // odd ones the odd, and a store covers 32 rows of two columns
        const bool odd = e.lane & 1;
        uint16_t* to = mat + static_cast<size_t>(x + odd) * p.out_pitch + y + (e.lane & ~1);
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const uint32_t other = __shfl_xor_sync(0xffffffffu, w[u], 1);
          const uint32_t both = odd ? __byte_perm(other, w[u], 0x7632) : __byte_perm(w[u], other, 0x5410);
          if (x + 2 * u + odd < p.N)  // rows past the last one end before the pitch
            *reinterpret_cast<uint32_t*>(to + static_cast<size_t>(2 * u) * p.out_pitch) = both;
        }
      }
    }
  }
};

// ---------------------------------------------------------------- the norm
// Elements [lo, hi) of G in pieces of 16 bytes with the ends that are not whole
// pieces taken one by one: a matrix may begin anywhere in a piece.
template <typename F, bool BF16>
__device__ __forceinline__ void for_elements(const void* G, size_t lo, size_t hi, int tid, int threads, F f) {
  constexpr int VE = BF16 ? 8 : 4;
  const size_t a = min((lo + VE - 1) / VE * VE, hi), b = max(a, hi / VE * VE);
  auto one = [&](size_t i) {
    f(i, BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(G)[i]) << 16)
              : static_cast<const float*>(G)[i]);
  };
  if (tid < static_cast<int>(a - lo)) one(lo + tid);
  if (tid < static_cast<int>(hi - b)) one(b + tid);
  for (size_t i = a + static_cast<size_t>(tid) * VE; i < b; i += static_cast<size_t>(threads) * VE) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(G) + i * (BF16 ? 2 : 4));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16) {
        f(i + 2 * k, bf16_lo(ws[k]));
        f(i + 2 * k + 1, bf16_hi(ws[k]));
      } else {
        f(i + k, __uint_as_float(ws[k]));
      }
    }
  }
}

// Elements of the part-th of `parts` parts of a matrix.
__device__ __forceinline__ void part_range(size_t n, int mat, int part, int parts, size_t& lo, size_t& hi) {
  const size_t per = (n + parts - 1) / parts;
  lo = static_cast<size_t>(mat) * n + min(n, per * part);
  hi = static_cast<size_t>(mat) * n + min(n, per * (part + 1));
}

// Sums of squares of the parts of each matrix.
template <bool BF16>
__global__ void __launch_bounds__(256) ortho_norm_kernel(const void* __restrict__ G, size_t n, int mats,
                                                         double* __restrict__ sums) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ double ws[8];
  const int parts = gridDim.x;
  for (int mat = blockIdx.y; mat < mats; mat += gridDim.y) {
    size_t lo, hi;
    part_range(n, mat, blockIdx.x, parts, lo, hi);
    float s = 0.f;
    auto add = [&](size_t, float v) { s = fmaf(v, v, s); };
    for_elements<decltype(add), BF16>(G, lo, hi, threadIdx.x, 256, add);
    double d = s;
#pragma unroll
    for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
      d = 0.;
      for (int i = 0; i < 8; ++i) d += ws[i];
      sums[static_cast<size_t>(mat) * parts + blockIdx.x] = d;
    }
    __syncthreads();
  }
}

// G to fp16 with its norm between 2^9 and 2^10, and what the first step makes of
// that.  A matrix of zeros, or so small beside eps that the steps are linear, or
// without a finite norm, is finished here.
template <bool BF16>
__global__ void __launch_bounds__(256)
    ortho_cast_kernel(const void* __restrict__ G, int rows, int cols, int pitch, int mats, const double* __restrict__ sums,
                      int steps, float* __restrict__ scal, __half* __restrict__ X, uint8_t* __restrict__ rest, uint16_t* __restrict__ O) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float shared_norm;
  const size_t n = static_cast<size_t>(rows) * cols;
  const int parts = gridDim.x;
  for (int mat = blockIdx.y; mat < mats; mat += gridDim.y) {
    if (threadIdx.x < 32) {
      double d = 0.;
      for (int i = threadIdx.x; i < parts; i += 32) d += sums[static_cast<size_t>(mat) * parts + i];
#pragma unroll
      for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      if (threadIdx.x == 0) shared_norm = norm_of(d);
    }
    __syncthreads();
    const float norm = shared_norm;
    __syncthreads();
    const float inv = 1.f / (norm + kNsEps);
    size_t lo, hi;
    part_range(n, mat, blockIdx.x, parts, lo, hi);
    const size_t at = static_cast<size_t>(mat) * n;
    if (!(norm * inv >= kTiny) || isinf(norm)) {  // also where the norm is NaN
      float f = isfinite(norm) ? inv : __uint_as_float(0x7fc00000u);
      for (int i = 0; i < steps; ++i) f *= kNsA;
      auto put = [&](size_t i, float v) { O[i] = static_cast<uint16_t>(pack_bf16(f * v, 0.f)); };
      if (isfinite(norm))
        for_elements<decltype(put), BF16>(G, lo, hi, threadIdx.x, 256, put);
      else
        for (size_t i = lo + threadIdx.x; i < hi; i += 256) O[i] = 0x7fc0;
      if (blockIdx.x == 0 && threadIdx.x == 0) scal[mat] = 0.f;
      continue;
    }
    int ex;
    frexpf(norm, &ex);
    const int k = kSXLog2 - ex;
    if (blockIdx.x == 0 && threadIdx.x == 0) scal[mat] = ldexpf(inv, -k);
    const float up = ldexpf(1.f, k);  // the norm is between 2^-104 and 2^64 here: 2^k is a normal number
    __half* Xm = X + static_cast<size_t>(mat) * rows * pitch;
    uint8_t* Lm = rest + static_cast<size_t>(mat) * rows * pitch;  // a bf16 G is fp16 exactly
    constexpr int VE = BF16 ? 8 : 4;
    if (cols % VE == 0) {  // whole 16-byte pieces of G in a row: one place for each
      const uint32_t v0 = static_cast<uint32_t>((lo - at + VE - 1) / VE), v1 = static_cast<uint32_t>((hi - at + VE - 1) / VE);
      const uint32_t vc = cols / VE;
      const uint4* from = reinterpret_cast<const uint4*>(G) + at / VE;
      for (uint32_t i = v0 + threadIdx.x; i < v1; i += 256) {
        const uint4 w = from[i];
        const uint32_t row = i / vc;
        __half* to = Xm + static_cast<size_t>(row) * pitch + (i - row * vc) * VE;
        if constexpr (BF16) {
          *reinterpret_cast<uint4*>(to) =
              make_uint4(pack_f16(up * bf16_lo(w.x), up * bf16_hi(w.x)), pack_f16(up * bf16_lo(w.y), up * bf16_hi(w.y)),
                         pack_f16(up * bf16_lo(w.z), up * bf16_hi(w.z)), pack_f16(up * bf16_lo(w.w), up * bf16_hi(w.w)));
        } else {
          const float x0 = up * __uint_as_float(w.x), x1 = up * __uint_as_float(w.y);
          const float x2 = up * __uint_as_float(w.z), x3 = up * __uint_as_float(w.w);
          const uint32_t h0 = pack_f16(x0, x1), h1 = pack_f16(x2, x3);
          *reinterpret_cast<uint2*>(to) = make_uint2(h0, h1);
          *reinterpret_cast<uint32_t*>(Lm + (to - Xm)) = rest_e4m3(x0, x1, h0) | rest_e4m3(x2, x3, h1) << 16;
        }
      }
    } else {
      auto put = [&](size_t i, float v) {
        const uint32_t j = static_cast<uint32_t>(i - at), row = j / cols;
        const size_t to = static_cast<size_t>(row) * pitch + (j - row * cols);
        const float x = up * v;
        const uint32_t h = pack_f16(x, 0.f);
        reinterpret_cast<uint16_t*>(Xm)[to] = static_cast<uint16_t>(h);
        if constexpr (!BF16) Lm[to] = static_cast<uint8_t>(rest_e4m3(x, 0.f, h));
      };
      for_elements<decltype(put), BF16>(G, lo, hi, threadIdx.x, 256, put);
    }
  }
}

// Padded rows of bf16 to the caller's, a warp a row; matrices that the cast
// finished are left alone.
__global__ void __launch_bounds__(256) ortho_rows_kernel(const uint16_t* __restrict__ X, const float* __restrict__ scal,
                                                         long long n, int rows, int cols, int pitch,
                                                         uint16_t* __restrict__ O) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  for (long long r = blockIdx.x * 8ll + (threadIdx.x >> 5); r < n; r += gridDim.x * 8ll) {
    if (scal[r / rows] == 0.f) continue;
    for (int c = lane; c < cols; c += 32) O[r * cols + c] = X[r * pitch + c];
  }
}

// ------------------------------------------------------------------ host
struct Plan {
  int small, pitch, spitch, parts;
  size_t err, sums, scal, X[2], lo, A, B, total;
};
Plan plan(int mats, int rows, int cols) {
  Plan p{};
  p.small = std::min(rows, cols);
  p.pitch = ceil_div(cols, 64) * 64;
  p.spitch = ceil_div(p.small, 64) * 64;
  const long long n = static_cast<long long>(rows) * cols;
  // enough for every SM where there are few matrices, 32,768 elements each else
  const long long few = std::min<long long>(n / 1024, 1216 / mats);
  p.parts = static_cast<int>(std::max(1ll, std::min<long long>(kNormParts, std::max(n / 32768, few))));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  p.err = take(kErrRegionBytes);
  p.sums = take(sizeof(double) * p.parts * mats);
  p.scal = take(sizeof(float) * mats);
  for (int i = 0; i < 2; ++i) p.X[i] = take(size_t(2) * mats * rows * p.pitch);
  p.lo = take(size_t(1) * mats * rows * p.pitch);
  p.A = take(size_t(2) * mats * p.small * p.spitch);
  p.B = take(size_t(2) * mats * p.small * p.spitch);
  p.total = o;
  return p;
}

}  // namespace

size_t ortho_workspace_bytes(int mats, int rows, int cols) { return plan(mats, rows, cols).total; }

int launch_ortho(const OrthoArgs& a, cudaStream_t s) {
  if (ortho_small(a.mats, a.rows, a.cols)) return launch_ortho_small(a, s);
  const Plan L = plan(a.mats, a.rows, a.cols);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  int* err = reinterpret_cast<int*>(ws + L.err);
  double* sums = reinterpret_cast<double*>(ws + L.sums);
  float* scal = reinterpret_cast<float*>(ws + L.scal);
  __half* X[2] = {reinterpret_cast<__half*>(ws + L.X[0]), reinterpret_cast<__half*>(ws + L.X[1])};
  uint8_t* lo = ws + L.lo;
  __half* A = reinterpret_cast<__half*>(ws + L.A);
  __half* B = reinterpret_cast<__half*>(ws + L.B);
  const bool bf = a.g_type == MOE_Y_BF16, wide = a.rows <= a.cols;
  const dim3 grid(L.parts, std::min(a.mats, 65535));
  {
    TraceScope trace_scope(MOE_K_ORTHO_NORM, s);
    const size_t n = static_cast<size_t>(a.rows) * a.cols;
    cudaError_t e = bf ? launch_pdl(ortho_norm_kernel<true>, grid, dim3(256), 0, s, a.G, n, a.mats, sums)
                       : launch_pdl(ortho_norm_kernel<false>, grid, dim3(256), 0, s, a.G, n, a.mats, sums);
    if (e == cudaSuccess)
      e = bf ? launch_pdl(ortho_cast_kernel<true>, grid, dim3(256), 0, s, a.G, a.rows, a.cols, L.pitch, a.mats, sums, a.steps,
                          scal, X[0], lo, a.O)
             : launch_pdl(ortho_cast_kernel<false>, grid, dim3(256), 0, s, a.G, a.rows, a.cols, L.pitch, a.mats, sums,
                          a.steps, scal, X[0], lo, a.O);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  const int m = L.small;
  // rows that are not whole 32-byte pieces come out padded and are then brought together
  const bool copy = a.cols % 16 != 0;
  auto base = [&](DenseParams& p, int code, int M, int N, int K) {
    p.M = M;
    p.N = N;
    p.nkb = ceil_div(K, kBK);
    p.run_kb = p.nkb;  // rounded to 16 bits
    p.code = kCodeOrtho + code;
    p.err = err;
  };
  const DenseShape gram_shape = dense_pick(m, m, a.mats, ceil_div(wide ? a.cols : a.rows, kBK), true, 1);
  const DenseShape square_shape = dense_pick(m, m, a.mats, ceil_div(m, kBK), true, 1);
  const DenseShape update_shape = dense_pick(a.rows, a.cols, a.mats, ceil_div(m, kBK), false, 1);
  const int upper = gram_shape.cg == 2 && square_shape.cg == 2;
  int rc = MOE_OK;
  for (int it = 0; it < a.steps && rc == MOE_OK; ++it) {
    const __half* Xi = X[it & 1];
    __half* Xo = X[(it + 1) & 1];
    const bool last = it + 1 == a.steps;
    const float shift = it >= a.steps - kShiftSteps ? kNsShift : 0.f;
    const float grown = std::pow(kNsA, static_cast<float>(it)), grows = grown * kNsA;
    auto gram = [&](auto& p) {
      std::memset(&p, 0, sizeof(p));
      base(p, 0, m, m, wide ? a.cols : a.rows);
      dense_shape(p, gram_shape.cg, gram_shape.tn, a.mats, true);
      p.scal = scal;
      p.first = it == 0;
      p.grown = grown;
      p.grows = grows;
      p.upper = upper;
      p.out = A;
      p.out_pitch = L.spitch;
      bool ok;
      if (wide)
        ok = dense_map_k(&p.tmA, Xi, true, a.cols, a.rows, a.mats, L.pitch, 128) &&
             dense_map_k(&p.tmB, Xi, true, a.cols, a.rows, a.mats, L.pitch, p.b_bytes / 128);
      else
        ok = dense_map_mn(&p.tmA, Xi, true, L.pitch, a.rows, a.mats, 2) &&
             dense_map_mn(&p.tmB, Xi, true, L.pitch, a.rows, a.mats, p.b_bytes / kBoxBytes);
      return ok;
    };
    if (wide) {
      OrthoOp<kGramWide>::Params p;
      rc = gram(p) ? dense_launch<OrthoOp<kGramWide>>(gram_shape.cg, p, a.grid_limit, MOE_K_ORTHO_GRAM, s) : MOE_ERR_CUDA;
    } else {
      OrthoOp<kGramTall>::Params p;
      rc = gram(p) ? dense_launch<OrthoOp<kGramTall>>(gram_shape.cg, p, a.grid_limit, MOE_K_ORTHO_GRAM, s) : MOE_ERR_CUDA;
    }
    if (rc != MOE_OK) break;
    {
      OrthoOp<kSquare>::Params p;
      std::memset(&p, 0, sizeof(p));
      base(p, 1, m, m, m);
      dense_shape(p, square_shape.cg, square_shape.tn, a.mats, true);
      p.scal = scal;
      p.upper = upper;
      p.old = A;
      p.shift = shift;
      p.pitch = L.spitch;
      if (!dense_map_k(&p.tmA, A, true, m, m, a.mats, L.spitch, 128) ||
          !dense_map_k(&p.tmB, A, true, m, m, a.mats, L.spitch, p.b_bytes / 128) ||
          !dense_map_mn(&p.tmT, A, true, L.spitch, m, a.mats, 2))
        return MOE_ERR_CUDA;
      p.out = B;
      p.out_pitch = L.spitch;
      if ((rc = dense_launch<OrthoOp<kSquare>>(square_shape.cg, p, a.grid_limit, MOE_K_ORTHO_SQUARE, s)) != MOE_OK) break;
    }
    auto update = [&](auto& p) {
      std::memset(&p, 0, sizeof(p));
      base(p, 2, a.rows, a.cols, m);
      dense_shape(p, update_shape.cg, update_shape.tn, a.mats, false);
      p.scal = scal;
      p.first = it == 0;
      p.grown = grown;
      p.grows = grows;
      p.upper = upper;
      p.old = Xi;
      p.lo = lo;
      p.lo_in = !last && (it > 0 || !bf);  // a bf16 G is fp16 exactly
      p.lo_out = it + 2 < a.steps;
      p.shift = shift;
      p.pitch = L.pitch;
      p.bf16 = last;
      p.out = last && !copy ? a.O : reinterpret_cast<uint16_t*>(Xo);
      p.out_pitch = last && !copy ? a.cols : L.pitch;
      p.apart = (reinterpret_cast<uintptr_t>(p.out) & 31) != 0;
      // rows of A of one CTA, or its columns of B
      bool ok = dense_map_mn(&p.tmT, B, true, L.spitch, m, a.mats, wide ? 2 : p.b_bytes / kBoxBytes);
      if (wide)
        ok = ok && dense_map_k(&p.tmA, B, true, m, m, a.mats, L.spitch, 128) &&
             dense_map_mn(&p.tmB, Xi, true, L.pitch, a.rows, a.mats, p.b_bytes / kBoxBytes);
      else
        ok = ok && dense_map_k(&p.tmA, Xi, true, a.cols, a.rows, a.mats, L.pitch, 128) &&
             dense_map_k(&p.tmB, B, true, m, m, a.mats, L.spitch, p.b_bytes / 128);
      return ok;
    };
    if (wide) {
      OrthoOp<kUpdateWide>::Params p;
      rc = update(p) ? dense_launch<OrthoOp<kUpdateWide>>(update_shape.cg, p, a.grid_limit, MOE_K_ORTHO_UPDATE, s) : MOE_ERR_CUDA;
    } else {
      OrthoOp<kUpdateTall>::Params p;
      rc = update(p) ? dense_launch<OrthoOp<kUpdateTall>>(update_shape.cg, p, a.grid_limit, MOE_K_ORTHO_UPDATE, s) : MOE_ERR_CUDA;
    }
  }
  if (rc == MOE_OK && copy) {
    TraceScope trace_scope(MOE_K_ORTHO_NORM, s);
    const long long n = static_cast<long long>(a.mats) * a.rows;
    if (launch_pdl(ortho_rows_kernel, dim3(static_cast<int>(std::min<long long>((n + 7) / 8, num_sms() * 8))), dim3(256), 0, s,
                   reinterpret_cast<const uint16_t*>(X[a.steps & 1]), scal, n, a.rows, a.cols, L.pitch,
                   a.O) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return rc;
}

}  // namespace moe
