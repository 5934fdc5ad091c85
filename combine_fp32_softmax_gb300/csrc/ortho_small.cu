// moe_orthogonalize for matrices whose smaller side is at most 128 (gate
// projections), in one launch: a cluster of CTAs holds a matrix, each CTA a slice
// of its long side in shared memory, for all steps.
//
// A step is: the slice's part of X X^T on the tensor cores; the parts added up
// over the cluster through distributed shared memory (each CTA adds its share of
// the entries, in the order of the CTAs, and gives the sums to all); then b A + c A A
// and a X + B X without leaving the CTA.  What bounds it is latency: two cluster
// barriers a step and the shared-memory passes between them.  The matrices are far
// too small for tcgen05's 128-row tiles and TMEM round trips (launched one by one
// the products of a 64 x 2048 matrix took 91 us); 16 x 16 pieces of mma.sync spread
// over eight warps fit them: it takes 40 us in this form.  fp16 values and their
// scales are those of ortho.cu.
//
// Up to a side of 48 (FINE) there is no averaging over many roundings, and a random
// square matrix has a singular value near 0 that the steps raise 485-fold: with fp16
// values a 4 x 4 matrix comes out off by 3e-3 of its norm in the middle and 6e-3 at
// the worst of 40.  X, A and B are then kept in two fp16 values each (22 bits) and every
// product has its two cross terms, on tensor cores that are idle otherwise: 1.6e-3,
// bf16's rounding, in the same 14 us; 32 x 2048 3.7e-3 -> 1.7e-3 in 27 us, 48 x 2048
// 2.7e-3 -> 1.7e-3 in 35 instead of 32 us.  (64 x 2048 would take 47 instead of 41 us for
// 2.2e-3 -> 1.7e-3, 112 x 2048 101 instead of 76.)
#include <algorithm>

#include <cuda_fp16.h>

#include "gemm_tiles.cuh"
#include "ortho.h"
#include "ortho.cuh"

namespace moe {
namespace {

constexpr int kSmallThreads = 256;
constexpr int kMaxCluster = 16;

// A CTA's shared memory may be written from its cluster once it has started: every
// CTA arrives first of all and waits, the norm's reads later, before it writes.
__device__ __forceinline__ void cluster_arrive_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_started() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster64(uint32_t a, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(v) : "memory");
}
// Four 8 x 8 blocks of 16-bit values, a row address a lane; TRANS: transposed.
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const __half* p) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p))
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p))
                 : "memory");
}
// c += a (16 x 16) . b (16 x 8)
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Row strides in shared memory: 16 bytes past a multiple of 32, so the eight rows
// of an ldmatrix block lie in different banks.
__host__ __device__ constexpr int half_stride(int n) { return n + 8; }
__host__ __device__ constexpr int sum_stride(int n) { return n + 4; }

struct SmallShape {
  int s, n;    // smaller and larger side
  int sp, nc;  // s rounded up to 16; columns of a slice, a multiple of 16
  int C;       // CTAs of a cluster
  int fine;    // two fp16 values each
};
constexpr int kFineSide = 48;
constexpr float kFineLo = 2048.f;  // scale of the second value beside the first
int small_smem(int sp, int nc, bool fine) {
  const int x = 2 * sp * half_stride(nc), ab = 2 * 2 * sp * half_stride(sp);
  return 256 + x + ab + 4 * sp * sum_stride(sp) + (fine ? x + ab : sp * nc);
}
// x to the two fp16 values of a pair each.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(x0, x1);
  const float2 h = unpack_f16(hi);
  lo = pack_f16(kFineLo * (x0 - h.x), kFineLo * (x1 - h.y));
}

// C = M . M^T (16 x 16 pieces on and above the diagonal, spread over the warps) for
// M [sp][k] with rows `stride` apart (FINE: and what it leaves, `low` elements
// further); put gets columns j and j + 1 of a row and whether its piece lies off the
// diagonal, so that the transposed entries are wanted too.
template <bool FINE, typename F>
__device__ __forceinline__ void gram_pieces(const __half* M, int low, int stride, int sp, int k, int warp, int lane, F put) {
  const int mt = sp / 16, pieces = mt * (mt + 1) / 2;
  for (int piece = warp; piece < pieces; piece += kSmallThreads / 32) {
    int mi = 0, j = piece;
    while (j >= mt - mi) j -= mt - mi++;
    const int ni = mi + j;
    float c[2][4] = {}, cross[2][4] = {};
    const __half* pa = M + (16 * mi + (lane & 15)) * stride + 8 * (lane >> 4);
    const __half* pb = M + (16 * ni + (lane & 7) + 8 * (lane >> 4)) * stride + 8 * ((lane >> 3) & 1);
    for (int kk = 0; kk < k; kk += 16) {
      uint32_t a[4], b[4];
      ldmatrix4<false>(a, pa + kk);
      ldmatrix4<false>(b, pb + kk);
      mma16816(c[0], a, b[0], b[1]);
      mma16816(c[1], a, b[2], b[3]);
      if constexpr (FINE) {
        uint32_t al[4], bl[4];
        ldmatrix4<false>(al, pa + low + kk);
        ldmatrix4<false>(bl, pb + low + kk);
        mma16816(cross[0], a, bl[0], bl[1]);
        mma16816(cross[1], a, bl[2], bl[3]);
        mma16816(cross[0], al, b[0], b[1]);
        mma16816(cross[1], al, b[2], b[3]);
      }
    }
    if constexpr (FINE)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int v = 0; v < 4; ++v) c[h][v] = fmaf(1.f / kFineLo, cross[h][v], c[h][v]);
    const int r = 16 * mi + (lane >> 2), col = 16 * ni + 2 * (lane & 3);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < 2; ++v) put(r + 8 * v, col + 8 * h, c[h][2 * v], c[h][2 * v + 1], mi != ni);
  }
}

template <bool BF16, bool FINE>
__global__ void __launch_bounds__(kSmallThreads)
    ortho_small_kernel(const void* __restrict__ G, uint16_t* __restrict__ O, int rows, int cols, SmallShape sh, int steps) {
  cluster_arrive_started();
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = sh.C, rank = static_cast<int>(cluster_ctarank()), sp = sh.sp, nc = sh.nc;
  const int xs = half_stride(nc), as = half_stride(sp), ps = sum_stride(sp);
  double* norms = reinterpret_cast<double*>(smem);  // one of each CTA
  __half* X = reinterpret_cast<__half*>(smem + 256);
  const int xlow = sp * xs, alow = sp * as;  // FINE: from a first value to the second
  __half* A = X + (FINE ? 2 : 1) * xlow;
  __half* B = A + (FINE ? 2 : 1) * alow;
  float* P = reinterpret_cast<float*>(B + (FINE ? 2 : 1) * alow);
  uint8_t* lo = reinterpret_cast<uint8_t*>(P + sp * ps);  // else: what rounding left of X
  __shared__ double wsum[kSmallThreads / 32];
  const size_t base = static_cast<size_t>(blockIdx.x / C) * rows * cols;
  const bool wide = rows <= cols;
  const int c0 = rank * nc, c1 = min(sh.n, c0 + nc);  // this slice of the long side
  auto at = [&](int i, int j) {                       // element i of the short side, j of the long one
    return base + (wide ? static_cast<size_t>(i) * cols + j : static_cast<size_t>(j) * cols + i);
  };
  auto load = [&](size_t i) {
    return BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(G)[i]) << 16)
                : static_cast<const float*>(G)[i];
  };
  // Neighbouring threads take neighbouring elements of G: along the long side of a
  // wide matrix, along the short one of a tall one.
  auto each = [&](auto f) {
    const int inner = wide ? max(0, c1 - c0) : sh.s, outer = wide ? sh.s : max(0, c1 - c0);
    if (inner > 0)
      for (int e = tid; e < inner * outer; e += kSmallThreads) {
        const int o = e / inner, i = e - o * inner;
        if (wide)
          f(o, c0 + i);
        else
          f(i, c0 + o);
      }
  };

  float sq = 0.f;
  each([&](int i, int j) {
    const float v = load(at(i, j));
    sq = fmaf(v, v, sq);
  });
  double d = sq;
#pragma unroll
  for (int off = 16; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
  if (lane == 0) wsum[warp] = d;
  for (int i = tid; i < (FINE ? 2 : 1) * xlow / 2; i += kSmallThreads) reinterpret_cast<uint32_t*>(X)[i] = 0u;  // padding too
  if (!FINE)
    for (int i = tid; i < sp * nc / 4; i += kSmallThreads) reinterpret_cast<uint32_t*>(lo)[i] = 0u;
  __syncthreads();
  cluster_wait_started();
  if (tid < C) {
    d = 0.;
    for (int w = 0; w < kSmallThreads / 32; ++w) d += wsum[w];
    st_cluster64(cluster_addr(norms + rank, tid), d);
  }
  cluster_sync();
  d = 0.;
  for (int r = 0; r < C; ++r) d += norms[r];
  const float norm = norm_of(d), inv = 1.f / (norm + kNsEps);
  if (!(norm * inv >= kTiny) || isinf(norm)) {  // the same in every CTA of the cluster
    float f = isfinite(norm) ? inv : __uint_as_float(0x7fc00000u);
    for (int i = 0; i < steps; ++i) f *= kNsA;
    each([&](int i, int j) {
      O[at(i, j)] = isfinite(norm) ? static_cast<uint16_t>(pack_bf16(f * load(at(i, j)), 0.f)) : 0x7fc0;
    });
    return;
  }
  int ex;
  frexpf(norm, &ex);
  const float up = ldexpf(1.f, kSXLog2 - ex);
  each([&](int i, int j) {
    const float x = up * load(at(i, j));
    uint32_t h, l;
    split2(x, 0.f, h, l);
    uint16_t* to = reinterpret_cast<uint16_t*>(X) + i * xs + j - c0;
    to[0] = static_cast<uint16_t>(h);
    if constexpr (FINE)
      to[xlow] = static_cast<uint16_t>(l);
    else
      lo[i * nc + j - c0] = static_cast<uint8_t>(rest_e4m3(x, 0.f, h));
  });
  __syncthreads();

  const float scal = ldexpf(inv, ex - kSXLog2);
  float grown = 1.f;  // kNsA to the power of the step
  for (int step = 0; step < steps; ++step) {
    const float r = step == 0 ? scal : step_scale(scal, grown);
    grown *= kNsA;
    const float shift = step >= steps - kShiftSteps ? kNsShift : 0.f;
    gram_pieces<FINE>(X, xlow, xs, sp, nc, warp, lane, [&](int i, int j, float a, float b, bool off) {
      *reinterpret_cast<float2*>(P + i * ps + j) = make_float2(a, b);
      if (off) {
        P[j * ps + i] = a;
        P[(j + 1) * ps + i] = b;
      }
    });
    cluster_sync();
    // this CTA's share of the entries, two at a time
    const float fa = r * r * kSA;
    const int pairs = sp * sp / 2, share = (pairs + C - 1) / C;
    for (int q = rank * share + tid; q < min(pairs, (rank + 1) * share); q += kSmallThreads) {
      const int i = 2 * q / sp, j = 2 * q - i * sp;
      float2 sum = make_float2(0.f, 0.f);
      for (int c = 0; c < C; ++c) {
        const float2 v = ld_cluster2(cluster_addr(P + i * ps + j, c));
        sum.x += v.x;
        sum.y += v.y;
      }
      uint32_t w, l;
      split2(fa * sum.x, fa * sum.y, w, l);
      for (int c = 0; c < C; ++c) {
        st_cluster(cluster_addr(A + i * as + j, c), w);
        if (FINE) st_cluster(cluster_addr(A + alow + i * as + j, c), l);
      }
    }
    cluster_sync();
    constexpr float fs2 = kNsC * (kSB / (kSA * kSA)), fo2 = kNsB * (kSB / kSA);
    gram_pieces<FINE>(A, alow, as, sp, sp, warp, lane, [&](int i, int j, float a, float b, bool off) {
      float2 o = unpack_f16(*reinterpret_cast<const uint32_t*>(A + i * as + j));
      if constexpr (FINE) {
        const float2 l = unpack_f16(*reinterpret_cast<const uint32_t*>(A + alow + i * as + j));
        o.x = fmaf(1.f / kFineLo, l.x, o.x);
        o.y = fmaf(1.f / kFineLo, l.y, o.y);
      }
      const float di = i == j ? shift * kSB : 0.f, dj = i == j + 1 ? shift * kSB : 0.f;
      uint32_t w[2];
      split2(fmaf(fo2, o.x, fmaf(fs2, a, di)), fmaf(fo2, o.y, fmaf(fs2, b, dj)), w[0], w[1]);
#pragma unroll
      for (int k = 0; k < (FINE ? 2 : 1); ++k) {
        uint16_t* to = reinterpret_cast<uint16_t*>(B) + k * alow;
        *reinterpret_cast<uint32_t*>(to + i * as + j) = w[k];
        if (off) {
          to[j * as + i] = static_cast<uint16_t>(w[k]);
          to[(j + 1) * as + i] = static_cast<uint16_t>(w[k] >> 16);
        }
      }
    });
    __syncthreads();
    const bool last = step + 1 == steps;
    const float ro = last ? r : r / step_scale(scal, grown), fs = ro / kSB, fo = (kNsA - shift) * ro;
    // a warp takes 16 columns: it reads all of theirs before it writes any
    for (int slab = warp; slab < nc / 16; slab += kSmallThreads / 32) {
      constexpr int MI = (FINE ? kFineSide : 128) / 16;
      float c[MI][2][4] = {}, cross[FINE ? MI : 1][2][4] = {};
      for (int kk = 0; kk < sp; kk += 16) {
        uint32_t b[4], bl[4];
        const __half* pb = X + (kk + (lane & 15)) * xs + 16 * slab + 8 * (lane >> 4);
        ldmatrix4<true>(b, pb);
        if constexpr (FINE) ldmatrix4<true>(bl, pb + xlow);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
          if (16 * mi < sp) {
            uint32_t a[4];
            const __half* pa = B + (16 * mi + (lane & 15)) * as + kk + 8 * (lane >> 4);
            ldmatrix4<false>(a, pa);
            mma16816(c[mi][0], a, b[0], b[1]);
            mma16816(c[mi][1], a, b[2], b[3]);
            if constexpr (FINE) {
              mma16816(cross[mi][0], a, bl[0], bl[1]);
              mma16816(cross[mi][1], a, bl[2], bl[3]);
              ldmatrix4<false>(a, pa + alow);
              mma16816(cross[mi][0], a, b[0], b[1]);
              mma16816(cross[mi][1], a, b[2], b[3]);
            }
          }
      }
      __syncwarp();
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
        if (16 * mi < sp)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int i = 16 * mi + (lane >> 2) + 8 * v, j = 16 * slab + 8 * h + 2 * (lane & 3);
              uint32_t* x = reinterpret_cast<uint32_t*>(X + i * xs + j);
              float2 o = unpack_f16(*x);
              uint32_t* xl = reinterpret_cast<uint32_t*>(X + (FINE ? xlow : 0) + i * xs + j);
              uint16_t* l = reinterpret_cast<uint16_t*>(lo + i * nc + j);
              float s0 = c[mi][h][2 * v], s1 = c[mi][h][2 * v + 1];
              if constexpr (FINE) {
                const float2 more = unpack_f16(*xl);
                o.x = fmaf(1.f / kFineLo, more.x, o.x);
                o.y = fmaf(1.f / kFineLo, more.y, o.y);
                s0 = fmaf(1.f / kFineLo, cross[mi][h][2 * v], s0);
                s1 = fmaf(1.f / kFineLo, cross[mi][h][2 * v + 1], s1);
              } else if (!last) {
                const float2 more = unpack_e4m3(*l);
                o.x = fmaf(1.f / kLo, more.x, o.x);
                o.y = fmaf(1.f / kLo, more.y, o.y);
              }
              const float y0 = fmaf(fo, o.x, fs * s0), y1 = fmaf(fo, o.y, fs * s1);
              if (!last) {
                uint32_t hi, low;
                split2(y0, y1, hi, low);
                *x = hi;
                if constexpr (FINE)
                  *xl = low;
                else
                  *l = static_cast<uint16_t>(rest_e4m3(y0, y1, hi));
              } else if (i < sh.s) {
                const uint32_t w = pack_bf16(y0, y1);
                if (c0 + j < c1) O[at(i, c0 + j)] = static_cast<uint16_t>(w);
                if (c0 + j + 1 < c1) O[at(i, c0 + j + 1)] = static_cast<uint16_t>(w >> 16);
              }
            }
    }
    __syncthreads();
  }
}

// The cluster's size: as many CTAs as have at least 64 columns each, while all
// matrices' clusters run at one time.  Sides up to kFineSide take this form for any
// number of matrices, a CTA each if need be.  False where the slices do not fit.
bool small_shape(int mats, int rows, int cols, SmallShape& sh) {
  sh.s = std::min(rows, cols);
  sh.n = std::max(rows, cols);
  if (sh.s > 128) return false;
  sh.sp = ceil_div(sh.s, 16) * 16;
  for (sh.C = kMaxCluster; sh.C >= 1; sh.C /= 2) {
    const bool wave = static_cast<long long>(mats) * sh.C <= 128 || (sh.C == 1 && sh.sp <= kFineSide);
    if (!wave || (sh.C > 1 && sh.n < 64 * sh.C)) continue;
    sh.nc = ceil_div(ceil_div(sh.n, sh.C), 16) * 16;
    sh.fine = sh.sp <= kFineSide && small_smem(sh.sp, sh.nc, true) <= kSmemBudget - 1024;
    return small_smem(sh.sp, sh.nc, sh.fine) <= kSmemBudget - 1024;
  }
  return false;
}

template <bool BF16, bool FINE>
int launch_small(const OrthoArgs& a, const SmallShape& sh, cudaStream_t s) {
  auto kern = ortho_small_kernel<BF16, FINE>;
  const int smem = small_smem(sh.sp, sh.nc, FINE);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget - 1024) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  set_pdl_attr(attr[0]);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(sh.C), 1, 1};
  cfg.blockDim = dim3(kSmallThreads);
  cfg.gridDim = dim3(sh.C * a.mats);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  TraceScope trace_scope(MOE_K_ORTHO_SMALL, s);
  return cudaLaunchKernelEx(&cfg, kern, a.G, a.O, a.rows, a.cols, sh, a.steps) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

bool ortho_small(int mats, int rows, int cols) {
  SmallShape sh;
  return small_shape(mats, rows, cols, sh);
}

int launch_ortho_small(const OrthoArgs& a, cudaStream_t s) {
  SmallShape sh;
  if (!small_shape(a.mats, a.rows, a.cols, sh)) return MOE_ERR_SHAPE;
  const bool bf = a.g_type == MOE_Y_BF16;
  if (sh.fine) return bf ? launch_small<true, true>(a, sh, s) : launch_small<false, true>(a, sh, s);
  return bf ? launch_small<true, false>(a, sh, s) : launch_small<false, false>(a, sh, s);
}

}  // namespace moe
