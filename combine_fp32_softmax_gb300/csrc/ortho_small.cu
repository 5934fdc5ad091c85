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
// over eight warps fit them.  fp16 values and their scales are those of ortho.cu.
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
};
int small_smem(int sp, int nc) {
  return 256 + 2 * sp * half_stride(nc) + 2 * 2 * sp * half_stride(sp) + 4 * sp * sum_stride(sp) + sp * nc;
}

// C = M . M^T (16 x 16 pieces on and above the diagonal, spread over the warps) for
// M [sp][k] with rows `stride` apart; put(row, column, value pair) gets columns
// j and j + 1 of a row, and each piece's transposed ones by put1.
template <typename F>
__device__ __forceinline__ void gram_pieces(const __half* M, int stride, int sp, int k, int warp, int lane, F put) {
  const int mt = sp / 16, pieces = mt * (mt + 1) / 2;
  for (int piece = warp; piece < pieces; piece += kSmallThreads / 32) {
    int mi = 0, j = piece;
    while (j >= mt - mi) j -= mt - mi++;
    const int ni = mi + j;
    float c[2][4] = {};
    const __half* pa = M + (16 * mi + (lane & 15)) * stride + 8 * (lane >> 4);
    const __half* pb = M + (16 * ni + (lane & 7) + 8 * (lane >> 4)) * stride + 8 * ((lane >> 3) & 1);
    for (int kk = 0; kk < k; kk += 16) {
      uint32_t a[4], b[4];
      ldmatrix4<false>(a, pa + kk);
      ldmatrix4<false>(b, pb + kk);
      mma16816(c[0], a, b[0], b[1]);
      mma16816(c[1], a, b[2], b[3]);
    }
    const int r = 16 * mi + (lane >> 2), col = 16 * ni + 2 * (lane & 3);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int v = 0; v < 2; ++v) put(r + 8 * v, col + 8 * h, c[h][2 * v], c[h][2 * v + 1], mi != ni);
  }
}

template <bool BF16>
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
  __half* A = X + sp * xs;
  __half* B = A + sp * as;
  float* P = reinterpret_cast<float*>(B + sp * as);
  uint8_t* lo = reinterpret_cast<uint8_t*>(P + sp * ps);  // what rounding left of X
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
  for (int i = tid; i < sp * xs / 2; i += kSmallThreads) reinterpret_cast<uint32_t*>(X)[i] = 0u;  // padding too
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
  const float norm = static_cast<float>(sqrt(d)), inv = 1.f / (norm + kNsEps);
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
    const uint32_t h = pack_f16(x, 0.f);
    reinterpret_cast<uint16_t*>(X)[i * xs + j - c0] = static_cast<uint16_t>(h);
    lo[i * nc + j - c0] = static_cast<uint8_t>(rest_e4m3(x, 0.f, h));
  });
  __syncthreads();

  const float scal = ldexpf(inv, ex - kSXLog2);
  float grown = 1.f;  // kNsA to the power of the step
  for (int step = 0; step < steps; ++step) {
    const float r = step == 0 ? scal : step_scale(scal, grown);
    grown *= kNsA;
    const float shift = step >= steps - kShiftSteps ? kNsShift : 0.f;
    gram_pieces(X, xs, sp, nc, warp, lane, [&](int i, int j, float a, float b, bool off) {
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
      const uint32_t w = pack_f16(fa * sum.x, fa * sum.y);
      for (int c = 0; c < C; ++c) st_cluster(cluster_addr(A + i * as + j, c), w);
    }
    cluster_sync();
    constexpr float fs2 = kNsC * (kSB / (kSA * kSA)), fo2 = kNsB * (kSB / kSA);
    gram_pieces(A, as, sp, sp, warp, lane, [&](int i, int j, float a, float b, bool off) {
      const float2 o = __half22float2(*reinterpret_cast<const __half2*>(A + i * as + j));
      const float di = i == j ? shift * kSB : 0.f, dj = i == j + 1 ? shift * kSB : 0.f;
      const __half2 v = __floats2half2_rn(fmaf(fo2, o.x, fmaf(fs2, a, di)), fmaf(fo2, o.y, fmaf(fs2, b, dj)));
      *reinterpret_cast<__half2*>(B + i * as + j) = v;
      if (off) {
        B[j * as + i] = __low2half(v);
        B[(j + 1) * as + i] = __high2half(v);
      }
    });
    __syncthreads();
    const bool last = step + 1 == steps;
    const float ro = last ? r : r / step_scale(scal, grown), fs = ro / kSB, fo = (kNsA - shift) * ro;
    // a warp takes 16 columns: it reads all of theirs before it writes any
    for (int slab = warp; slab < nc / 16; slab += kSmallThreads / 32) {
      float c[8][2][4] = {};
      for (int kk = 0; kk < sp; kk += 16) {
        uint32_t b[4];
        ldmatrix4<true>(b, X + (kk + (lane & 15)) * xs + 16 * slab + 8 * (lane >> 4));
#pragma unroll
        for (int mi = 0; mi < 8; ++mi)
          if (16 * mi < sp) {
            uint32_t a[4];
            ldmatrix4<false>(a, B + (16 * mi + (lane & 15)) * as + kk + 8 * (lane >> 4));
            mma16816(c[mi][0], a, b[0], b[1]);
            mma16816(c[mi][1], a, b[2], b[3]);
          }
      }
      __syncwarp();
#pragma unroll
      for (int mi = 0; mi < 8; ++mi)
        if (16 * mi < sp)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int i = 16 * mi + (lane >> 2) + 8 * v, j = 16 * slab + 8 * h + 2 * (lane & 3);
              __half2* x = reinterpret_cast<__half2*>(X + i * xs + j);
              float2 o = __half22float2(*x);
              uint16_t* l = reinterpret_cast<uint16_t*>(lo + i * nc + j);
              if (!last) {
                const float2 more = unpack_e4m3(*l);
                o.x = fmaf(1.f / kLo, more.x, o.x);
                o.y = fmaf(1.f / kLo, more.y, o.y);
              }
              const float y0 = fmaf(fo, o.x, fs * c[mi][h][2 * v]), y1 = fmaf(fo, o.y, fs * c[mi][h][2 * v + 1]);
              if (!last) {
                const uint32_t h = pack_f16(y0, y1);
                *reinterpret_cast<uint32_t*>(x) = h;
                *l = static_cast<uint16_t>(rest_e4m3(y0, y1, h));
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
// matrices' clusters run at one time; 0 where the slices do not fit or there are
// more matrices than that.
bool small_shape(int mats, int rows, int cols, SmallShape& sh) {
  sh.s = std::min(rows, cols);
  sh.n = std::max(rows, cols);
  if (sh.s > 128) return false;
  sh.sp = ceil_div(sh.s, 16) * 16;
  for (sh.C = kMaxCluster; sh.C >= 1; sh.C /= 2) {
    if (static_cast<long long>(mats) * sh.C > 128 || (sh.C > 1 && sh.n < 64 * sh.C)) continue;
    sh.nc = ceil_div(ceil_div(sh.n, sh.C), 16) * 16;
    return small_smem(sh.sp, sh.nc) <= kSmemBudget - 1024;
  }
  return false;
}

template <bool BF16>
int launch_small(const OrthoArgs& a, const SmallShape& sh, cudaStream_t s) {
  auto kern = ortho_small_kernel<BF16>;
  const int smem = small_smem(sh.sp, sh.nc);
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
  return a.g_type == MOE_Y_BF16 ? launch_small<true>(a, sh, s) : launch_small<false>(a, sh, s);
}

}  // namespace moe
