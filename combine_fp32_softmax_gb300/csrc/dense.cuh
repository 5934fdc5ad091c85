// Batched matrix products with the operation's own epilogue on tcgen05 tensor
// cores: C[i] = A[i] . B[i]^T, 16-bit operands, fp32 sums.
//
// One persistent kernel per operation; CG = 2 runs it on CTA pairs (a 256 x 256
// tile of C for each pair, tcgen05 MMAs of the CTA group of two), CG = 1 on
// single CTAs (128 x 256), for products whose C has at most 128 rows: half of
// a pair's tile would be empty there.  384 threads:
//   warp 0      TMA producer, 64-deep K blocks through a ring of 192 KB;
//   warp 1      issues the MMAs (warps 2 and 3 fill up their warpgroup, whose
//               registers go to the other two);
//   warps 4-11  epilogue: two warps for each TMEM lane quadrant, so a thread has
//               one row and 128 of its 256 columns, all of them in registers.
// The sums of a tile are taken out of TMEM in runs of run_kb K blocks and
// added up in registers, rounded to nearest: the tensor core's own fp32
// additions cut off what a sum has no room for, and an operation whose results
// are kept in fp32 keeps those runs short (the other accumulator fills
// meanwhile, so this costs the tensor core nothing).  An operation whose
// results are rounded to 16 bits takes one run.
//
// Matrices are seen by TMA as [matrix][row][column] with the exact number of
// rows, so tiles that reach past an end read zeros and their stores are cut:
// no tail code.  Rows are padded to 64 columns in the library's own buffers;
// the callers' have widths that are multiples of 64.
#pragma once
#include "gemm_tiles.cuh"

namespace moe {
namespace {

constexpr int kDenseThreads = 128 + 32 * 8;
// Registers a thread: 168 at launch (384 of them fill the SM's 65,536), then 40 for
// the first warpgroup and 232 for the epilogue's two: 40 + 2 * 232 = 3 * 168.
constexpr int kDenseRegs = 168, kIssueRegs = 40, kEpiRegs = 232;
static_assert(kIssueRegs + 2 * kEpiRegs == 3 * kDenseRegs && kDenseRegs * kDenseThreads <= 65536, "register shares");
constexpr int kDenseStg = 2 * kChunkBytes;  // staging of one epilogue warp: two chunks in flight
template <int CG>
struct DensePipe {
  static constexpr int STAGES = CG == 1 ? 4 : 6;
  static constexpr int B_BYTES = kBBytes / CG;
  static constexpr int STAGE_BYTES = kABytes + B_BYTES;
  static constexpr int TILE_M = kBM * CG;
};
struct DenseState {
  uint64_t full[6], empty[6], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kDenseSmem = 6 * DensePipe<2>::STAGE_BYTES + 8 * kDenseStg + static_cast<int>(sizeof(DenseState));
static_assert(DensePipe<1>::STAGES * DensePipe<1>::STAGE_BYTES == DensePipe<2>::STAGES * DensePipe<2>::STAGE_BYTES,
              "one shared-memory layout for both");
static_assert(kDenseSmem <= kSmemBudget, "shared memory budget of one CTA");

// What every operation's launch has.
struct DenseParams {
  CUtensorMap tmA, tmB;  // operands
  CUtensorMap tmO;       // what the epilogue stores by TMA
  int M, N;              // rows and columns of C
  int mt, nt;            // tiles of its rows (of TILE_M) and columns (of tn)
  int tn;                // columns of a tile: 256, on single CTAs also fewer (a multiple of 16)
  int b_bytes;           // of B in one CTA's part of a stage
  int nkb;               // K blocks
  int run_kb;            // K blocks of a run of sums
  int total;             // tiles of the launch
  int code;              // names the operation in the error word of a wait that ran out
  int* err;
};

// This CTA's part of a tile.
struct DenseTile {
  int mat, m0, n0;  // matrix, first row (of this CTA) and column
  int kb0, kb1;     // its K blocks
};
// Columns of C in a tile, and the N of its MMAs: a last tile with fewer columns
// takes less of the tensor core's time.  A pair's CTAs hold half of them each, in
// whole groups of 64 where B is MN-major.
__device__ __forceinline__ int dense_cols(const DenseParams& p, const DenseTile& t) { return min(p.tn, p.N - t.n0); }
template <int CG, bool B_MN>
__device__ __forceinline__ int dense_mma_n(const DenseParams& p, const DenseTile& t) {
  constexpr int unit = CG == 1 ? 16 : B_MN ? 128 : 64;
  return (dense_cols(p, t) + unit - 1) / unit * unit;
}

struct DenseEpi {
  uint8_t* stg;
  uint32_t chunks = 0;  // staged chunks so far
  int lane, q, part;
};

// Stages the warp's 32 rows x 64 bytes (16 words of each lane's row) and stores
// them at column x, row y of matrix z; what lies outside is cut off.
__device__ __forceinline__ void dense_store(DenseEpi& e, const uint32_t* w, const CUtensorMap* map, int x, int y, int z) {
  uint8_t* buf = e.stg + (e.chunks & 1) * kChunkBytes;
  staging_reuse_wait<1>(e.chunks);
  stage_row64(buf, e.lane, w);
  staging_publish();
  if (e.lane == 0) {
    tma_store_3d(map, buf, x, y, z);
    bulk_commit();
  }
  ++e.chunks;
}

// mbar_wait without a call: an epilogue thread holds 128 sums that a call would
// have to save.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int where) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (int i = 1; !mbar_try_wait(a, parity); ++i) {
    if (i & 63) continue;
    if (t0 == 0) t0 = globaltimer_ns();
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, MOE_ERR_TIMEOUT_CODE, where);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// One stage of loads.
template <class Op, int CG>
__device__ __forceinline__ void dense_loads(const typename Op::Params& p, const DenseTile& t, int kb, int b_off,
                                            uint8_t* sA, uint8_t* sB, uint64_t* bar, int rank) {
  int ak, am, bk, bn;
  Op::coords(p, t, kb, ak, am, bk, bn);
  bn += b_off;
  const bool to_even = CG == 2 && rank == 1;
  const int mat = Op::ONE ? 0 : t.mat;  // ONE: a single A and B, t.mat tells results apart
  if constexpr (Op::A_MN) {
    if (to_even)
      tma_load_4d_to_even(sA, &p.tmA, bar, 0, ak, am / 64, mat);
    else
      tma_load_4d(sA, &p.tmA, bar, 0, ak, am / 64, mat);
  } else {
    if (to_even)
      tma_load_3d_to_even(sA, &p.tmA, bar, ak, am, mat);
    else
      tma_load_3d(sA, &p.tmA, bar, ak, am, mat);
  }
  if constexpr (Op::B_MN) {
    if (to_even)
      tma_load_4d_to_even(sB, &p.tmB, bar, 0, bk, bn / 64, mat);
    else
      tma_load_4d(sB, &p.tmB, bar, 0, bk, bn / 64, mat);
  } else {
    if (to_even)
      tma_load_3d_to_even(sB, &p.tmB, bar, bk, bn, mat);
    else
      tma_load_3d(sB, &p.tmB, bar, bk, bn, mat);
  }
}

template <class Op, int CG>
__global__ void __launch_bounds__(kDenseThreads, 1) dense_kernel(const __grid_constant__ typename Op::Params p) {
  using Pipe = DensePipe<CG>;
  constexpr int NST = Pipe::STAGES, SB = Pipe::STAGE_BYTES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {  // as in grouped_gemm_kernel: reported, never computed on
    if (threadIdx.x == 0) record_error(p.err, MOE_ERR_CUDA, 0x5A11);
    return;
  }
  uint8_t* smem = smem_raw;
  uint8_t* stg_base = smem + NST * SB;
  DenseState& ss = *reinterpret_cast<DenseState*>(stg_base + 8 * kDenseStg);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&ss.full[s], 1);
      mbar_init(&ss.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ss.tfull[a], 1);
      mbar_init(&ss.tempty[a], 8 * CG);
    }
    mbar_init(&ss.drain, 1);
    ss.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<CG>(&ss.tmem_base, kTmemCols);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = ss.tmem_base;
  volatile int* abort = &ss.abort;
  const int first = CG == 2 ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int step = CG == 2 ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int where0 = p.code << 24 | rank << 23;
  auto where = [&](int role, int i) { return where0 | role << 20 | (i & 0xfffff); };

  if (warp < 4) {
    regs_give<kIssueRegs>();
    if (warp == 0 && lane == 0) {
      tma_prefetch_desc(&p.tmA);
      tma_prefetch_desc(&p.tmB);
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_par = 0;
      bool ok = true;
      for (int i = first; ok && i < p.total && !*abort; i += step) {
        const DenseTile t = Op::template tile<CG>(p, i, rank);
        const int b_off = CG == 2 ? rank * dense_mma_n<CG, Op::B_MN>(p, t) / 2 : 0;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!mbar_wait(&ss.empty[stage], phase ^ 1, abort, p.err, where(0, i))) {
            ok = false;
            break;
          }
          uint8_t* sA = smem + stage * SB;
          // a pair's loads are all counted on the even CTA's barrier
          if (rank == 0) {
            mbar_arrive_expect_tx(&ss.full[stage], CG * (kABytes + p.b_bytes));
            filled |= 1u << stage;
            fill_par = (fill_par & ~(1u << stage)) | phase << stage;
          }
          dense_loads<Op, CG>(p, t, kb, b_off, sA, sA + kABytes, &ss.full[stage], rank);
          if (++stage == NST) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort)
        for (int s = 0; s < NST; ++s)
          if (filled & (1u << s)) mbar_wait_drain(&ss.full[s], (fill_par >> s) & 1);
    }
    __syncwarp();
    if (warp == 1 && rank == 0) {
      constexpr uint32_t idesc0 = Op::F16 ? idesc_f16_f32(kBM * CG, 0, Op::A_MN ? 1 : 0, Op::B_MN ? 1 : 0)
                                          : idesc_bf16_f32(kBM * CG, 0, Op::A_MN ? 1 : 0, Op::B_MN ? 1 : 0);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      for (int i = first; ok && i < p.total && !*abort; i += step) {
        const DenseTile t = Op::template tile<CG>(p, i, rank);
        const uint32_t idesc = idesc0 | static_cast<uint32_t>(dense_mma_n<CG, Op::B_MN>(p, t) >> 3) << 17;
        int left = 0;  // K blocks left of the run
        uint32_t dtm = 0;
        for (int kb = t.kb0; ok && kb < t.kb1; ++kb) {
          const bool fresh = left == 0;
          if (fresh) {
            ok = mbar_wait<CG == 2>(&ss.tempty[it & 1], ((it >> 1) & 1) ^ 1, abort, p.err, where(2, i));
            if (!ok) break;
            tc_fence_after();
            dtm = tmem + (it & 1) * kBN;
            left = min(p.run_kb, t.kb1 - kb);
          }
          ok = mbar_wait(&ss.full[stage], phase, abort, p.err, where(3, i));
          if (!ok) break;
          tc_fence_after();
          --left;
          if (lane == 0) {
            const uint32_t a0 = smem_u32(smem + stage * SB), b0 = a0 + kABytes;
#pragma unroll
            for (int k4 = 0; k4 < kBK / 16; ++k4) {
              const uint64_t ad = Op::A_MN ? smem_desc_sw128(a0 + k4 * 2048, kBoxBytes, 1024)
                                           : smem_desc_sw128(a0 + k4 * 32, 16, 1024);
              const uint64_t bd = Op::B_MN ? smem_desc_sw128(b0 + k4 * 2048, kBoxBytes, 1024)
                                           : smem_desc_sw128(b0 + k4 * 32, 16, 1024);
              umma_bf16<CG>(dtm, ad, bd, idesc, !(fresh && k4 == 0));
            }
            if constexpr (CG == 2)
              umma_commit_pair(&ss.empty[stage]);
            else
              umma_commit(&ss.empty[stage]);
            if (left == 0) {
              if constexpr (CG == 2)
                umma_commit_pair(&ss.tfull[it & 1]);
              else
                umma_commit(&ss.tfull[it & 1]);
            }
            issued = true;
          }
          __syncwarp();
          if (left == 0) ++it;
          if (++stage == NST) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort) {
        if (lane == 0 && issued) {
          umma_commit<CG>(&ss.drain);
          mbar_wait_drain(&ss.drain, 0);
        }
        __syncwarp();
      }
    }
  } else {
    regs_take<kEpiRegs>();
    DenseEpi e;
    e.stg = stg_base + (warp - 4) * kDenseStg;
    e.lane = lane;
    e.q = warp & 3;  // TMEM lanes [32q, 32q + 32) are reachable from this warp
    e.part = (warp - 4) >> 2;
    int it = 0;
    bool ok = true;
    for (int i = first; ok && i < p.total && !*abort; i += step) {
      const DenseTile t = Op::template tile<CG>(p, i, rank);
      const bool active = t.m0 + 32 * e.q < p.M;
      const auto pre = Op::pre(p, t, e);
      uint32_t acc[4][32];
      const int runs = (t.kb1 - t.kb0 + p.run_kb - 1) / p.run_kb;
      if (runs == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c][j] = 0u;
      }
#pragma unroll 1
      for (int r = 0; r < runs; ++r) {
        const int buf = it & 1;
        if (!mbar_wait_inline(&ss.tfull[buf], (it >> 1) & 1, abort, p.err, where(4, i))) {
          ok = false;
          break;
        }
        ++it;
        tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(e.q * 32) << 16) + buf * kBN + e.part * 128;
        if (r == 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32(ta + 32 * c, acc[c]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld_32x32(ta + 32 * c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              acc[c][j] = __float_as_uint(__uint_as_float(acc[c][j]) + __uint_as_float(v[j]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && rank == 1)
            mbar_arrive_rank(&ss.tempty[buf], 0);
          else
            mbar_arrive(&ss.tempty[buf]);
        }
      }
      if (ok && active) Op::epilogue(p, t, e, pre, acc);
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  // No CTA of a pair leaves while the other may still arrive on its barriers
  // or have MMAs read its shared memory.
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<CG>(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host
constexpr int kDenseDevices = 64;

// CTA pairs (CG = 2) or CTAs that are resident at once; the attributes of the
// kernel are set the first time on each device.
template <class Op, int CG>
int dense_resident() {
  static int cached[kDenseDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDenseDevices) return 0;
  if (cached[dev] > 0) return cached[dev];
  auto kern = dense_kernel<Op, CG>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDenseSmem) != cudaSuccess) return 0;
  int n = num_sms();
  if constexpr (CG == 2) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.blockDim = dim3(kDenseThreads);
    cfg.gridDim = dim3(2 * (n / 2));
    cfg.dynamicSmemBytes = kDenseSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return 0;
  }
  return cached[dev] = n;
}

template <class Op, int CG>
int dense_launch(typename Op::Params& p, int grid_limit, int trace, cudaStream_t s) {
  if (p.tn == 0) {  // whole tiles
    p.tn = kBN;
    p.b_bytes = DensePipe<CG>::B_BYTES;
  }
  const int resident = dense_resident<Op, CG>();
  if (resident <= 0) return MOE_ERR_CUDA;
  int units = resident;
  if (grid_limit > 0) units = std::min(units, std::max(1, grid_limit / CG));
  units = std::min(units, p.total);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  set_pdl_attr(attr[0]);
  cfg.numAttrs = 1;
  if constexpr (CG == 2) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {2, 1, 1};
    cfg.numAttrs = 2;
  }
  cfg.blockDim = dim3(kDenseThreads);
  cfg.gridDim = dim3(CG * units);
  cfg.dynamicSmemBytes = kDenseSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  TraceScope trace_scope(trace, s);
  return cudaLaunchKernelEx(&cfg, dense_kernel<Op, CG>, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Matrices [mats][rows][cols] of 16-bit elements, rows `pitch` elements apart, as
// K-major operand tiles: boxes of 64 columns x box_rows rows.
bool dense_map_k(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t mats, uint64_t pitch,
                 uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, mats};
  const cuuint64_t strides[2] = {pitch * 2, rows * pitch * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The same matrices (cols a multiple of 64) as MN-major tiles: boxes of 64 rows x
// `chunks` groups of 64 columns (see map3d_mn).
bool dense_map_mn(CUtensorMap* m, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t mats, uint32_t chunks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || cols % 64) return false;
  const cuuint64_t dims[4] = {64, rows, cols / 64, mats};
  const cuuint64_t strides[3] = {cols * 2, 128, rows * cols * 2};
  const cuuint32_t box[4] = {64, 64, chunks, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// What epilogues store: chunks of 32 rows x 64 bytes.
bool dense_map_out(CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t cols, uint64_t rows, uint64_t mats,
                   uint64_t pitch) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint32_t es = dt == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
  const cuuint64_t dims[3] = {cols, rows, mats};
  const cuuint64_t strides[2] = {pitch * es, rows * pitch * es};
  const cuuint32_t box[3] = {64 / es, 32, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe
