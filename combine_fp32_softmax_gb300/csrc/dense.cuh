// Batched matrix products with the operation's own epilogue on tcgen05 tensor
// cores: C[i] = A[i] . B[i]^T, 16-bit operands, fp32 sums.
//
// One persistent kernel per operation; CG = 2 runs it on CTA pairs (a 256 x 256
// tile of C for each pair, tcgen05 MMAs of the CTA group of two), CG = 1 on
// single CTAs (128 rows x up to 256 columns), for products that would leave
// pairs without work (dense_pick).  384 threads:
//   warp 0      loads A by TMA, 64-deep K blocks through a ring of 224 KB;
//   warp 1      issues the MMAs;
//   warp 2      loads B (warp 3 fills up the warpgroup, whose registers go to the
//               other two);
//   warps 4-11  epilogue: two warps for each TMEM lane quadrant, so a thread has
//               one row and 128 of its 256 columns, all of them in registers.
// The sums of a tile are taken out of TMEM in runs of run_kb K blocks and
// added up in registers, rounded to nearest: the tensor core's own fp32
// additions cut off what a sum has no room for, and an operation whose results
// are kept in fp32 keeps those runs short (the other accumulator fills
// meanwhile; what it costs stands at the operations).  An operation whose
// results are rounded to 16 bits takes one run or a few long ones, and with one may
// have its sums 32 columns at a time (CHUNKS), which leaves it registers for what it
// reads beside them.
//
// Matrices are seen by TMA as [matrix][row][column] with the exact number of
// rows, so tiles that reach past an end read zeros and their stores are cut:
// no tail code.  Rows are padded to 64 columns in the library's own buffers;
// the callers' have widths that are multiples of 64.
#pragma once
#include <type_traits>

#include "gemm_tiles.cuh"

namespace moe {
namespace {

constexpr int kDenseThreads = 128 + 32 * 8;
// Registers a thread: 168 at launch (384 of them fill the SM's 65,536), then 56 for
// the first warpgroup and 224 for the epilogue's two: 56 + 2 * 224 = 3 * 168.
constexpr int kDenseRegs = 168, kIssueRegs = 56, kEpiRegs = 224;
static_assert(kIssueRegs + 2 * kEpiRegs == 3 * kDenseRegs && kDenseRegs * kDenseThreads <= 65536, "register shares");
// The ring takes nearly all shared memory (the epilogue stores from registers):
// seven stages of 32 KB on pairs, as many as fit of what a K block takes on single
// CTAs.
constexpr int kDenseRing = 7 * (kABytes + kBBytes / 2);
constexpr int kDenseMaxStages = 14;
constexpr uint64_t kDrainNs = 2000000;  // after a wait that ran out
struct DenseState {
  uint64_t full[kDenseMaxStages], empty[kDenseMaxStages], tfull[2], tempty[2], drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kDenseSmem = kDenseRing + static_cast<int>(sizeof(DenseState));
static_assert(kDenseSmem <= kSmemBudget, "shared memory budget of one CTA");

// What every operation's launch has.
struct DenseParams {
  CUtensorMap tmA, tmB;  // operands
  CUtensorMap tmT;       // a symmetric operand's MN-major view (see dense_flip)
  int M, N;              // rows and columns of C
  int mt, nt;            // tiles of its rows (128 for each CTA) and columns (of tn)
  int tn;                // columns of a tile: 256, on single CTAs also fewer (a multiple of 16)
  int half;              // columns of a tile that the first half of the epilogue's warps takes, a multiple of 32
  int a_bytes, b_bytes;  // of A and B in one CTA's part of a stage
  int nst;               // stages of the ring
  int nkb;               // K blocks
  int run_kb;            // K blocks of a run of sums
  int upper;             // a symmetric operand holds only its tiles from the diagonal on
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
  constexpr int unit = CG == 1 ? 16 : B_MN ? 128 : 64;  // B_MN: for some K blocks at least
  return (dense_cols(p, t) + unit - 1) / unit * unit;
}

// Of a symmetric matrix only the 256 x 256 tiles on and above the diagonal need be
// stored: an operand's rows of a lower tile are the columns of an upper one, read
// as an MN-major tile.  True where K block kb of the rows from `row` on is such a
// one.
__device__ __forceinline__ bool dense_flip(const DenseParams& p, int kb, int row) {
  return p.upper && kb * kBK / kBN < row / kBN;
}

// Where an epilogue thread stands: lane of its warp, TMEM lane quadrant, half of
// the columns.
struct DenseEpi {
  int lane, q, part;
};

// First column of C of an epilogue thread, and how many it has (0 or less: none).
__device__ __forceinline__ int dense_col(const DenseParams& p, const DenseTile& t, const DenseEpi& e) {
  return t.n0 + p.half * e.part;
}
__device__ __forceinline__ int dense_width(const DenseParams& p, const DenseTile& t, const DenseEpi& e) {
  return min(p.half, dense_cols(p, t) - p.half * e.part);
}

// 32 bytes from or to a 32-byte boundary: whole sectors, one row a lane.
__device__ __forceinline__ void st_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void ld_32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
// Two 16-byte halves where a caller's array does not begin on a 32-byte boundary.
__device__ __forceinline__ void st_2x16(void* p, const uint32_t* w) {
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Arrives on `bar` (in both CTAs of a pair) when the MMAs that the lane with
// `lead` issued before are done.
template <int CG>
__device__ __forceinline__ void dense_commit(uint32_t lead, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(
            bar),
        "r"(lead), "h"(static_cast<uint16_t>(3))
        : "memory");
}
// The four MMAs (16 deep each) of a K block and the release of its stage, from
// the lane with `lead`.  a and b: shared-memory addresses / 16 of the tiles, each
// MN-major or K-major; the first MMA overwrites C unless `add`.
template <int CG>
__device__ __forceinline__ void dense_mma(uint32_t lead, uint32_t d, uint32_t a, uint32_t b, bool a_mn, bool b_mn,
                                          uint32_t idesc, bool add, uint32_t empty) {
  // descriptor words as in smem_desc_sw128: leading byte offset above the address,
  // stride byte offset, version and swizzle in the upper word
  constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;
  const uint32_t alo = a | (a_mn ? kBoxBytes >> 4 : 1u) << 16, blo = b | (b_mn ? kBoxBytes >> 4 : 1u) << 16;
  const uint32_t sa = a_mn ? 128 : 2, sb = b_mn ? 128 : 2;  // 16 elements of K further
  idesc |= (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
#define MOE_DENSE_MMA(GROUP)                                                                                         \
  asm volatile(                                                                                                      \
      "{\n\t.reg .pred q, f, t;\n\t.reg .b32 x, y;\n\t.reg .b64 u, v;\n\t"                                             \
      "setp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 f, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"                                   \
      "mov.b64 u, {%2, %5};\n\tmov.b64 v, {%3, %5};\n\t"                                                             \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%1], u, v, %4, f;\n\t"                                         \
      "add.u32 x, %2, %7;\n\tadd.u32 y, %3, %8;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"                   \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%1], u, v, %4, t;\n\t"                                         \
      "add.u32 x, x, %7;\n\tadd.u32 y, y, %8;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"                     \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%1], u, v, %4, t;\n\t"                                         \
      "add.u32 x, x, %7;\n\tadd.u32 y, y, %8;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"                     \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::f16 [%1], u, v, %4, t;\n\t}" ::"r"(lead),                           \
      "r"(d), "r"(alo), "r"(blo), "r"(idesc), "r"(kHi), "r"(add ? 1u : 0u), "r"(sa), "r"(sb)                         \
      : "memory")
  if constexpr (CG == 1)
    MOE_DENSE_MMA("1");
  else
    MOE_DENSE_MMA("2");
#undef MOE_DENSE_MMA
  dense_commit<CG>(lead, empty);
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

// A's (B's) part of a stage.
template <class Op, int CG, bool IS_B>
__device__ __forceinline__ void dense_load(const typename Op::Params& p, const DenseTile& t, int kb, int b_off, uint8_t* to,
                                           uint64_t* bar, int rank) {
  int ak, am, bk, bn;
  Op::coords(p, t, kb, ak, am, bk, bn);
  const int k = IS_B ? bk : ak, x = IS_B ? bn + b_off : am;
  const bool to_even = CG == 2 && rank == 1;
  const int mat = Op::ONE ? 0 : t.mat;  // ONE: a single A and B, t.mat tells results apart
  const bool flip = (IS_B ? Op::FLIP_B : Op::FLIP_A) && dense_flip(p, kb, IS_B ? t.n0 : t.m0);
  const CUtensorMap* own = IS_B ? &p.tmB : &p.tmA;
  if ((IS_B ? Op::B_MN : Op::A_MN) || flip) {
    const CUtensorMap* map = flip ? &p.tmT : own;
    if (to_even)
      tma_load_4d_to_even(to, map, bar, 0, k, x / 64, mat);
    else
      tma_load_4d(to, map, bar, 0, k, x / 64, mat);
  } else {
    if (to_even)
      tma_load_3d_to_even(to, own, bar, k, x, mat);
    else
      tma_load_3d(to, own, bar, k, x, mat);
  }
}

// The tiles of a CTA one after the other.  Whether a tile has products at all is
// read from memory for some operations: a tile ahead, so that no role waits for it
// (a first tile without is computed all the same; the epilogue drops it).
template <class Op, int CG>
struct DenseWalk {
  int step, rank;
  float flag = 1.f;
  __device__ __forceinline__ DenseWalk(int step_, int rank_) : step(step_), rank(rank_) {}
  __device__ __forceinline__ DenseTile next(const typename Op::Params& p, int i) {
    DenseTile t = Op::template tile<CG>(p, i, rank);
    if (flag == 0.f) t.kb1 = t.kb0;
    if (i + step < p.total) flag = Op::flag(p, i + step);
    return t;
  }
};

template <class Op, int CG>
__global__ void __launch_bounds__(kDenseThreads, 1) dense_kernel(const __grid_constant__ typename Op::Params p) {
  const int NST = p.nst, SB = p.a_bytes + p.b_bytes;  // both multiples of 1024
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023) {  // as in grouped_gemm_kernel: reported, never computed on
    if (threadIdx.x == 0) record_error(p.err, MOE_ERR_CUDA, 0x5A11);
    return;
  }
  uint8_t* smem = smem_raw;
  DenseState& ss = *reinterpret_cast<DenseState*>(smem + kDenseRing);
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
  if (threadIdx.x == 32 * 2) {  // while the kernel before still runs
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB);
    if (Op::FLIP_A || Op::FLIP_B) tma_prefetch_desc(&p.tmT);
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
    // A's loads from one warp, B's from another: one thread took 365 to 590 cycles
    // from one K block's two loads to the next, a pair's MMAs take 512 (b A + c A A of
    // 66 x 1408 x 1408 1040 -> 845 us, dx and dW of 2000 tokens 158 -> 147 and 152 -> 137).
    auto load = [&](auto is_b) {
      constexpr bool IS_B = decltype(is_b)::value;
      int stage = 0;
      uint32_t phase = 0, filled = 0, fill_par = 0;
      bool ok = true;
      DenseWalk<Op, CG> walk(step, rank);
      for (int i = first; ok && i < p.total && !*abort; i += step) {
        const DenseTile t = walk.next(p, i);
        const int b_off = CG == 2 ? rank * dense_mma_n<CG, Op::B_MN || Op::FLIP_B>(p, t) / 2 : 0;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!mbar_wait(&ss.empty[stage], phase ^ 1, abort, p.err, where(IS_B, i))) {
            ok = false;
            break;
          }
          // a pair's loads are all counted on the even CTA's barrier (B's may be there
          // before the bytes are announced: the phase waits for the announcement)
          if (!IS_B && rank == 0) {
            mbar_arrive_expect_tx(&ss.full[stage], CG * SB);
            filled |= 1u << stage;
            fill_par = (fill_par & ~(1u << stage)) | phase << stage;
          }
          dense_load<Op, CG, IS_B>(p, t, kb, b_off, smem + stage * SB + (IS_B ? p.a_bytes : 0), &ss.full[stage], rank);
          if (++stage == NST) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort) {
        for (int s = 0; s < NST; ++s)
          if (filled & (1u << s)) mbar_wait_drain(&ss.full[s], (fill_par >> s) & 1);
        // copies whose bytes the other role no longer announced: long done by then
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kDrainNs;) __nanosleep(1000);
      }
    };
    if (lane == 0 && warp == 0) load(std::false_type{});
    if (lane == 0 && warp == 2) load(std::true_type{});
    __syncwarp();
    if (warp == 1 && rank == 0) {
      // The warp stays together: one lane issues by predicate, everything it needs
      // is the same in all lanes, and the next stage's barrier is asked while this
      // one's MMAs go out.
      constexpr uint32_t idesc0 = Op::F16 ? idesc_f16_f32(kBM * CG, 0, 0, 0) : idesc_bf16_f32(kBM * CG, 0, 0, 0);
      const uint32_t lead = elect_one();
      const uint32_t ring = smem_u32(smem) >> 4, sb16 = SB >> 4, a16 = p.a_bytes >> 4;
      const uint32_t full0 = smem_u32(&ss.full[0]), empty0 = smem_u32(&ss.empty[0]), tfull0 = smem_u32(&ss.tfull[0]);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      bool ready = false;  // the stage's data is known to be there
      DenseWalk<Op, CG> walk(step, rank);
      for (int i = first; ok && i < p.total && !*abort; i += step) {
        const DenseTile t = walk.next(p, i);
        const uint32_t idesc = idesc0 | static_cast<uint32_t>(dense_mma_n<CG, Op::B_MN || Op::FLIP_B>(p, t) >> 3) << 17;
        int left = 0;  // K blocks left of the run
        uint32_t dtm = 0;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          const bool fresh = left == 0;
          if (fresh) {
            ok = mbar_wait<CG == 2>(&ss.tempty[it & 1], ((it >> 1) & 1) ^ 1, abort, p.err, where(2, i));
            if (!ok) break;
            dtm = tmem + (it & 1) * kBN;
            left = min(p.run_kb, t.kb1 - kb);
          }
          if (!ready) {
            ok = mbar_wait(&ss.full[stage], phase, abort, p.err, where(3, i));
            if (!ok) break;
          }
          tc_fence_after();
          --left;
          const uint32_t a = ring + stage * sb16, empty = empty0 + 8 * stage;
          if (++stage == NST) {
            stage = 0;
            phase ^= 1;
          }
          ready = __all_sync(0xffffffffu, mbar_test_wait(full0 + 8 * stage, phase));
          const bool a_mn = Op::A_MN || (Op::FLIP_A && dense_flip(p, kb, t.m0));
          const bool b_mn = Op::B_MN || (Op::FLIP_B && dense_flip(p, kb, t.n0));
          dense_mma<CG>(lead, dtm, a, a + a16, a_mn, b_mn, idesc, !fresh, empty);
          issued = true;
          if (left == 0) {
            dense_commit<CG>(lead, tfull0 + 8 * (it & 1));
            ++it;
          }
        }
      }
      if (*abort && issued) {
        if (lead) {
          umma_commit<CG>(&ss.drain);
          mbar_wait_drain(&ss.drain, 0);
        }
        __syncwarp();
      }
    }
  } else {
    regs_take<kEpiRegs>();
    DenseEpi e;
    e.lane = lane;
    e.q = warp & 3;  // TMEM lanes [32q, 32q + 32) are reachable from this warp
    e.part = (warp - 4) >> 2;
    int it = 0;
    bool ok = true;
    DenseWalk<Op, CG> walk(step, rank);
    for (int i = first; ok && i < p.total && !*abort; i += step) {
      const DenseTile t = walk.next(p, i);
      const bool active = t.m0 + 32 * e.q < p.M;
      auto release = [&](int buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && rank == 1)
            mbar_arrive_rank(&ss.tempty[buf], 0);
          else
            mbar_arrive(&ss.tempty[buf]);
        }
      };
      if constexpr (Op::CHUNKS) {
        // one run: 32 columns at a time, the next ones on their way meanwhile
        if (t.kb1 == t.kb0) continue;
        const auto pre = Op::pre(p, t, e);
        const int buf = it & 1;
        if (!mbar_wait_inline(&ss.tfull[buf], (it >> 1) & 1, abort, p.err, where(4, i))) break;
        ++it;
        tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(e.q * 32) << 16) + buf * kBN + e.part * p.half;
        const int chunks = active ? (dense_width(p, t, e) + 31) / 32 : 0;
        uint32_t v[2][32];
        if (chunks > 0) {
          tmem_ld_32x32(ta, v[0]);
          tmem_ld_wait();
        } else {
          release(buf);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= chunks) break;
          if (c + 1 < chunks)
            tmem_ld_32x32(ta + 32 * (c + 1), v[(c + 1) & 1]);
          else
            release(buf);
          Op::chunk(p, t, e, pre, c, v[c & 1]);
          if (c + 1 < chunks) tmem_ld_wait();
        }
        continue;
      }
      decltype(Op::pre(p, t, e)) pre{};
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
        // in the first pause: the products of the run after next wait for the first run's buffer
        if (r == min(1, runs - 1)) pre = Op::pre(p, t, e);
        if (!mbar_wait_inline(&ss.tfull[buf], (it >> 1) & 1, abort, p.err, where(4, i))) {
          ok = false;
          break;
        }
        ++it;
        tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(e.q * 32) << 16) + buf * kBN + e.part * p.half;
        if (!active) {
          // rows that are not there
        } else if (r == 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32(ta + 32 * c, acc[c]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            if (32 * c >= p.half) break;
            uint32_t v[2][32];
            tmem_ld_32x32(ta + 32 * c, v[0]);
            tmem_ld_32x32(ta + 32 * c + 32, v[1]);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                acc[c + h][j] = __float_as_uint(__uint_as_float(acc[c + h][j]) + __uint_as_float(v[h][j]));
          }
        }
        release(buf);
      }
      if constexpr (!Op::CHUNKS)
        if (ok && active) Op::epilogue(p, t, e, pre, acc);
    }
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

// Tile shape and splits of K of a product of an M x N C.
struct DenseShape {
  int cg, tn, splits;
};

// The shape with the shortest estimated time: rounds of tiles over the SMs, each
// its K blocks (us each: a CTA takes in about 100 GB/s, a pair's MMAs 0.3) and an
// epilogue; splits of K (a matrix of fp32 sums each, added up by another launch)
// cost their bytes twice at 5 TB/s.  sym: C is symmetric, its tiles square and only
// those from the diagonal on computed.  152: the SMs of the GB300; fixed, so that
// results and workspaces do not depend on the device asked.
DenseShape dense_pick(long long M, long long N, int mats, int nkb, bool sym, int max_splits) {
  struct Option {
    int cg, tn;
    double kb, epi;
  };
  constexpr Option kOptions[] = {{2, 256, 0.30, 3.0}, {1, 256, 0.40, 3.0}, {1, 128, 0.28, 2.0}, {1, 64, 0.22, 1.5}};
  DenseShape best{2, 256, 1};
  double least = 1e30;
  for (const Option& o : kOptions) {
    const int tm = kBM * o.cg;
    if (sym && o.tn != tm) continue;
    const long long nt = (N + o.tn - 1) / o.tn, mt = (M + tm - 1) / tm;
    const long long tiles = mats * (sym ? nt * (nt + 1) / 2 : nt * mt);
    for (int sp = 1; sp <= max_splits && sp <= nkb; sp += (sp + 3) / 4) {  // 1 to 5, 7, 9, 12, 15, 19, ...
      const long long units = 152 / o.cg, rounds = (tiles * sp + units - 1) / units;
      const double us = rounds * (o.kb * ((nkb + sp - 1) / sp) + o.epi) + (sp > 1 ? 3.0 + (sp - 1) * 8.0 * M * N / 5e6 : 0.0);
      if (us < 0.97 * least) {
        least = us;
        best = {o.cg, o.tn, sp};
      }
    }
  }
  return best;
}

// Rows and columns of tiles, what a K block brings, and the tiles of `mats`
// matrices (or splits).
void dense_shape(DenseParams& p, int cg, int tn, int mats, bool sym) {
  p.tn = tn;
  p.half = ceil_div(tn, 64) * 32;
  p.a_bytes = kABytes;
  p.b_bytes = tn * 128 / cg;
  p.mt = ceil_div(p.M, kBM * cg);
  p.nt = ceil_div(p.N, tn);
  p.total = mats * (sym ? p.nt * (p.nt + 1) / 2 : p.mt * p.nt);
}

template <class Op, int CG>
int dense_launch(typename Op::Params& p, int grid_limit, int trace, cudaStream_t s) {
  // The MMAs read 128 rows of A, also where fewer are loaded: what lies behind
  // them (B, the next stage) then gives rows of C that are not there.
  p.nst = std::min(kDenseMaxStages, (kDenseRing - (kABytes - p.a_bytes)) / (p.a_bytes + p.b_bytes));
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
template <class Op>
int dense_launch(int cg, typename Op::Params& p, int grid_limit, int trace, cudaStream_t s) {
  return cg == 1 ? dense_launch<Op, 1>(p, grid_limit, trace, s) : dense_launch<Op, 2>(p, grid_limit, trace, s);
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
}  // namespace
}  // namespace moe
