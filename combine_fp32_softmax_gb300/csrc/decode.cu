// The layer for a few tokens (T <= 64) and its linear form, y = x W^T, with
// bf16 or 4-bit weights, as one persistent launch that streams the weights.
//
//   hidden  h[r, i] = w_r * silu(x_t . W1_e[i]) * (x_t . W3_e[i])
//   out     y[t, c] = sum over the token's rows r, slots first, of h[r] . W2_e[c]
//
// What bounds it: at 64 tokens the products need 8 flops per weight byte,
// the tensor cores balance at 280, so the weights' bytes are the work.  The
// kernel is built around keeping them coming:
//   - A producer warp keeps a ring of shared-memory stages full of weight
//     tiles (128 rows x 128 bytes, two TMA boxes of 64 rows), up to 200 KB in
//     flight per SM.  It needs nothing but the routing, so it runs ahead into
//     W2 while the hidden values of this and other CTAs are still being made:
//     the grid-wide dependency between the two products costs no bandwidth.
//   - A second producer warp brings the activation columns of the same tiles
//     (16-byte asynchronous copies, rows gathered by token) and is the one
//     that waits for the hidden values of all CTAs before the second product.
//     One bulk copy per row instead took 1300 clocks a stage at 32 rows, twice
//     what the weights of the stage need.
//   - The tiles of all picked experts form one sequence of K blocks, cut into
//     equal contiguous ranges, one per SM, so no SM idles whatever the number
//     of experts, rows and tokens.  A tile cut by a range border belongs to
//     the range it begins in.  The ranges it goes on in work on it first and
//     leave their sums in the workspace; its owner comes to it last, long
//     after, and adds them in range order: no floating-point atomics, and
//     nobody waits in the middle of a range.
//   - Sixteen consumer warps multiply: weights are the 16-row operand of
//     mma.sync.m16n8k16, activations its 8 columns, so one token wastes
//     tensor throughput that nothing else needs, and no shared-memory copy of
//     converted 4-bit weights is made: codes become bf16 pairs in the
//     registers that feed the instruction.  The warp-level instruction has
//     the rate for it: a weight fragment arrives every 21 clocks per SM
//     (bf16).  Each warp takes 8 rows of either box (W1 and W3 rows of the
//     same hidden columns, so silu(a) * b stays in a thread) and one half of
//     the stage's columns.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "decode.h"
#include "kernels.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "route.cuh"
#include "tensor_map.h"
#include "trace.h"

namespace moe {

namespace {

constexpr int kRowGroups = 8;            // 8 rows of either box each
constexpr int kMmaWarps = 2 * kRowGroups;   // row groups x halves of a stage's columns
constexpr int kWeightWarp = kMmaWarps;      // producer of weight tiles
constexpr int kColumnWarp = kMmaWarps + 1;  // producer of activation columns
constexpr int kWarps = kMmaWarps + 2;
constexpr int kThreads = kWarps * 32;
constexpr int kBoxRows = 64;             // rows of one weight box
constexpr int kBoxBytes = kBoxRows * 128;
constexpr int kMaxStages = 12;
constexpr int kMaxTokens = MOE_DECODE_MAX_T;
constexpr int kMaxPicks = kMaxTokens * 8;
constexpr int kMaxRows = kMaxTokens * 12;   // k <= 8 slots and 4 shared experts
// Experts in the work list: all routed ones and the shared ones.
constexpr int kMaxActive = 256 + 4;
// Most ranges (SMs) that a workspace has room for.
constexpr int kMaxWorkers = 256;

// Counters in the error region (ints), all 0 between launches.
constexpr int kCtrHidden = 8;   // finishing warps (one per row group) done with the first product
constexpr int kCtrOut = 9;      // ... with the second
constexpr int kCtrExit = 10;    // CTAs done

// Columns of a stage and bytes between activation rows in it.  The padding
// puts the 8 rows an instruction reads into different banks: ldmatrix reads
// 16 bytes of each (bf16), 16-byte loads 64 bytes of two at a time (4 bits).
template <int G>
struct Geo {
  static constexpr bool Q4 = G != 0;
  static constexpr int KB = Q4 ? 256 : 64;
  static constexpr int PITCH = Q4 ? 512 + 64 : 128 + 16;
  // Activation rows (MMA columns) of a tile.  An expert with more has its
  // weight tiles visited again, from L2.  32 rows of 512 bytes in several
  // parts would leave no room for a ring.
  static constexpr int COLS = Q4 ? 16 : 32;
  static constexpr int GROUPS = Q4 ? KB / (Q4 ? G : 1) : 0;   // scale rows of a stage
  static constexpr int SCALE_BYTES = GROUPS * kBoxRows * 2;   // of one box
};

// One product of the launch: weight tiles of `row_step` output rows.
struct Product {
  CUtensorMap w0, w1;   // weight boxes: W1 and W3, or the two halves of a W2 tile
  CUtensorMap s0, s1;   // their scales (4 bits)
  int K, kblocks, rows, row_step, row_tiles;
};

struct StreamParams {
  Product p[2];         // layer: hidden, out; linear form: the second only
  int T, d, f, E, k, S, renorm, n;
  const float* logits;
  const uint16_t* x;
  int32_t* topk_idx;
  float* topk_w;
  uint16_t* h;          // [parts][Rs][f]
  float* o;             // [Rs][d]
  float* part;          // sums of the tile that a range begins in: [workers][row groups][16][32]
  int* arrive;          // parts there, by the owning range: [2][workers][row groups]
  void* y;
  int* err;             // error word and counters
  int y_type, workers, stages, stage_bytes, xbuf_bytes;
  int cols8, parts;     // activation rows of a stage; bf16 parts of a hidden value
};

struct alignas(16) Shared {
  uint64_t full_w[kMaxStages], full_x[kMaxStages], empty[kMaxStages];
  uint64_t xfull[kRowGroups], xfree[kRowGroups];  // exchange of the column halves
  int abort;
  int nact, nblk;                  // work list entries, column blocks of 32 rows in all
  int e[kMaxActive];               // expert
  int m[kMaxActive];               // its rows
  int row0[kMaxActive];            // its first row in h and o
  int blk0[kMaxActive + 1];        // column blocks before it
  unsigned mask[256][2];           // tokens that picked expert e
  float row_w[kMaxRows];
  float pick_w[kMaxPicks];
  short pick_e[kMaxPicks];
  short pick_row[kMaxPicks];
  unsigned char row_token[kMaxRows];
};

constexpr int kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

// ---------------------------------------------------------------- work list
// Routes every token and lists the experts that have rows, each CTA for
// itself (64 tokens x 64 experts are 16 KB of logits from L2).  A token picks
// an expert at most once, so an expert's tokens are a 64-bit mask and a row's
// place in its expert's list is a population count: ascending tokens,
// whatever the order of the atomics that set the bits.
template <int EPL>
__device__ __forceinline__ void route_tokens(const StreamParams& p, Shared& ss) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float ahead[EPL];  // the next token's logits
  if (warp < p.T) row_load<EPL>(p.logits + static_cast<size_t>(warp) * p.E, p.E, lane, ahead);
  for (int t = warp; t < p.T; t += kWarps) {
    RowSoftmax<EPL> r;
#pragma unroll
    for (int i = 0; i < EPL; ++i) r.v[i] = ahead[i];
    if (t + kWarps < p.T) row_load<EPL>(p.logits + static_cast<size_t>(t + kWarps) * p.E, p.E, lane, ahead);
    int idx;
    float w;
    route_token<EPL>(r, t, p.E, p.k, p.renorm, lane, p.err, idx, w);
    if (lane < p.k) {
      ss.pick_e[t * p.k + lane] = static_cast<short>(idx);
      ss.pick_w[t * p.k + lane] = w;
      atomicOr(&ss.mask[idx][t >> 5], 1u << (t & 31));
      if (blockIdx.x == 0) {
        p.topk_idx[t * p.k + lane] = idx;
        p.topk_w[t * p.k + lane] = w;
      }
    }
  }
}

template <int COLS>
__device__ void build_work_list(const StreamParams& p, Shared& ss) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < 512; i += kThreads) (&ss.mask[0][0])[i] = 0;
  __syncthreads();
  if (p.E <= 32)
    route_tokens<1>(p, ss);
  else if (p.E <= 64)
    route_tokens<2>(p, ss);
  else if (p.E <= 128)
    route_tokens<4>(p, ss);
  else
    route_tokens<8>(p, ss);
  __syncthreads();
  const int R = p.T * p.k;
  if (tid < 32) {  // experts 8 lane .. 8 lane + 7: exclusive sums of entries, rows and column blocks
    int n[8], na = 0, nr = 0, nb = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane * 8 + j;
      n[j] = e < p.E ? __popc(ss.mask[e][0]) + __popc(ss.mask[e][1]) : 0;
      na += n[j] > 0;
      nr += n[j];
      nb += (n[j] + COLS - 1) / COLS;
    }
    int ia = na, ir = nr, ib = nb;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int xa = __shfl_up_sync(kFull, ia, off), xr = __shfl_up_sync(kFull, ir, off),
                xb = __shfl_up_sync(kFull, ib, off);
      if (lane >= off) ia += xa, ir += xr, ib += xb;
    }
    const int all_a = __shfl_sync(kFull, ia, 31), all_b = __shfl_sync(kFull, ib, 31);
    ia -= na, ir -= nr, ib -= nb;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n[j] == 0) continue;
      ss.e[ia] = lane * 8 + j;
      ss.m[ia] = n[j];
      ss.row0[ia] = ir;
      ss.blk0[ia] = ib;
      ++ia;
      ir += n[j];
      ib += (n[j] + COLS - 1) / COLS;
    }
    const int per = (p.T + COLS - 1) / COLS;
    if (lane < p.S) {
      ss.e[all_a + lane] = p.E + lane;
      ss.m[all_a + lane] = p.T;
      ss.row0[all_a + lane] = R + lane * p.T;
      ss.blk0[all_a + lane] = all_b + lane * per;
    }
    if (lane == 0) {
      ss.nact = all_a + p.S;
      ss.nblk = all_b + p.S * per;
      ss.blk0[all_a + p.S] = all_b + p.S * per;
    }
  }
  __syncthreads();
  // rows: first row of the expert (entry by binary search) + earlier tokens of its mask
  for (int i = tid; i < R; i += kThreads) {
    const int e = ss.pick_e[i], t = i / p.k;
    int lo = 0, hi = ss.nact - p.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (ss.e[mid] < e)
        lo = mid + 1;
      else
        hi = mid;
    }
    const unsigned m0 = ss.mask[e][0], m1 = ss.mask[e][1], below = (1u << (t & 31)) - 1u;
    const int row = ss.row0[lo] + (t < 32 ? __popc(m0 & below) : __popc(m0) + __popc(m1 & below));
    ss.pick_row[i] = static_cast<short>(row);
    ss.row_token[row] = static_cast<unsigned char>(t);
    ss.row_w[row] = ss.pick_w[i];
  }
  for (int i = tid; i < p.S * p.T; i += kThreads) {
    ss.row_token[R + i] = static_cast<unsigned char>(i % p.T);
    ss.row_w[R + i] = 1.f;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ ranges
// The K blocks of a product, tile after tile (expert, row tile, column
// block), cut into `workers` contiguous ranges.  Every role of a CTA walks
// the same segments: the K blocks [kb0, kb1) of one tile.
struct Segment {
  int worker, item, kb0, kb1;
  int a, rt, nb;   // work list entry, row tile, column block
};

struct Walk {
  const Product& pr;
  const Shared& ss;
  int workers, v;
  int units, u, u1;
  int item, kb, a;

  // A CTA takes the ranges blockIdx.x + i * gridDim.x in descending order:
  // the owner of a cut tile waits for ranges after its own, so on a capped
  // grid those come first.
  __device__ Walk(const Product& product, const Shared& shared, int most) : pr(product), ss(shared) {
    units = ss.nblk * pr.row_tiles * pr.kblocks;
    workers = min(most, units);  // no range is empty
    const int b = static_cast<int>(blockIdx.x), n = static_cast<int>(gridDim.x);
    v = b < workers ? b + ((workers - 1 - b) / n + 1) * n : 0;
    u = u1 = 0;
    item = kb = a = 0;
  }
  __device__ int begin_of(int worker) const {
    return static_cast<int>(static_cast<long long>(units) * worker / workers);
  }
  // The range that holds K block `unit`.
  __device__ int worker_of(int unit) const {
    return static_cast<int>((static_cast<long long>(unit + 1) * workers - 1) / units);
  }
  __device__ bool next(Segment& s) {
    if (u >= u1) {
      v -= static_cast<int>(gridDim.x);
      if (v < 0) return false;
      u = begin_of(v);
      u1 = begin_of(v + 1);
      item = u / pr.kblocks;
      kb = u - item * pr.kblocks;
      int lo = 0, hi = ss.nact - 1;   // last entry with blk0 * row_tiles <= item
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (ss.blk0[mid] * pr.row_tiles <= item)
          lo = mid;
        else
          hi = mid - 1;
      }
      a = lo;
    }
    while (item >= ss.blk0[a + 1] * pr.row_tiles) ++a;
    const int nblk = ss.blk0[a + 1] - ss.blk0[a], r = item - ss.blk0[a] * pr.row_tiles;
    s.worker = v;
    s.item = item;
    s.kb0 = kb;
    s.kb1 = min(pr.kblocks, kb + (u1 - u));
    s.a = a;
    s.rt = r / nblk;
    s.nb = r - s.rt * nblk;
    u += s.kb1 - s.kb0;
    kb = 0;
    ++item;
    return true;
  }
};

struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

__device__ bool drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(a, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}
// Lets the copies that this producer issued land before the CTA may leave
// its shared memory (after an abort nobody else waits for them).
struct Drain {
  uint32_t filled = 0, parity = 0;
  __device__ __forceinline__ void note(int stage, uint32_t phase) {
    filled |= 1u << stage;
    parity = (parity & ~(1u << stage)) | (phase << stage);
  }
  __device__ void wait(uint64_t* bars) const {
    for (int s = 0; s < kMaxStages; ++s)
      if (filled >> s & 1) drain_wait(&bars[s], parity >> s & 1);
  }
};

// Waits until `target` arrivals are counted (bounded).
__device__ bool wait_count(const int* c, int target, volatile int* abort, int* err, int where) {
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire_gpu(c) < target) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, MOE_ERR_TIMEOUT_CODE, where);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// --------------------------------------------------------------- producers
template <int G>
__device__ bool produce_weights(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg, Drain& dr,
                                volatile int* abort) {
  using Ge = Geo<G>;
  const Product& pr = p.p[which];
  Walk walk(pr, ss, p.workers);
  Segment s;
  while (walk.next(s)) {
    const int row = ss.e[s.a] * pr.rows + s.rt * pr.row_step;
    const int second = which == 0 ? row : row + kBoxRows;  // W3 beside W1, or the tile's other rows
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
      if (!mbar_wait(&ss.empty[rg.stage], rg.phase ^ 1, abort, p.err, (0x21 << 24) | which)) return false;
      uint8_t* st = ring + static_cast<size_t>(rg.stage) * p.stage_bytes;
      uint64_t* bar = &ss.full_w[rg.stage];
      mbar_arrive_expect_tx(bar, 2 * (kBoxBytes + Ge::SCALE_BYTES));
      dr.note(rg.stage, rg.phase);
      const int col = kb * (Ge::Q4 ? 128 : 64);  // bytes or bf16
      tma_load_2d(st, &pr.w0, bar, col, row);
      tma_load_2d(st + kBoxBytes, &pr.w1, bar, col, second);
      if constexpr (Ge::Q4) {
        uint8_t* sc = st + 2 * kBoxBytes;
        const int at = ss.e[s.a] * (pr.K / G) + kb * Ge::GROUPS, r0 = s.rt * pr.row_step;
        tma_load_2d(sc, &pr.s0, bar, r0, at);
        tma_load_2d(sc + Ge::SCALE_BYTES, &pr.s1, bar, which == 0 ? r0 : r0 + kBoxRows, at);
      }
      rg.step(p.stages);
    }
  }
  return true;
}

// Columns: the rows of x by token (hidden, linear) or the parts of h.  16
// bytes a lane; a lane's arrival on the stage's barrier follows its copies.
template <int G, bool LAYER>
__device__ bool produce_columns(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg,
                                volatile int* abort) {
  using Ge = Geo<G>;
  constexpr int LANES = Ge::KB / 8;         // lanes of a row
  constexpr int ROWS = 32 / LANES;          // rows of an instruction
  const Product& pr = p.p[which];
  const int lane = threadIdx.x & 31;
  const bool hidden_in = LAYER && which == 1;
  const uint16_t* base = hidden_in ? p.h : p.x;
  const int parts = hidden_in ? p.parts : 1;
  const size_t part_step = static_cast<size_t>(p.T) * (p.k + p.S) * p.f;
  const int col = (lane % LANES) * 8;
  Walk walk(pr, ss, p.workers);
  Segment s;
  while (walk.next(s)) {
    const int m = min(Ge::COLS, ss.m[s.a] - s.nb * Ge::COLS);
    const int r = ss.row0[s.a] + s.nb * Ge::COLS;
    int mine = 0;  // row of `base` that this lane keeps for the warp
    if (lane < m) mine = hidden_in ? r + lane : ss.row_token[r + lane];
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
      const bool ok = mbar_wait(&ss.empty[rg.stage], rg.phase ^ 1, abort, p.err, (0x22 << 24) | which);
      if (!__all_sync(kFull, ok)) return false;
      uint64_t* bar = &ss.full_x[rg.stage];
      const uint32_t dst = smem_u32(ring) + static_cast<uint32_t>(rg.stage) * p.stage_bytes +
                           2 * (kBoxBytes + Ge::SCALE_BYTES) + (lane / LANES) * Ge::PITCH + col * 2;
      const bool in = kb * Ge::KB + col < pr.K;
      for (int i = 0; i < m; i += ROWS) {
        const int at = i + lane / LANES;
        const int row = __shfl_sync(kFull, mine, at & 31);
        const uint16_t* src = base + static_cast<size_t>(row) * pr.K + kb * Ge::KB + col;
        if (in && at < m)
          for (int q = 0; q < parts; ++q)
            cp_async16(dst + (q * p.cols8 + i) * Ge::PITCH, src + q * part_step);
      }
      cp_async_arrive(bar);
      rg.step(p.stages);
    }
  }
  return true;
}

// --------------------------------------------------------------- consumers
// The hidden values enter the second product in bf16 parts that add up to
// them: two (16 significant bits) for a bf16 y, three (24) for an fp32 y.
// One part alone would cost 2^-9 of each value, as much as the rounding of a
// bf16 y, and the tensor instructions of more parts are free beside the
// weights' bytes.  The lower parts are held times 2^8, so that they leave
// bf16's range no sooner than the upper one does.
constexpr float kLowScale = 256.f;

// Sums of the upper part, and of the lower ones together.
template <int PARTS>
constexpr int kSums = PARTS > 1 ? 2 : 1;

template <int SUMS, int NT>
__device__ __forceinline__ float join_parts(const float (&s)[SUMS][NT][4], int n, int i) {
  if constexpr (SUMS == 2)
    return fmaf(s[1][n][i], 1.f / kLowScale, s[0][n][i]);
  else
    return s[0][n][i];
}

// One stage, this warp's 8 rows of either box and half of the columns:
// acc[n][..] += weights . columns.  The 16-row operand holds the first box's
// rows on top and the second box's below.  Sums of a stage (bf16) or of a
// group (4 bits) start from zero in the tensor core and are added to acc in
// fp32, so the chain of additions inside the tensor core, which truncates, is
// short.
template <int G, int NT, int PARTS>
__device__ __forceinline__ void multiply_stage(uint32_t st, int part_bytes, int kleft, int m, float (&acc)[NT][4]) {
  using Ge = Geo<G>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rgrp = warp % kRowGroups, half = warp / kRowGroups;
  const uint32_t cols = st + 2 * (kBoxBytes + Ge::SCALE_BYTES);
  // matrices (box 0, 16 bytes c), (box 1, c), (box 0, c + 1), (box 1, c + 1)
  const uint32_t arow = st + ((lane >> 3) & 1) * kBoxBytes + (rgrp * 8 + (lane & 7)) * 128;
  auto frag = [&](int c, uint32_t (&a)[4]) {
    ldmatrix_x4(arow + ((static_cast<uint32_t>(c + (lane >> 4)) ^ (lane & 7)) << 4), a);
  };
  if constexpr (!Ge::Q4) {
    float s[kSums<PARTS>][NT][4] = {};
    uint32_t a[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) frag(half * 4 + 2 * i, a[i]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        uint32_t b[4];  // four matrices: 16 bytes c .. c + 3 of the 8 activation rows
        ldmatrix_x4(cols + q * part_bytes + (n * 8 + (lane & 7)) * Ge::PITCH + (half * 4 + (lane >> 3)) * 16, b);
        mma_bf16(s[q > 0][n], a[0][0], a[0][1], a[0][2], a[0][3], b[0], b[1]);
        mma_bf16(s[q > 0][n], a[1][0], a[1][1], a[1][2], a[1][3], b[2], b[3]);
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] += join_parts(s, n, i);
  } else {
    const int g = lane >> 2, t = lane & 3;
    const uint32_t scales = st + 2 * kBoxBytes + (rgrp * 8 + g) * 2;
    constexpr int CHUNKS = 4;                        // 32-column chunks of this warp's half
    float s[kSums<PARTS>][NT][4];
#pragma unroll
    for (int c2 = 0; c2 < CHUNKS; c2 += 2) {
      if (half * 128 + c2 * 32 >= kleft) break;      // columns past K (a multiple of 64)
      uint32_t w[4];
      frag(half * 4 + c2, w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {                  // chunk c2 + i
        const int c = half * 4 + c2 + i;
        const bool group_begins = G == 32 || (i == 0 && (G == 64 || c2 == 0));
        const bool group_ends = G == 32 || (i == 1 && (G == 64 || c2 == 2));
        if (group_begins)
#pragma unroll
          for (int j = 0; j < kSums<PARTS> * NT * 4; ++j) (&s[0][0][0])[j] = 0.f;
        uint32_t a[8];                               // pairs 0..3 of either box's row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[2 * j] = q4_pair(w[2 * i], j);
          a[2 * j + 1] = q4_pair(w[2 * i + 1], j);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            uint32_t b[4] = {0, 0, 0, 0};
            if (n * 8 + g < m) lds128(cols + q * part_bytes + (n * 8 + g) * Ge::PITCH + c * 64 + t * 16, b);
            mma_bf16(s[q > 0][n], a[0], a[1], a[2], a[3], b[0], b[1]);
            mma_bf16(s[q > 0][n], a[4], a[5], a[6], a[7], b[2], b[3]);
          }
        if (group_ends) {
          const uint32_t sc = scales + (c * 32 / G) * (kBoxRows * 2);
          const float f0 = lds_bf16(sc), f1 = lds_bf16(sc + Ge::SCALE_BYTES);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(f0, join_parts(s, n, 0), acc[n][0]);
            acc[n][1] = fmaf(f0, join_parts(s, n, 1), acc[n][1]);
            acc[n][2] = fmaf(f1, join_parts(s, n, 2), acc[n][2]);
            acc[n][3] = fmaf(f1, join_parts(s, n, 3), acc[n][3]);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void store_y(void* y, int y_type, size_t at, float v) {
  if (y_type == MOE_Y_BF16)
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(y)[at] = v;
}

// A finished tile's values, one thread's share: row g of either box, columns
// 2t and 2t + 1 of every 8.
template <int G, bool LAYER, int NT>
__device__ __forceinline__ void finish_tile(const StreamParams& p, int which, const Shared& ss, const Segment& s,
                                            const float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, rgrp = (threadIdx.x >> 5) % kRowGroups;
  const int row = rgrp * 8 + (lane >> 2), t2 = (lane & 3) * 2;
  const int m = min(Geo<G>::COLS, ss.m[s.a] - s.nb * Geo<G>::COLS), r0 = ss.row0[s.a] + s.nb * Geo<G>::COLS;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = n * 8 + t2 + i;
      if (col >= m) continue;
      const int r = r0 + col;
      if (LAYER && which == 0) {
        const float a = acc[n][i], b = acc[n][2 + i];
        const float h = ss.row_w[r] * (a / (1.f + expf(-a)) * b);
        const size_t part_step = static_cast<size_t>(p.T) * (p.k + p.S) * p.f;
        uint16_t* to = p.h + static_cast<size_t>(r) * p.f + s.rt * kBoxRows + row;
        float rest = h;
        for (int q = 0; q < p.parts; ++q) {
          const __nv_bfloat16 v = __float2bfloat16_rn(rest);
          to[q * part_step] = __bfloat16_as_ushort(v);
          rest = (rest - __bfloat162float(v)) * (q == 0 ? kLowScale : 1.f);
          if (!isfinite(rest)) rest = 0.f;  // a value that rounds to infinity keeps that alone
        }
      } else {
#pragma unroll
        for (int box = 0; box < 2; ++box) {
          const int c = s.rt * 2 * kBoxRows + box * kBoxRows + row;
          if (LAYER) {
            if (c < p.d) p.o[static_cast<size_t>(r) * p.d + c] = acc[n][2 * box + i];
          } else {
            if (c < p.n) store_y(p.y, p.y_type, static_cast<size_t>(r) * p.n + c, acc[n][2 * box + i]);
          }
        }
      }
    }
}

struct Consumer {
  Ring rg;
  uint32_t xphase = 0;  // exchange of the column halves
};

// Sums this warp's share of a segment and, on the lower column half's warp,
// finishes the tile or leaves its part for the range that does.  False after
// a wait that gave up.
template <int G, bool LAYER, int NT, int PARTS>
__device__ bool consume_segment(const StreamParams& p, int which, Shared& ss, uint8_t* ring, float* xbuf, const Walk& walk,
                                const Segment& s, Consumer& cs, volatile int* abort) {
  using Ge = Geo<G>;
  const Product& pr = p.p[which];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rgrp = warp % kRowGroups, half = warp / kRowGroups;
  const int m = min(Ge::COLS, ss.m[s.a] - s.nb * Ge::COLS);
  constexpr int N = NT * 4;
  float acc[NT][4] = {};
  bool ok = true;
  for (int kb = s.kb0; kb < s.kb1; ++kb) {
    ok = mbar_wait(&ss.full_w[cs.rg.stage], cs.rg.phase, abort, p.err, (0x23 << 24) | which) &&
         mbar_wait(&ss.full_x[cs.rg.stage], cs.rg.phase, abort, p.err, (0x24 << 24) | which);
    if (!__all_sync(kFull, ok)) return false;
    const uint32_t st = smem_u32(ring) + static_cast<uint32_t>(cs.rg.stage) * p.stage_bytes;
    multiply_stage<G, NT, PARTS>(st, p.cols8 * Ge::PITCH, pr.K - kb * Ge::KB, m, acc);
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.empty[cs.rg.stage]);
    cs.rg.step(p.stages);
  }
  // the two column halves
  float* xb = xbuf + rgrp * (p.xbuf_bytes / (kRowGroups * static_cast<int>(sizeof(float)))) + lane;
  if (half == 1) {
    ok = mbar_wait(&ss.xfree[rgrp], cs.xphase ^ 1, abort, p.err, (0x27 << 24) | which);
    cs.xphase ^= 1;
    if (!__all_sync(kFull, ok)) return false;
#pragma unroll
    for (int i = 0; i < N; ++i) xb[i * 32] = (&acc[0][0])[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.xfull[rgrp]);
    return true;
  }
  ok = mbar_wait(&ss.xfull[rgrp], cs.xphase, abort, p.err, (0x28 << 24) | which);
  cs.xphase ^= 1;
  if (!__all_sync(kFull, ok)) return false;
#pragma unroll
  for (int i = 0; i < N; ++i) (&acc[0][0])[i] += xb[i * 32];
  __syncwarp();
  if (lane == 0) mbar_arrive(&ss.xfree[rgrp]);

  const int first = s.item * pr.kblocks;
  auto part = [&](int v) { return p.part + (static_cast<size_t>(v) * kRowGroups + rgrp) * (16 * 32) + lane; };
  auto arrived = [&](int v) { return p.arrive + (static_cast<size_t>(which) * p.workers + v) * kRowGroups + rgrp; };
  if (s.kb0 != 0) {  // the tile began in an earlier range
    float* mine = part(s.worker);
#pragma unroll
    for (int i = 0; i < N; ++i) __stcg(mine + i * 32, (&acc[0][0])[i]);
    __syncwarp();
    if (lane == 0) red_release_gpu_add(arrived(walk.worker_of(first)), 1);
    return true;
  }
  if (s.kb1 != pr.kblocks) {  // it goes on in later ranges, which began with it
    const int v1 = walk.worker_of(first + pr.kblocks - 1);
    int* cnt = arrived(s.worker);
    if (lane == 0) {
      ok = wait_count(cnt, v1 - s.worker, abort, p.err, (0x29 << 24) | which);
      *cnt = 0;
    }
    if (!__shfl_sync(kFull, ok, 0)) return false;
    for (int v = s.worker + 1; v <= v1; ++v) {
      const float* from = part(v);
#pragma unroll
      for (int i = 0; i < N; ++i) (&acc[0][0])[i] += __ldcg(from + i * 32);
    }
  }
  finish_tile<G, LAYER, NT>(p, which, ss, s, acc);
  return true;
}

template <int G, bool LAYER, int PARTS>
__device__ bool consume(const StreamParams& p, int which, Shared& ss, uint8_t* ring, float* xbuf, Consumer& cs,
                        volatile int* abort) {
  Walk walk(p.p[which], ss, p.workers);
  Segment s;
  bool ok = true;
  while (ok && walk.next(s)) {
    const int m = min(Geo<G>::COLS, ss.m[s.a] - s.nb * Geo<G>::COLS);
    if (m <= 8)
      ok = consume_segment<G, LAYER, 1, PARTS>(p, which, ss, ring, xbuf, walk, s, cs, abort);
    else if (m <= 16)
      ok = consume_segment<G, LAYER, 2, PARTS>(p, which, ss, ring, xbuf, walk, s, cs, abort);
    else if constexpr (Geo<G>::COLS > 16)
      ok = consume_segment<G, LAYER, 4, PARTS>(p, which, ss, ring, xbuf, walk, s, cs, abort);
  }
  return ok;
}

// y[t] = its slots' rows in slot order, then the shared experts', in fp32.
__device__ void sum_rows(const StreamParams& p, const Shared& ss) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d4 = p.d / 4, R = p.T * p.k;
  const int units = p.T * d4, step = gridDim.x * kMmaWarps * 32;
  for (int i = (warp * gridDim.x + blockIdx.x) * 32 + lane; i < units; i += step) {
    const int t = i / d4, c = (i - t * d4) * 4;
    float4 v[12];
#pragma unroll
    for (int j = 0; j < 12; ++j)
      if (j < p.k + p.S) {
        const int row = j < p.k ? ss.pick_row[t * p.k + j] : R + (j - p.k) * p.T + t;
        v[j] = __ldcg(reinterpret_cast<const float4*>(p.o + static_cast<size_t>(row) * p.d + c));
      }
    float4 a = v[0];
#pragma unroll
    for (int j = 1; j < 12; ++j)
      if (j < p.k + p.S) a.x += v[j].x, a.y += v[j].y, a.z += v[j].z, a.w += v[j].w;
    const size_t at = static_cast<size_t>(t) * p.d + c;
    if (p.y_type == MOE_Y_BF16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = a;
    }
  }
}

template <int G, bool LAYER>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(const __grid_constant__ StreamParams p) {
  extern __shared__ uint8_t dyn[];
  Shared& ss = *reinterpret_cast<Shared*>(dyn);
  float* xbuf = reinterpret_cast<float*>(dyn + kSharedBytes);
  // stages on 1024-byte boundaries of shared memory (the swizzle's period)
  const uint32_t ring_at = (smem_u32(xbuf) + p.xbuf_bytes + 1023u) & ~1023u;
  uint8_t* ring = dyn + (ring_at - smem_u32(dyn));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ss.full_w[i], 1);
      mbar_init(&ss.full_x[i], 32);
      mbar_init(&ss.empty[i], kMmaWarps);
    }
    for (int i = 0; i < kRowGroups; ++i) {
      mbar_init(&ss.xfull[i], 1);
      mbar_init(&ss.xfree[i], 1);
    }
    ss.abort = 0;
    fence_mbar_init();
  }
  if (LAYER) {
    build_work_list<Geo<G>::COLS>(p, ss);
  } else {
    const int per = (p.T + Geo<G>::COLS - 1) / Geo<G>::COLS;
    if (tid < p.T) ss.row_token[tid] = static_cast<unsigned char>(tid);
    if (tid == 0) {
      ss.nact = 1;
      ss.nblk = per;
      ss.e[0] = 0;
      ss.m[0] = p.T;
      ss.row0[0] = 0;
      ss.blk0[0] = 0;
      ss.blk0[1] = per;
    }
    __syncthreads();
  }
  volatile int* abort = &ss.abort;
  const int arrivals = kRowGroups * gridDim.x;
  if (warp == kWeightWarp) {
    if (lane == 0) {
      Ring rg;
      Drain dr;
      bool ok = true;
      if (LAYER) ok = produce_weights<G>(p, 0, ss, ring, rg, dr, abort);
      if (ok) produce_weights<G>(p, 1, ss, ring, rg, dr, abort);
      dr.wait(ss.full_w);
    }
    __syncwarp();
  } else if (warp == kColumnWarp) {
    Ring rg;
    bool ok = true;
    if (LAYER) {
      ok = produce_columns<G, LAYER>(p, 0, ss, ring, rg, abort);
      if (ok) {  // every hidden value of every CTA
        if (lane == 0) ok = wait_count(p.err + kCtrHidden, arrivals, abort, p.err, 0x25 << 24);
        ok = __shfl_sync(kFull, ok, 0);
      }
    }
    if (ok) produce_columns<G, LAYER>(p, 1, ss, ring, rg, abort);
    cp_async_wait_all();
  } else {
    Consumer cs;
    bool ok;
    if (LAYER) {
      // Counted even after a wait that gave up, so that the counters come
      // back to 0 and the other CTAs go on (the error word is set by then).
      auto publish = [&](int counter) {
        __syncwarp();
        if (warp < kRowGroups && lane == 0) red_release_gpu_add(p.err + counter, 1);
      };
      ok = consume<G, LAYER, 1>(p, 0, ss, ring, xbuf, cs, abort);
      publish(kCtrHidden);
      if (ok) ok = p.parts == 3 ? consume<G, LAYER, 3>(p, 1, ss, ring, xbuf, cs, abort)
                                : consume<G, LAYER, 2>(p, 1, ss, ring, xbuf, cs, abort);
      publish(kCtrOut);
      if (lane == 0) ok = ok && wait_count(p.err + kCtrOut, arrivals, abort, p.err, 0x26 << 24);
      if (__shfl_sync(kFull, ok, 0)) sum_rows(p, ss);
    } else {
      consume<G, LAYER, 1>(p, 1, ss, ring, xbuf, cs, abort);
    }
  }
  if (LAYER) {  // the last CTA to pass its waits clears the counters
    __syncthreads();
    if (tid == 0 && atomicAdd(p.err + kCtrExit, 1) == static_cast<int>(gridDim.x) - 1) {
      p.err[kCtrHidden] = 0;
      p.err[kCtrOut] = 0;
      p.err[kCtrExit] = 0;
    }
  }
}

// -------------------------------------------------------------------- host
// Ranges the K blocks are cut into: one per SM of the device, whatever the
// grid, so that a capped grid gives the same bits.
int workers() { return std::min(num_sms(), kMaxWorkers); }

struct Layout {
  size_t part, arrive, h, o, total;
};
// Error region (with the counters), parts, their arrival counters, hidden rows, output rows.
Layout layout(size_t rows, size_t d, size_t f) {
  Layout L{};
  size_t o = kErrRegionBytes;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.arrive = take(sizeof(int) * 2 * kMaxWorkers * kRowGroups);
  L.part = take(sizeof(float) * kMaxWorkers * kRowGroups * 16 * 32);
  L.h = take(3 * sizeof(uint16_t) * rows * f);
  L.o = take(sizeof(float) * rows * d);
  L.total = o;
  return L;
}

template <int G>
bool fill_product(Product& pr, int which, const DecodeWeight& w0, const DecodeWeight& w1, uint64_t mats, int rows, int K) {
  using Ge = Geo<G>;
  pr.K = K;
  pr.kblocks = ceil_div(K, Ge::KB);
  pr.rows = rows;
  pr.row_step = which == 0 ? kBoxRows : 2 * kBoxRows;
  pr.row_tiles = ceil_div(rows, pr.row_step);
  auto box = [&](CUtensorMap* m, const DecodeWeight& w) {
    return Ge::Q4 ? map2d_any(m, w.w, 1, K / 2, mats * rows, 128, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B)
                  : map2d(m, w.w, K, mats * rows, 64, kBoxRows);
  };
  bool ok = box(&pr.w0, w0);
  if (w1.w == w0.w)
    pr.w1 = pr.w0;
  else
    ok = ok && box(&pr.w1, w1);
  if constexpr (Ge::Q4) {
    auto sc = [&](CUtensorMap* m, const DecodeWeight& w) {
      return map2d_any(m, w.scales, 2, q4_scale_pitch(rows), mats * (K / G), kBoxRows, Ge::GROUPS,
                       CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    ok = ok && sc(&pr.s0, w0);
    if (w1.scales == w0.scales)
      pr.s1 = pr.s0;
    else
      ok = ok && sc(&pr.s1, w1);
  }
  return ok;
}

constexpr int kSmemMax = 232448;  // 227 KB

// Stages that fit beside the tables, and the launch's shared memory.
template <int G>
size_t ring_shape(StreamParams& p, int parts) {
  using Ge = Geo<G>;
  const int cols = std::min(p.T, Ge::COLS);
  const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
  p.cols8 = nt * 8;  // rows that the widest tile's instructions read
  p.xbuf_bytes = kRowGroups * 32 * nt * 4 * static_cast<int>(sizeof(float));
  p.stage_bytes = static_cast<int>(align_up(2 * (kBoxBytes + Ge::SCALE_BYTES) + parts * p.cols8 * Ge::PITCH, 1024));
  const size_t fixed = kSharedBytes + p.xbuf_bytes + 1024;
  p.stages = std::min<int>(kMaxStages, static_cast<int>((kSmemMax - fixed) / p.stage_bytes));
  return fixed + static_cast<size_t>(p.stages) * p.stage_bytes;
}

template <int G, bool LAYER>
int launch_stream(StreamParams& p, size_t smem, int grid_limit, cudaStream_t s) {
  static bool sized = false;  // the attribute outlives the call; setting it twice is harmless
  if (!sized) {
    if (cudaFuncSetAttribute(stream_kernel<G, LAYER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return MOE_ERR_CUDA;
    sized = true;
  }
  const int grid = grid_limit > 0 ? std::min(grid_limit, p.workers) : p.workers;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident: they wait on one another
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, stream_kernel<G, LAYER>, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int G>
int decode_g(const DecodeArgs& a, cudaStream_t s) {
  const moe_cfg& c = a.c;
  StreamParams p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t mats = c.E + c.n_shared;
  if (!fill_product<G>(p.p[0], 0, a.W1, a.W3, mats, c.d_ff, c.d_model) ||
      !fill_product<G>(p.p[1], 1, a.W2, a.W2, mats, c.d_model, c.d_ff))
    return MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const Layout L = layout(static_cast<size_t>(c.T) * (c.k + c.n_shared), c.d_model, c.d_ff);
  p.T = c.T, p.d = c.d_model, p.f = c.d_ff, p.E = c.E, p.k = c.k, p.S = c.n_shared, p.renorm = c.renorm;
  p.logits = a.logits, p.x = a.x, p.topk_idx = a.topk_idx, p.topk_w = a.topk_w;
  p.h = reinterpret_cast<uint16_t*>(ws + L.h);
  p.o = reinterpret_cast<float*>(ws + L.o);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.arrive = reinterpret_cast<int*>(ws + L.arrive);
  p.y = a.y, p.y_type = a.y_type, p.err = reinterpret_cast<int*>(ws), p.workers = workers();
  p.parts = a.y_type == MOE_Y_F32 ? 3 : 2;
  const size_t smem = ring_shape<G>(p, p.parts);
  TraceScope trace_scope(MOE_K_DECODE, s);
  return launch_stream<G, true>(p, smem, a.grid_limit, s);
}

template <int G>
int linear_g(const LinearArgs& a, cudaStream_t s) {
  StreamParams p;
  std::memset(&p, 0, sizeof(p));
  if (!fill_product<G>(p.p[1], 1, a.W, a.W, 1, a.n, a.K)) return MOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const Layout L = layout(0, 0, 0);
  p.T = a.T, p.n = a.n, p.x = a.x;
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.arrive = reinterpret_cast<int*>(ws + L.arrive);
  p.y = a.y, p.y_type = a.y_type, p.err = reinterpret_cast<int*>(ws), p.workers = workers();
  const size_t smem = ring_shape<G>(p, 1);
  TraceScope trace_scope(MOE_K_LINEAR, s);
  return launch_stream<G, false>(p, smem, a.grid_limit, s);
}

}  // namespace

size_t decode_workspace_bytes(const moe_cfg& c) {
  return layout(static_cast<size_t>(c.T) * (c.k + c.n_shared), c.d_model, c.d_ff).total;
}
size_t linear_workspace_bytes() { return layout(0, 0, 0).total; }

int decode_ws_init(void* ws, cudaStream_t s) {
  // error word and counters, then the arrival counters, which follow them
  return cudaMemsetAsync(ws, 0, layout(0, 0, 0).part, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_decode(const DecodeArgs& a, cudaStream_t s) {
  switch (a.group) {
    case 0: return decode_g<0>(a, s);
    case 32: return decode_g<32>(a, s);
    case 64: return decode_g<64>(a, s);
    default: return decode_g<128>(a, s);
  }
}

int launch_linear(const LinearArgs& a, cudaStream_t s) {
  switch (a.group) {
    case 0: return linear_g<0>(a, s);
    case 32: return linear_g<32>(a, s);
    case 64: return linear_g<64>(a, s);
    default: return linear_g<128>(a, s);
  }
}

}  // namespace moe
