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
//     tiles (two TMA boxes of 128 rows x 128 bytes), 96 to 192 KB in flight
//     per SM.  It needs nothing but the routing, so it runs ahead into W2
//     while the hidden values of this and other CTAs are still being made:
//     the grid-wide dependency between the two products costs no bandwidth.
//   - A second producer brings the activation rows of the same tiles (the
//     tokens of an expert four at a time by TMA gather) and is the one that
//     waits for the hidden values of all CTAs before the second product.
//   - tcgen05: the weights are the 128-row operand, the tokens its columns,
//     so a handful of tokens costs the smallest instruction (N = 16).
//     bf16 weights are read from the stage.  4-bit codes are turned into
//     bf16 pairs by the warps that own the tile's rows, one thread a row, and
//     go to tensor memory, from where the instruction takes them: written
//     back to shared memory they would need four times the codes' bandwidth
//     there, twice.  Each group of columns is summed from zero and scaled in
//     fp32 on its way out, so no weight is rounded.  Operand and sums are
//     double-buffered: a warp turns codes while its last ones are multiplied.
//   - The tiles of all picked experts form one sequence of K blocks, cut into
//     equal contiguous ranges, one per SM, so no SM idles whatever the number
//     of experts, rows and tokens.  Every range that works on a cut tile
//     leaves its sums in the workspace and, once through its range, adds up
//     all of them, in range order, for its share of the tile's columns: no
//     floating-point atomics, and nobody waits in the middle of a range.
//     Where whole tiles are as fast, they are dealt or drawn whole.
//
// What it measures (a call in a graph, 1 to 2 us more for calls one by one;
// GB/s are of the bytes that have to be moved, the copy rate is 6770):
//   d=2048 f=1408 E=64 k=6 S=2, bf16: 1 token 39.2 us, 3530 GB/s; 64 tokens
//     197 to 201 us, 5780 GB/s (7100 while it streams).  One token: start and
//     router 5 us; W1 and W3 17 us, whole tiles on 88 SMs; W2 10 us, on 64; two
//     grid-wide meetings 5 us.
//   The same in 4 bits: 1 token 28.6 us; d=4096 f=14336 E=8 k=2, 16 tokens
//     164 us, 4550 GB/s.  An SM spends 1470 clocks on a K block of 32 KB while
//     it streams, with 90 % of its issue slots taken; turning the codes takes
//     906 at the least (measured alone: 5 integer instructions at half rate and
//     4 multiply-adds a word).
//   Linear form: 37 rows x 4097 x 4096 bf16 17.6 us, 1 row x 14336 x 4096 in 4
//     bits 15.8 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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

constexpr int kSets = 4;                 // of four row warps each, which cover the 128 rows of a tile
constexpr int kRowWarps = 4 * kSets;
constexpr int kWeightWarp = kRowWarps;   // producer of weight tiles
constexpr int kColumnWarp = kRowWarps + 1;  // producer of activation rows
constexpr int kMmaWarp = kRowWarps + 2;     // issues the tensor instructions; 4 bits: the first box's, the next warp the second's
constexpr int kWarps = kRowWarps + 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileRows = 128;           // rows of one weight box: an accumulator's lanes
constexpr int kBoxBytes = kTileRows * 128;
constexpr int kTmemCols = 512;
// bf16 weights: the tensor core cuts off what its running sum has no room for,
// always towards zero, which over K = 3840 comes to 1e-5 of an output.  For an
// fp32 y it adds up 3 K blocks (12 instructions) at a time, 4 where there are
// no two pairs of accumulators, and the row warps add those sums, rounded to
// nearest, in the last columns of tensor memory: 5e-7 to 7e-7, about what fp32
// multiply-adds come to.  A bf16 y, off by 2^-9, needs none of it.
constexpr int kRunBlocks = 3, kRunBlocksAlone = 4;
constexpr int kRunCols = 2 * MOE_DECODE_MAX_T;
// 4 bits: tensor memory of one of two buffers of a set of row warps, operand
// and sums.
constexpr int kBufferCols = 64;
constexpr int kMaxStages = 8;
constexpr int kTileSlots = 4;            // drawn tiles on their way to the other roles
constexpr int kMaxTokens = MOE_DECODE_MAX_T;
constexpr int kMaxPicks = kMaxTokens * 8;
constexpr int kMaxRows = kMaxTokens * 12;   // k <= 8 slots and 4 shared experts
// Experts in the work list: all routed ones and the shared ones.
constexpr int kMaxActive = 256 + 4;
// Most ranges (SMs) that a workspace has room for.
constexpr int kMaxWorkers = 256;

// Counters in the error region (ints), all 0 between launches.
constexpr int kCtrHidden = 8;   // CTAs through the first product; the next one: through the second
constexpr int kCtrExit = 10;    // CTAs done
constexpr int kCtrRouted = 11;  // tokens routed, where the CTAs share the routing
constexpr int kCtrTicket = 12;  // tiles drawn, by product
constexpr int kCtrEnd = 14;

// K blocks of W2 that a CTA asks into L2 when its part of the first product
// is on the way, beyond what its ring holds, where whole tiles are drawn.
// Memory then stays busy while the hidden values of all CTAs come together:
// 64 tokens of d=2048 f=1408 E=64 k=6 S=2 199 -> 197 us.  Cut tiles, whose
// parts are on their way at that time, measured 3% slower with it.
constexpr int kPrefetchBlocks = 6;

// A stage: 128 bytes of 2 x 128 weight rows, the scales of those columns (4
// bits) and the activation rows, 64 columns (128 bytes, swizzled) at a time.
// G: columns of a scale group, 0 for bf16 weights.
template <int G>
struct Geo {
  static constexpr bool Q4 = G != 0;
  static constexpr int KB = Q4 ? 256 : 64;                     // columns
  static constexpr int ATOMS = KB / 64;
  static constexpr int GROUPS = Q4 ? KB / (Q4 ? G : 1) : 0;    // scale rows
  static constexpr int SCALE_BYTES = GROUPS * kTileRows * 2;   // of one box
  static constexpr int WEIGHT_BYTES = 2 * (kBoxBytes + SCALE_BYTES);
  // Activation rows of a tile, in `parts` parts.  bf16 weights: all of an
  // expert's.  4 bits: what a buffer in tensor memory and a thread hold; an
  // expert with more rows has its weight tiles visited again, from L2.  Groups
  // of 32 come with half the pushes where rows are 16 at a time, so that two
  // visits cost what one for 32 rows does and the ranges come out even (33
  // tokens of d=4096 f=2048 E=128 k=8, skewed: 127 us against 147).
  static constexpr int block_log2(int parts) { return !Q4 ? 6 : parts == 1 && G != 32 ? 5 : 4; }
};

// What the columns of a product are.
//   kRowsOfX   the T rows of x (linear form)
//   kGathered  the rows of x of an expert's tokens (hidden values)
//   kRowsOfH   an expert's rows of h, all parts (output rows)
enum Kind { kRowsOfX, kGathered, kRowsOfH };

// One product of the launch: weight tiles of `row_step` output rows.
struct Product {
  CUtensorMap w0, w1;   // weight boxes: W1 and W3, or (the same) the two halves of a W2 tile
  CUtensorMap s0, s1;   // their scales (4 bits)
  CUtensorMap cols;     // activation rows
  int K, kblocks, rows, row_step, row_tiles;
  int block_log2;       // log2 of the most activation rows of a tile
};

struct StreamParams {
  Product p[2];         // layer: hidden, out; linear form: the second only
  int T, d, f, E, k, S, renorm, n;
  const float* logits;
  int32_t* topk_idx;
  float* topk_w;
  uint16_t* h;          // [parts][Rs][f]
  float* o;             // [Rs][d]
  float* part;          // sums of the tiles that a range begins and ends in: [workers][2][2 boxes][64][128]
  int* arrive;          // what has come in, by the first range of the tile: [2][workers]
  void* y;
  int* err;             // error word and counters
  int y_type, workers, stages, stage_bytes;
  int parts;            // bf16 parts of a hidden value
  int acc_cols, acc_bufs;  // bf16 weights: columns of an accumulator, accumulator pairs
  int run;                 // bf16 weights, fp32 y: K blocks that the tensor core adds up at a time
  int drop;                // testing aid: counts that are left out (kDrop...), 0: none
};

// Counts that the testing aid leaves out, so that the waits for them run out.
constexpr int kDropRouted = 1;   // token 0's routing, where the CTAs share it
constexpr int kDropParts = 2;    // all parts of cut tiles
constexpr int kDropMeeting = 3;  // CTA 0 at the end of the first product; the next one: of the second
constexpr int kDropMax = 4;
int g_drop = 0;

// One product's K blocks and their ranges: range v takes q grains, one more if
// v < extra.  The first range of this CTA begins at K block u of tile `item`,
// which is tile r of row tile rt and belongs to work list entry a.
struct Plan {
  int units, workers, grain, q, extra;   // grain: K blocks that a range takes at least of a tile
  int per, tiles;                        // tiles of a row tile, and of the product
  bool drawn;                            // whole tiles, drawn by the CTAs
  int u, item, rt, r, a;
  __device__ int begin_of(int v) const { return (v * q + min(v, extra)) * grain; }
  // The range that holds K block `unit`.
  __device__ int worker_of(int unit) const {
    const unsigned g = static_cast<unsigned>(unit) / static_cast<unsigned>(grain), wide = extra * (q + 1);
    return g < wide ? g / static_cast<unsigned>(q + 1) : extra + (g - wide) / static_cast<unsigned>(q);
  }
};

struct alignas(16) Shared {
  uint64_t full_w[kMaxStages], full_x[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[2], acc_empty[2];   // bf16: accumulator pairs
  uint64_t a_ready[2][2], d_full[2][2]; // 4 bits: [box][buffer]
  uint64_t swap_ready, swap_done;       // 4 bits: all sums of a tile in tensor memory
  uint64_t rows_done[2];                // this CTA's row warps are through a product: a barrier for each, as the
                                        // second may be over (no work) before anyone looked at the first
  uint64_t out_done;                    // every CTA's output rows are there
  uint64_t tile_full[kTileSlots], tile_empty[kTileSlots];
  int4 tile[kTileSlots];                // drawn tiles: item (-1: no more), entry, row tile, block
  uint64_t drained;                     // tensor instructions all complete
  uint32_t tmem;
  int abort;
  int nact, nblk[2];               // work list entries; blocks of rows in all, by product
  int e[kMaxActive];               // expert
  int m[kMaxActive];               // its rows
  int row0[kMaxActive];            // its first row in h and o
  int blk0[2][kMaxActive + 1];     // blocks of rows before it, by product
  Plan plan[2];                    // by product
  unsigned mask[256][2];           // tokens that picked expert e
  float row_w[kMaxRows];
  float pick_w[kMaxPicks];
  short pick_e[kMaxPicks];
  short pick_row[kMaxPicks];
  short entry[256];                // expert's place in the work list
  unsigned scan[8][2];             // packed sums of 32 experts each
  unsigned char row_token[kMaxRows];
};
constexpr int kSharedBytes = (sizeof(Shared) + 127) / 128 * 128;

// Waits until `target` arrivals are counted (bounded).
__device__ bool wait_count(const int* c, int target, volatile int* abort, int* err, int where) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (ld_acquire_gpu(c) >= target) return true;
    if (*abort) return false;
    if (t0 == 0) t0 = globaltimer_ns();
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, MOE_ERR_TIMEOUT_CODE, where);
      *abort = 1;
      return false;
    }
  }
}

// ---------------------------------------------------------------- work list
// The K blocks of a product, tile after tile, cut into contiguous ranges.
// The tiles of one row tile of all experts follow each other, so the shared
// experts, which have the most rows to finish, are spread over the ranges.
//
// Whole tiles or cut ones.  In units of 0.37 us: with all SMs at work a K
// block of 32 KB takes 2 of them (bf16: memory) or 3 (4 bits: turning codes);
// an SM that has the memory to itself takes 1 for a bf16 block.  Putting cut
// tiles together again costs 12 more (parts, count, wait, parts back).  Whole
// tiles take turns of all SMs and a last turn of the rest; one token's 88
// tiles of W1 and W3 of the layer d=2048 f=1408 k=6 S=2 are faster whole on 88
// SMs than cut for 152, 17 tiles of a 4097 x 4096 matrix are not.  No range of
// a cut product has fewer than kMinBlocks.  The estimate takes equal blocks as
// equal in time, which they are not where the SMs' shares of the memory's rate
// or the experts' rows differ: the ranges of 33 skewed tokens in 4 bits end
// between 97,000 and 160,000 clocks.
//
// Whole tiles of several turns are drawn from a counter: the SMs do not get
// equal shares of the memory's rate (64 tokens of that layer: 160,000 clocks
// for the first product on one SM, 246,000 on another with as many tiles).
// A tile's sums do not depend on the CTA that makes them.
constexpr int kMinBlocks = 3, kJoinUnits = 12;

template <bool Q4>
__device__ void make_plan(const StreamParams& p, int which, Shared& ss) {
  const Product& pr = p.p[which];
  Plan& pl = ss.plan[which];
  pl.per = ss.nblk[which];
  const int tiles = pl.per * pr.row_tiles, turns = tiles / p.workers, rest = tiles - turns * p.workers;
  pl.units = tiles * pr.kblocks;
  const int each = Q4 ? 3 : 2;
  const int whole_time = Q4 ? 3 * pr.kblocks * (turns + (rest > 0))
                            : pr.kblocks * each * turns + (rest ? max(pr.kblocks, each * pr.kblocks * rest / p.workers) : 0);
  const int cut_time = each * (pl.units / p.workers) + kJoinUnits;
  const bool whole = whole_time <= cut_time;
  pl.tiles = tiles;
  pl.drawn = whole && tiles > p.workers;
  pl.grain = whole ? pr.kblocks : 1;
  const int grains = whole ? tiles : pl.units;
  pl.workers = max(1, min(p.workers, whole ? grains : grains / kMinBlocks));  // no range is empty
  pl.q = grains / pl.workers;
  pl.extra = grains - pl.q * pl.workers;
  const int v = min(static_cast<int>(blockIdx.x), pl.workers - 1);
  pl.u = pl.begin_of(v);
  pl.item = pl.u / pr.kblocks;
  pl.rt = pl.item / pl.per;
  pl.r = pl.item - pl.rt * pl.per;
  int lo = 0, hi = ss.nact - 1;   // last entry with blk0 <= r
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (ss.blk0[which][mid] <= pl.r)
      lo = mid;
    else
      hi = mid - 1;
  }
  pl.a = lo;
}

// Routes the tokens.  Up to kWarps tokens: every CTA all of them, one warp a
// token.  More: token t is CTA t % gridDim.x's, and every CTA reads the picks
// of the others from the outputs once all are counted; 64 tokens routed by
// every CTA itself took 8 us, most of them in the warps' serial pick rounds.
// A token picks an expert at most once, so an expert's tokens are a 64-bit
// mask and a row's place in its expert's list is a population count:
// ascending tokens, whatever the order of the atomics that set the bits.
__device__ __forceinline__ void note_pick(Shared& ss, int at, int t, int e, float w) {
  ss.pick_e[at] = static_cast<short>(e);
  ss.pick_w[at] = w;
  atomicOr(&ss.mask[e][t >> 5], 1u << (t & 31));
}

template <int EPL>
__device__ __noinline__ void route_all(const StreamParams& p, Shared& ss) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool shared_out = p.T > kWarps;
  const int step = shared_out ? gridDim.x * kWarps : kWarps;
  int t = shared_out ? blockIdx.x + warp * gridDim.x : warp;
  RowSoftmax<EPL> r;
  if (t < p.T) row_load<EPL>(p.logits + static_cast<size_t>(t) * p.E, p.E, lane, r.v);  // in flight while the masks are cleared
  if (threadIdx.x < 512) (&ss.mask[0][0])[threadIdx.x] = 0;
  __syncthreads();
  while (t < p.T) {
    int idx;
    float w;
    route_token<EPL>(r, t, p.E, p.k, p.renorm, lane, p.err, idx, w);
    if (lane < p.k) {
      const int at = t * p.k + lane;
      if (!shared_out) note_pick(ss, at, t, idx, w);
      if (shared_out || blockIdx.x == 0) {
        p.topk_idx[at] = idx;
        p.topk_w[at] = w;
      }
    }
    if (shared_out) {
      __syncwarp();
      if (lane == 0 && (t != 0 || p.drop != kDropRouted)) red_release_gpu_add(p.err + kCtrRouted, 1);
    }
    t += step;
    if (t < p.T) row_load<EPL>(p.logits + static_cast<size_t>(t) * p.E, p.E, lane, r.v);
  }
}

template <bool Q4>
__device__ void build_work_list(const StreamParams& p, Shared& ss) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.T * p.k;
  if (p.E <= 32)
    route_all<1>(p, ss);
  else if (p.E <= 64)
    route_all<2>(p, ss);
  else if (p.E <= 128)
    route_all<4>(p, ss);
  else
    route_all<8>(p, ss);
  if (p.T > kWarps) {
    if (tid == 0) wait_count(p.err + kCtrRouted, p.T, &ss.abort, p.err, 0x20 << 24);
    __syncthreads();
    // After a wait that gave up (abort is set) the picks may be anything: clamped, they stay in bounds.
    for (int t = tid >> 3; t < p.T; t += kThreads / 8)
      if (const int i = t * p.k + (tid & 7); (tid & 7) < p.k)
        note_pick(ss, i, t, min(max(__ldcg(p.topk_idx + i), 0), p.E - 1), __ldcg(p.topk_w + i));
  }
  __syncthreads();
  // Thread e: expert e.  Exclusive sums over the experts of rows and entries
  // (at most 512 and 256) and of either product's blocks of rows (at most
  // 288), packed in pairs.
  unsigned mine[2] = {}, incl[2] = {};
  int n = 0;
  auto blocks = [&](int which, int rows) { return (rows + (1 << p.p[which].block_log2) - 1) >> p.p[which].block_log2; };
  if (tid < 256) {
    n = tid < p.E ? __popc(ss.mask[tid][0]) + __popc(ss.mask[tid][1]) : 0;
    mine[0] = n ? n | 1 << 16 : 0;
    mine[1] = blocks(0, n) | blocks(1, n) << 16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      incl[j] = mine[j];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned x = __shfl_up_sync(kFull, incl[j], off);
        if (lane >= off) incl[j] += x;
      }
      if (lane == 31) ss.scan[warp][j] = incl[j];
    }
  }
  __syncthreads();
  unsigned before[2] = {}, all[2] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const unsigned x = ss.scan[i][j];
      if (i < warp) before[j] += x;
      all[j] += x;
    }
  const int all_a = all[0] >> 16, all_b[2] = {static_cast<int>(all[1] & 0xFFFF), static_cast<int>(all[1] >> 16)};
  if (tid < 256 && n) {
    const unsigned at = before[0] + incl[0] - mine[0], blk = before[1] + incl[1] - mine[1];
    const int a = at >> 16;
    ss.entry[tid] = static_cast<short>(a);
    ss.e[a] = tid;
    ss.m[a] = n;
    ss.row0[a] = at & 0xFFFF;
    ss.blk0[0][a] = blk & 0xFFFF;
    ss.blk0[1][a] = blk >> 16;
  }
  if (tid < p.S) {
    ss.e[all_a + tid] = p.E + tid;
    ss.m[all_a + tid] = p.T;
    ss.row0[all_a + tid] = R + tid * p.T;
  }
  if (tid <= p.S) {  // the shared experts' blocks, and the ends
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = all_b[j] + tid * blocks(j, p.T);
      ss.blk0[j][all_a + tid] = at;
      if (tid == p.S) ss.nblk[j] = at;
    }
    if (tid == p.S) ss.nact = all_a + p.S;
  }
  __syncthreads();
  if (tid == kThreads - 32 || tid == kThreads - 64) {
    make_plan<Q4>(p, tid == kThreads - 64, ss);
  } else {
    // rows: first row of the expert + earlier tokens of its mask; eight lanes a token
    const int j = tid & 7;
    for (int t = tid >> 3; t < p.T; t += kThreads / 8) {
      if (j < p.k) {
        const int i = t * p.k + j, e = ss.pick_e[i];
        const unsigned m0 = ss.mask[e][0], m1 = ss.mask[e][1], below = (1u << (t & 31)) - 1u;
        const int row = ss.row0[ss.entry[e]] + (t < 32 ? __popc(m0 & below) : __popc(m0) + __popc(m1 & below));
        ss.pick_row[i] = static_cast<short>(row);
        ss.row_token[row] = static_cast<unsigned char>(t);
        ss.row_w[row] = ss.pick_w[i];
      }
      if (j < p.S) {
        ss.row_token[R + j * p.T + t] = static_cast<unsigned char>(t);
        ss.row_w[R + j * p.T + t] = 1.f;
      }
    }
  }
}

// Every role of a CTA walks the same segments: the K blocks [kb0, kb1) of one
// tile.  The ranges and the first position come from the plan: the few
// divisions take a lone warp a microsecond and more, on every role's way to
// its first copy.
struct Segment {
  int worker, item, kb0, kb1;
  int a, rt, nb;   // work list entry, row tile, block of the expert's rows
};

struct Walk {
  const Product& pr;
  const Plan& pl;
  const int* blk0;
  int v, u, u1;
  int item, rt, r, a, kb;

  __device__ Walk(const StreamParams& p, int which, const Shared& ss)
      : pr(p.p[which]), pl(ss.plan[which]), blk0(ss.blk0[which]) {
    v = static_cast<int>(blockIdx.x);
    u = u1 = 0;
    if (v >= pl.workers) return;
    u = pl.u;
    u1 = pl.begin_of(v + 1);
    item = pl.item, rt = pl.rt, r = pl.r, a = pl.a;
    kb = u - item * pr.kblocks;
  }
  __device__ bool next(Segment& s) {
    if (u >= u1) {  // a capped grid: the CTA's next range
      if (v >= pl.workers || (v += static_cast<int>(gridDim.x)) >= pl.workers) return false;
      u = pl.begin_of(v);
      u1 = pl.begin_of(v + 1);
      item = u / pr.kblocks;
      kb = u - item * pr.kblocks;
      rt = item / pl.per;
      r = item - rt * pl.per;
      a = 0;
    }
    while (r >= blk0[a + 1]) ++a;
    s.worker = v;
    s.item = item;
    s.kb0 = kb;
    s.kb1 = min(pr.kblocks, kb + (u1 - u));
    s.a = a;
    s.rt = rt;
    s.nb = r - blk0[a];
    u += s.kb1 - s.kb0;
    kb = 0;
    ++item;
    if (++r == pl.per) {
      r = 0;
      a = 0;
      ++rt;
    }
    return true;
  }
};

// The segments of a product for one role.  Where tiles are drawn, the producer
// of weights draws them and passes them on through a short queue.
struct Queue {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kTileSlots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// A whole warp's wait.  INLINE: the first poll in the open, without a call,
// where the warps' instructions are what bounds the kernel (4 bits, 3%); bf16
// weights measured 4% faster without it.
template <bool INLINE>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err, int where) {
  if (INLINE && __all_sync(kFull, mbar_try_wait(smem_u32(bar), parity))) return true;
  const bool ok = mbar_wait(bar, parity, abort, err, where);
  return __all_sync(kFull, ok);
}

template <bool DRAWS>
struct Tiles {
  Walk walk;
  const StreamParams& p;
  Shared& ss;
  Queue& queue;
  volatile int* abort;
  int which, ticket;
  bool through = true;  // false once a wait gave up: the role must not take the other product's tiles for this one's

  __device__ Tiles(const StreamParams& params, int product, Shared& shared, Queue& q, volatile int* ab)
      : walk(params, product, shared), p(params), ss(shared), queue(q), abort(ab), which(product), ticket(blockIdx.x) {}

  // Item, work list entry, row tile and block of a tile.
  __device__ int4 locate(int item) const {
    const int rt = item / walk.pl.per, r = item - rt * walk.pl.per;
    int lo = 0, hi = ss.nact - 1;   // last entry with blk0 <= r
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (walk.blk0[mid] <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    return make_int4(item, lo, rt, r - walk.blk0[lo]);
  }

  __device__ __forceinline__ bool next(Segment& s) {
    if (!walk.pl.drawn) return walk.next(s);
    const bool lead = (threadIdx.x & 31) == 0;
    int4 t;
    if (DRAWS) {
      const Plan& pl = walk.pl;
      const int item = __shfl_sync(kFull, ticket, 0);
      t = item < pl.tiles ? locate(item) : make_int4(-1, 0, 0, 0);
      if (!warp_wait<false>(&ss.tile_empty[queue.slot], queue.phase ^ 1, abort, p.err, 0x2B << 24)) return through = false;
      if (lead) {
        ss.tile[queue.slot] = t;
        mbar_arrive(&ss.tile_full[queue.slot]);
        // the next one's round trip overlaps this tile
        if (t.x >= 0) ticket = static_cast<int>(gridDim.x) + atomicAdd(p.err + kCtrTicket + which, 1);
      }
    } else {
      if (!warp_wait<false>(&ss.tile_full[queue.slot], queue.phase, abort, p.err, 0x2C << 24)) return through = false;
      t = ss.tile[queue.slot];
      __syncwarp();
      if (lead) mbar_arrive(&ss.tile_empty[queue.slot]);
    }
    queue.step();
    if (t.x < 0) return false;
    s.worker = 0;
    s.item = t.x;
    s.a = t.y;
    s.rt = t.z;
    s.nb = t.w;
    s.kb0 = 0;
    s.kb1 = walk.pr.kblocks;
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

// Columns of a tile, each part's rounded up to 16.
template <Kind KIND>
struct Columns {
  int m;       // real ones: rows of the expert in this tile
  int r0;      // its first row in h and o (linear form: in x)
  int n16;     // 16-row boxes of one part
  int n;       // columns of the tensor instruction
  __device__ Columns(const StreamParams& p, int which, const Shared& ss, const Segment& s) {
    const int log2 = p.p[which].block_log2, first = s.nb << log2;
    m = min(1 << log2, ss.m[s.a] - first);
    r0 = ss.row0[s.a] + first;
    n16 = (m + 15) / 16;
    n = 16 * n16 * (KIND == kRowsOfH ? p.parts : 1);
  }
};

// The producers and the issuer of the tensor instructions run as whole warps
// and elect a lane for the asynchronous instructions: their operands are warp
// registers, and the compiler gets them there without a loop over the lanes
// only where it sees that the warp is together (64 and more clocks an
// instruction otherwise, against 19 for the smallest tensor instruction).
template <int G, Kind KIND>
__device__ bool produce_weights(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg, Queue& qu, Drain& dr,
                                volatile int* abort) {
  using Ge = Geo<G>;
  const Product& pr = p.p[which];
  Tiles<true> walk(p, which, ss, qu, abort);
  Segment s;
  if (KIND == kRowsOfH && walk.walk.pl.drawn) {  // the tiles that the CTAs draw first
    int n = -p.stages;
    for (int item = blockIdx.x; item < walk.walk.pl.tiles && n < kPrefetchBlocks; item += gridDim.x) {
      const int4 t = walk.locate(item);
      const int row = ss.e[t.y] * pr.rows + t.z * pr.row_step;
      for (int kb = 0; kb < pr.kblocks && n < kPrefetchBlocks; ++kb, ++n)
        if (n >= 0 && elect_one()) {
          tma_prefetch_2d(&pr.w0, kb * (Ge::Q4 ? 128 : 64), row);
          tma_prefetch_2d(&pr.w1, kb * (Ge::Q4 ? 128 : 64), row + kTileRows);
        }
    }
    __syncwarp();
  }
  while (walk.next(s)) {
    const int row = ss.e[s.a] * pr.rows + s.rt * pr.row_step;
    const int beside = which == 0 ? 0 : kTileRows;  // W3 beside W1, or the tile's other rows
    [[maybe_unused]] const int scale_row = Ge::Q4 ? ss.e[s.a] * (pr.K / (Ge::Q4 ? G : 1)) : 0;
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
      if (!warp_wait<Ge::Q4>(&ss.empty[rg.stage], rg.phase ^ 1, abort, p.err, (0x21 << 24) | which)) return false;
      uint8_t* st = ring + static_cast<size_t>(rg.stage) * p.stage_bytes;
      uint64_t* bar = &ss.full_w[rg.stage];
      dr.note(rg.stage, rg.phase);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, Ge::WEIGHT_BYTES);
        const int col = kb * (Ge::Q4 ? 128 : 64);  // bytes or bf16
        tma_load_2d(st, &pr.w0, bar, col, row);
        tma_load_2d(st + kBoxBytes, &pr.w1, bar, col, row + beside);
        if constexpr (Ge::Q4) {
          uint8_t* sc = st + 2 * kBoxBytes;
          const int at = scale_row + kb * Ge::GROUPS, r0 = s.rt * pr.row_step;
          tma_load_2d(sc, &pr.s0, bar, r0, at);
          tma_load_2d(sc + Ge::SCALE_BYTES, &pr.s1, bar, r0 + beside, at);
        }
      }
      __syncwarp();
      rg.step(p.stages);
    }
  }
  return walk.through;
}

// Activation rows: 64 columns at a time, the parts of h below one another.
// What a box or a gather leaves of the 16 rows keeps old values; they are
// columns that nobody reads.
template <int G, Kind KIND>
__device__ bool produce_columns(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg, Queue& qu, Drain& dr,
                                volatile int* abort) {
  using Ge = Geo<G>;
  const Product& pr = p.p[which];
  const int Rs = p.T * (p.k + p.S);
  Tiles<false> walk(p, which, ss, qu, abort);
  Segment s;
  while (walk.next(s)) {
    const Columns<KIND> c(p, which, ss, s);
    const int gathers = (c.m + 3) / 4;
    const uint32_t bytes = Ge::ATOMS * (KIND == kGathered ? gathers * 512 : c.n * 128);
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
      if (!warp_wait<Ge::Q4>(&ss.empty[rg.stage], rg.phase ^ 1, abort, p.err, (0x22 << 24) | which)) return false;
      uint8_t* st = ring + static_cast<size_t>(rg.stage) * p.stage_bytes + Ge::WEIGHT_BYTES;
      uint64_t* bar = &ss.full_x[rg.stage];
      dr.note(rg.stage, rg.phase);
      if (elect_one()) {
        mbar_arrive_expect_tx(bar, bytes);
        if (KIND == kGathered) {
          for (int i = 0; i < gathers; ++i) {
            int t[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = ss.row_token[c.r0 + min(i * 4 + j, c.m - 1)];
#pragma unroll
            for (int at = 0; at < Ge::ATOMS; ++at)
              tma_gather4(st + at * c.n * 128 + i * 512, &pr.cols, bar, (kb * Ge::ATOMS + at) * 64, t[0], t[1], t[2], t[3]);
          }
        } else {
          const int parts = KIND == kRowsOfH ? p.parts : 1;
          for (int q = 0; q < parts; ++q)
            for (int i = 0; i < c.n16; ++i)
#pragma unroll
              for (int at = 0; at < Ge::ATOMS; ++at)
                tma_load_2d(st + at * c.n * 128 + (q * c.n16 + i) * 2048, &pr.cols, bar, (kb * Ge::ATOMS + at) * 64,
                            q * Rs + c.r0 + i * 16);
        }
      }
      __syncwarp();
      rg.step(p.stages);
    }
  }
  return walk.through;
}

// ----------------------------------------------------- tensor instructions
// bf16: position in the ring of accumulator pairs, one a segment.  4 bits: the
// buffers' phase, and which of them holds the sums of a group that fills a
// stage.
struct Turn {
  int buf = 0, sums = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step(int bufs) {
    if (++buf == bufs) {
      buf = 0;
      phase ^= 1;
    }
  }
};

// 4 bits: both sets of a box hand the tensor core 64 columns each at a time (a
// push): a group, two, or a part of one; 32 where a buffer would not hold the
// sums.  N16, PARTS: steps of 16 rows and their parts.  Pushes alternate
// between two buffers, and every stage makes the same number of them (empty
// ones behind K), so that everything about a push but its phase is known to
// the compiler: worked out by the row warps, four to a scheduler, that took as
// long as turning the codes.
constexpr int kChunk = 32;  // columns of 16 bytes of codes
template <int G, int N16, int PARTS>
struct Push {
  static constexpr int N = 16 * N16 * PARTS;
  static constexpr int GROUPS = G == 32 ? 2 : 1;                   // of a push of two chunks, at most
  static constexpr int SIZE = 2 * (kChunk / 2) + GROUPS * N <= kBufferCols ? 2 : 1;  // chunks of a set's push
  static constexpr int SLAB = G == 32 ? SIZE : G / kChunk;         // consecutive chunks that are one set's
  static constexpr int EACH = SLAB / SIZE;                         // pushes of a slab
  static constexpr int COUNT = Geo<G>::KB / kChunk / 2 / SIZE;     // pushes of a stage
  static_assert(SIZE * (kChunk / 2) + (SIZE == 2 ? GROUPS : 1) * N <= kBufferCols, "tensor memory of a buffer");
  // The first chunk of set 0's push j; set 1's is SLAB further on.
  __host__ __device__ static constexpr int first(int j) { return j / EACH * 2 * SLAB + j % EACH * SIZE; }
  __host__ __device__ static constexpr bool begins(int j) { return j % EACH == 0; }
  __host__ __device__ static constexpr bool ends(int j) { return j % EACH == EACH - 1; }
  __host__ __device__ static constexpr int buf(int j) { return j & 1; }
  static __device__ uint32_t phase(const Turn& tn, int j) { return tn.phase ^ ((j >> 1) & 1); }
  static __device__ int sums(const Turn& tn, int j) { return COUNT == EACH ? tn.sums : (j / EACH) & 1; }
  static __device__ void stage_done(Turn& tn) {
    if (COUNT == 2) tn.phase ^= 1;
    tn.sums ^= 1;
  }
  static __device__ int chunks(int K, int kb) { return min(Geo<G>::KB, K - kb * Geo<G>::KB) / kChunk; }
};
// Calls f with the Push of a segment.
template <int G, Kind KIND, typename F>
__device__ __forceinline__ bool with_push(int n16, int parts, const F& f) {
  if constexpr (KIND == kRowsOfH)  // at most 16 rows at a time, as with groups of 32
    return parts == 3 ? f(Push<G, 1, 3>{}) : f(Push<G, 1, 2>{});
  else if constexpr (G == 32)
    return f(Push<G, 1, 1>{});
  else
    return n16 == 1 ? f(Push<G, 1, 1>{}) : f(Push<G, 2, 1>{});
}
__device__ __forceinline__ uint32_t operand_at(uint32_t tmem, int box, int set, int buf) {
  return tmem + ((box * 2 + set) * 2 + buf) * kBufferCols;
}
__device__ __forceinline__ uint32_t sums_at(uint32_t tmem, int box, int set, int buf, int size) {
  return operand_at(tmem, box, set, buf) + size * (kChunk / 2);
}

template <Kind KIND, bool RUNS>
__device__ bool issue_bf16(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg, Queue& qu, Turn& tn,
                           volatile int* abort) {
  Tiles<false> walk(p, which, ss, qu, abort);
  Segment s;
  while (walk.next(s)) {
    const Columns<KIND> c(p, which, ss, s);
    const uint32_t idesc = idesc_bf16_f32(kTileRows, c.n, 0, 0);
    uint32_t acc = 0;
    const auto begin = [&]() {
      acc = ss.tmem + tn.buf * 2 * p.acc_cols;
      return warp_wait<false>(&ss.acc_empty[tn.buf], tn.phase ^ 1, abort, p.err, (0x31 << 24) | which);
    };
    if (!RUNS && !begin()) return false;
    for (int kb = s.kb0, done = 0; kb < s.kb1; ++kb) {
      if (RUNS && done == 0 && !begin()) return false;
      const uint32_t st = smem_u32(ring) + static_cast<uint32_t>(rg.stage) * p.stage_bytes;
      const uint32_t x = st + Geo<0>::WEIGHT_BYTES;
      if (!warp_wait<false>(&ss.full_x[rg.stage], rg.phase, abort, p.err, (0x24 << 24) | which)) return false;
      if (!warp_wait<false>(&ss.full_w[rg.stage], rg.phase, abort, p.err, (0x23 << 24) | which)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const uint64_t bd = smem_desc_sw128(x + k4 * 32, 16, 1024);
          const uint32_t go_on = ((RUNS ? done != 0 : kb != s.kb0) || k4 != 0) ? 1u : 0u;
#pragma unroll
          for (int box = 0; box < 2; ++box)
            umma_bf16(acc + box * p.acc_cols, smem_desc_sw128(st + box * kBoxBytes + k4 * 32, 16, 1024), bd, idesc, go_on);
        }
        umma_commit(&ss.empty[rg.stage]);
        if ((RUNS && done + 1 == p.run) || kb == s.kb1 - 1) umma_commit(&ss.acc_full[tn.buf]);
      }
      __syncwarp();
      rg.step(p.stages);
      if (RUNS && ++done == p.run && kb < s.kb1 - 1) {
        tn.step(p.acc_bufs);
        done = 0;
      }
    }
    tn.step(p.acc_bufs);
  }
  return walk.through;
}

template <int G, int N16, int PARTS>
__device__ __forceinline__ bool issue_segment(Push<G, N16, PARTS>, const StreamParams& p, int which, int box, Shared& ss,
                                              uint8_t* ring, const Segment& s, Ring& rg, Turn& tn, volatile int* abort) {
  using Pu = Push<G, N16, PARTS>;
  constexpr uint32_t idesc = idesc_bf16_f32(kTileRows, Pu::N, 0, 0);
  constexpr uint32_t atom = Pu::N * 128;  // 64 columns of the stage start this many bytes apart
  const uint32_t tmem = ss.tmem;
  for (int kb = s.kb0; kb < s.kb1; ++kb) {
    const uint32_t x = smem_u32(ring) + static_cast<uint32_t>(rg.stage) * p.stage_bytes + Geo<G>::WEIGHT_BYTES;
    const uint64_t xd = smem_desc_sw128(x, 16, 1024);
    const int chunks = Pu::chunks(p.p[which].K, kb);
    if (!warp_wait<true>(&ss.full_x[rg.stage], rg.phase, abort, p.err, (0x24 << 24) | which)) return false;
#pragma unroll
    for (int j = 0; j < Pu::COUNT; ++j) {
      if (!warp_wait<true>(&ss.a_ready[box][Pu::buf(j)], Pu::phase(tn, j), abort, p.err, (0x32 << 24) | which)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int set = 0; set < 2; ++set) {
          const int ch = Pu::first(j) + set * Pu::SLAB;
          if (ch >= chunks) continue;
          const uint32_t a = operand_at(tmem, box, set, Pu::buf(j)), d = sums_at(tmem, box, set, Pu::sums(tn, j), Pu::SIZE);
#pragma unroll
          for (int i = 0; i < 2 * Pu::SIZE; ++i)
            umma_bf16_ta(d + (G == 32 ? (i / 2) * Pu::N : 0), a + i * 8, xd + (ch / 2 * atom + ch % 2 * 64 + i * 32) / 16,
                         idesc, G == 32 ? i % 2 : i != 0 || !Pu::begins(j));
        }
        umma_commit(&ss.d_full[box][Pu::buf(j)]);
        if (j == Pu::COUNT - 1) umma_commit(&ss.empty[rg.stage]);
      }
      __syncwarp();
    }
    Pu::stage_done(tn);
    rg.step(p.stages);
  }
  return true;
}

template <int G, Kind KIND>
__device__ bool issue_q4(const StreamParams& p, int which, int box, Shared& ss, uint8_t* ring, Ring& rg, Queue& qu, Turn& tn,
                         volatile int* abort) {
  Tiles<false> walk(p, which, ss, qu, abort);
  Segment s;
  while (walk.next(s)) {
    const Columns<KIND> c(p, which, ss, s);
    if (!with_push<G, KIND>(c.n16, p.parts, [&](auto push) { return issue_segment(push, p, which, box, ss, ring, s, rg, tn, abort); }))
      return false;
  }
  return walk.through;
}

// --------------------------------------------------------------- row warps
// The hidden values enter the second product in bf16 parts that add up to
// them: two (16 significant bits) for a bf16 y, three (24) for an fp32 y.
// One part alone would cost 2^-9 of each value, as much as the rounding of a
// bf16 y, and the tensor instructions of more parts are free beside the
// weights' bytes.  The lower parts are held times 2^8, so that they leave
// bf16's range no sooner than the upper one does.
constexpr float kLowScale = 256.f;

__device__ __forceinline__ void store_hidden(const StreamParams& p, int r, int i, float w, float a, float b) {
  const float h = w * (a / (1.f + expf(-a)) * b);
  const size_t part_step = static_cast<size_t>(p.T) * (p.k + p.S) * p.f;
  uint16_t* to = p.h + static_cast<size_t>(r) * p.f + i;
  float rest = h;
  for (int q = 0; q < p.parts; ++q) {
    const __nv_bfloat16 v = __float2bfloat16_rn(rest);
    to[q * part_step] = __bfloat16_as_ushort(v);
    rest = (rest - __bfloat162float(v)) * (q == 0 ? kLowScale : 1.f);
    if (!isfinite(rest)) rest = 0.f;  // a value that rounds to infinity keeps that alone
  }
}

template <Kind KIND>
__device__ __forceinline__ void store_out(const StreamParams& p, int r, int c, float v) {
  if (KIND == kRowsOfH) {
    if (c < p.d) p.o[static_cast<size_t>(r) * p.d + c] = v;
  } else if (c < p.n) {
    const size_t at = static_cast<size_t>(r) * p.n + c;
    if (p.y_type == MOE_Y_BF16)
      static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(p.y)[at] = v;
  }
}

// Which share of its tile a segment is: all of it, or a part that ranges
// v0..v1 put together.  A range has at most two such parts: of the tile that
// it begins in the middle of (slot 0) and of the one that it does not end
// (slot 1).
struct Share {
  bool whole;
  int v0, v1;
  __device__ Share(const Walk& walk, const Segment& s) {
    const int kblocks = walk.pr.kblocks;
    whole = s.kb0 == 0 && s.kb1 == kblocks;
    v0 = s.kb0 == 0 ? s.worker : walk.pl.worker_of(s.item * kblocks);
    v1 = s.kb1 == kblocks ? s.worker : walk.pl.worker_of(s.item * kblocks + kblocks - 1);
  }
};
// Column 0 of a part, this thread's row.  Range v has the tile in slot 1 only
// if the tile begins there.
__device__ __forceinline__ float* part_of(const StreamParams& p, int v, bool begins, int box, int row) {
  return p.part + ((static_cast<size_t>(v) * 2 + begins) * 2 + box) * (kMaxTokens * kTileRows) + row;
}
__device__ __forceinline__ int* arrivals_of(const StreamParams& p, int which, int v0) {
  return p.arrive + static_cast<size_t>(which) * kMaxWorkers + v0;
}
// Counts a part in: a row warp's share of it (bf16), or all of it, by thread 0
// after a barrier of the row warps that is there anyhow (4 bits; 4% of a call
// at one token.  A barrier for this alone costs bf16 what it saves).
template <bool WARPS>
__device__ __forceinline__ void count_part(const StreamParams& p, int which, const Share& sh) {
  __syncwarp();
  if ((threadIdx.x & (WARPS ? 31 : ~0u)) == 0 && p.drop != kDropParts) red_release_gpu_add(arrivals_of(p, which, sh.v0), 1);
}

// A tile's finished column i, this thread's row of either box.
template <Kind KIND>
__device__ __forceinline__ void finish_column(const StreamParams& p, const Shared& ss, const Segment& s, int r0, int i,
                                              int row, float v0, float v1) {
  const int r = r0 + i;
  if (KIND == kGathered) {
    const int at = s.rt * kTileRows + row;
    if (at < p.f) store_hidden(p, r, at, ss.row_w[r], v0, v1);
  } else {
    store_out<KIND>(p, r, s.rt * 2 * kTileRows + row, v0);
    store_out<KIND>(p, r, (s.rt * 2 + 1) * kTileRows + row, v1);
  }
}

// After the segments of a product: the cut tiles of this CTA's ranges, this
// range's share of their columns (column i belongs to the i-th part, modulo
// the parts), dealt to the sets of row warps.
template <Kind KIND, bool WARPS>
__device__ bool join_parts(const StreamParams& p, int which, const Shared& ss, volatile int* abort) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (warp & 3) * 32 + lane, set = warp >> 2;
  if (ss.plan[which].grain > 1) return true;  // no tile is cut
  Walk walk(p, which, ss);
  Segment s;
  while (walk.next(s)) {
    const Share sh(walk, s);
    if (sh.whole) continue;
    const Columns<KIND> c(p, which, ss, s);
    const int parts = sh.v1 - sh.v0 + 1, step = kSets * parts;
    const int first = s.worker - sh.v0 + set * parts;
    if (first >= c.m) continue;
    bool ok = true;
    if (lane == 0) ok = wait_count(arrivals_of(p, which, sh.v0), parts * (WARPS ? kRowWarps : 1), abort, p.err, (0x29 << 24) | which);
    __syncwarp();  // what lane 0 acquired, to all lanes: a shuffle orders no memory
    if (!__shfl_sync(kFull, ok, 0)) return false;
    constexpr int C = 2, B = 4;  // columns and parts on the way at a time
    for (int i0 = first; i0 < c.m; i0 += C * step) {
      float v[C][2] = {};
      for (int w0 = 0; w0 < parts; w0 += B) {
        float u[B][C][2];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int j = 0; j < C; ++j)
#pragma unroll
            for (int box = 0; box < 2; ++box) {
              const int i = i0 + j * step;
              u[b][j][box] = 0.f;
              if (w0 + b < parts && i < c.m)
                u[b][j][box] = __ldcg(part_of(p, sh.v0 + w0 + b, w0 + b == 0, box, row) + i * kTileRows);
            }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int j = 0; j < C; ++j)
#pragma unroll
            for (int box = 0; box < 2; ++box) v[j][box] += u[b][j][box];
      }
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (i0 + j * step < c.m) finish_column<KIND>(p, ss, s, c.r0, i0 + j * step, row, v[j][0], v[j][1]);
    }
  }
  return true;
}

// Every set sees all sums of its rows in tensor memory and takes its share of
// the m columns, two at a time.  `read(box, at, u)` starts the loads of one
// column, `value(u)` makes its sum of them, `done(i, v0, v1)` takes both boxes'.
template <int LOADS, typename Read, typename Value, typename Done>
__device__ __forceinline__ void each_column(int m, const Read& read, const Value& value, const Done& done) {
  const int set = threadIdx.x >> 7;
  constexpr int B = 2;
  for (int i0 = set * B; i0 < m; i0 += kSets * B) {
    uint32_t u[B][2][LOADS];
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int i = min(i0 + j, m - 1);  // past the end: the last column again
#pragma unroll
      for (int box = 0; box < 2; ++box) read(box, i, u[j][box]);
    }
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < B; ++j) {
      if (i0 + j >= m) break;
      done(i0 + j, value(u[j][0]), value(u[j][1]));
    }
  }
}

// A segment's sums are in tensor memory: finishes its tile, or leaves them as
// a part.
template <Kind KIND, int LOADS, typename Read, typename Value>
__device__ __forceinline__ void finish_segment(const StreamParams& p, const Shared& ss, const Segment& s, const Share& sh,
                                               const Columns<KIND>& c, const Read& read, const Value& value) {
  const int row = threadIdx.x & (kTileRows - 1);
  each_column<LOADS>(c.m, read, value, [&](int i, float v0, float v1) {
    if (sh.whole) {
      finish_column<KIND>(p, ss, s, c.r0, i, row, v0, v1);
    } else {
      __stcg(part_of(p, s.worker, s.kb0 == 0, 0, row) + i * kTileRows, v0);
      __stcg(part_of(p, s.worker, s.kb0 == 0, 1, row) + i * kTileRows, v1);
    }
  });
}

// bf16 weights: the accumulators hold the sums of a run of a segment's K blocks.
template <Kind KIND, bool RUNS>
__device__ bool rows_bf16(const StreamParams& p, int which, Shared& ss, Queue& qu, Turn& tn, volatile int* abort) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Tiles<false> walk(p, which, ss, qu, abort);
  Segment s;
  while (walk.next(s)) {
    const Columns<KIND> c(p, which, ss, s);
    const Share sh(walk.walk, s);
    constexpr int PARTS = KIND == kRowsOfH ? 3 : 1;
    const uint32_t lanes = ss.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16), sums = lanes + kTmemCols - kRunCols;
    for (int kb = s.kb0; kb < s.kb1; kb = RUNS ? kb + p.run : s.kb1) {
      if (!warp_wait<false>(&ss.acc_full[tn.buf], tn.phase, abort, p.err, (0x33 << 24) | which)) return false;
      tc_fence_after();
      const uint32_t acc = lanes + tn.buf * 2 * p.acc_cols;
      const auto read = [&](int box, int at, uint32_t* u) {
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          u[q] = 0;
          if (q < 2 || p.parts == 3) u[q] = tmem_ld1(acc + box * p.acc_cols + q * 16 * c.n16 + at);
        }
        if (RUNS) u[PARTS] = kb == s.kb0 ? 0 : tmem_ld1(sums + box * kMaxTokens + at);  // of the runs before
      };
      const auto value = [&](const uint32_t* u) {
        float v = __uint_as_float(u[0]);
        // An infinite weight: the sum of the upper parts of h is the infinity or NaN that h has; those of the lower
        // parts, which are 0 or of the other sign, would turn it into NaN.
        if constexpr (PARTS == 3) {
          if (isfinite(v)) v = fmaf(__uint_as_float(u[1]) + __uint_as_float(u[2]), 1.f / kLowScale, v);
        }
        return RUNS ? v + __uint_as_float(u[PARTS]) : v;
      };
      if (RUNS && kb + p.run < s.kb1) {
        each_column<PARTS + RUNS>(c.m, read, value, [&](int i, float v0, float v1) {
          tmem_st1(sums + i, __float_as_uint(v0));
          tmem_st1(sums + kMaxTokens + i, __float_as_uint(v1));
        });
        tmem_st_wait();
      } else {
        finish_segment<KIND, PARTS + RUNS>(p, ss, s, sh, c, read, value);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.acc_empty[tn.buf]);
      tn.step(p.acc_bufs);
    }
    if (!sh.whole) count_part<true>(p, which, sh);
  }
  return walk.through && join_parts<KIND, true>(p, which, ss, abort);
}

// 4-bit weights: two sets share a box, a thread one row of it.  A thread turns
// 64 of its row's codes into one of two buffers in tensor memory and hands it
// over, and adds, scaled, the sums of the groups that the push before ended.
// The tensor core's way from a push to its sums (600 clocks) is as long as a
// thread's from one push to the next.
template <int G, int N16, int PARTS, Kind KIND>
struct RowsQ4 {
  using Ge = Geo<G>;
  using Pu = Push<G, N16, PARTS>;
  static constexpr int NC = 16 * N16;
  // The parts of 16 rows of h lie N16 steps of 16 columns apart.
  static __device__ __forceinline__ void add_group(uint32_t acc, float scale, float (&sum)[NC]) {
#pragma unroll
    for (int b = 0; b < N16; ++b) {
      uint32_t u[16], lo[16];
      tmem_ld16(acc + b * 16, u);
      if constexpr (PARTS > 1) tmem_ld16(acc + (N16 + b) * 16, lo);
      tmem_ld_wait();
      if constexpr (PARTS > 2) {
        uint32_t lo2[16];
        tmem_ld16(acc + (2 * N16 + b) * 16, lo2);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) lo[i] = __float_as_uint(__uint_as_float(lo[i]) + __uint_as_float(lo2[i]));
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float v = __uint_as_float(u[i]);
        if constexpr (PARTS > 1) v = fmaf(__uint_as_float(lo[i]), 1.f / kLowScale, v);
        sum[b * 16 + i] = fmaf(scale, v, sum[b * 16 + i]);
      }
    }
  }

  static __device__ __forceinline__ bool segment(const StreamParams& p, int which, Shared& ss, uint8_t* ring,
                                                 const Walk& walk, const Segment& s, Ring& rg, Turn& tn, uint32_t& swap,
                                                 volatile int* abort) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quad = warp & 3, box = warp >> 3, set = (warp >> 2) & 1, row = quad * 32 + lane;
    const uint32_t lanes = ss.tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const Columns<KIND> c(p, which, ss, s);
    const Share sh(walk, s);
    const int K = p.p[which].K;
    // A row's chunks are swizzled; chunk numbers of different j and set differ in different bits.
    const uint32_t codes_at = box * kBoxBytes + row * 128 + (((set * Pu::SLAB) ^ (row & 7)) << 4);
    const uint32_t scales_at = 2 * kBoxBytes + box * Ge::SCALE_BYTES + row * 2 + set * (G == 32 ? Pu::SIZE : 1) * (kTileRows * 2);
    float sum[NC], scale[2] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i) sum[i] = 0.f;
    int before = -1;  // whether the last stage's last push had codes; -1: there was none
    // Adds what push j ended; `tn` is at its stage.
    auto take = [&](int j, uint32_t phase, int sums, bool some) {
      if (!warp_wait<true>(&ss.d_full[box][Pu::buf(j)], phase, abort, p.err, (0x34 << 24) | which)) return false;
      tc_fence_after();
      if (Pu::ends(j) && some) {
        const uint32_t at = sums_at(lanes, box, set, sums, Pu::SIZE);
        add_group(at, scale[0], sum);
        if (G == 32 && Pu::SIZE == 2) add_group(at + Pu::N, scale[1], sum);
      }
      return true;
    };
    for (int kb = s.kb0; kb < s.kb1; ++kb) {
      const uint32_t st = smem_u32(ring) + static_cast<uint32_t>(rg.stage) * p.stage_bytes;
      const uint32_t codes = st + codes_at, scales = st + scales_at;
      const int chunks = Pu::chunks(K, kb) - set * Pu::SLAB;
      if (!warp_wait<true>(&ss.full_w[rg.stage], rg.phase, abort, p.err, (0x23 << 24) | which)) return false;
#pragma unroll
      for (int j = 0; j < Pu::COUNT; ++j) {
        const bool some = Pu::first(j) < chunks;
        // The push's scales, long before they are needed: read after the codes were handed over, they cost 3%.
        float ahead[2] = {};
        if (Pu::ends(j) && some) {
          constexpr int step = kTileRows * 2;
          ahead[0] = lds_bf16(scales + (G == 32 ? Pu::first(j) : j / Pu::EACH * 2) * step);
          if (G == 32 && Pu::SIZE == 2) ahead[1] = lds_bf16(scales + (Pu::first(j) + 1) * step);
        }
        if (some) {
          const uint32_t operand = operand_at(lanes, box, set, Pu::buf(j));
#pragma unroll
          for (int i = 0; i < Pu::SIZE; ++i) {
            uint32_t w[4], v[16];
            lds128(codes ^ ((Pu::first(j) + i) << 4), w);
#pragma unroll
            for (int t = 0; t < 4; ++t) q4_pairs(w[t], *reinterpret_cast<uint32_t(*)[4]>(&v[4 * t]));
            tmem_st16(operand + i * (kChunk / 2), v);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.a_ready[box][Pu::buf(j)]);
        if (j > 0) {
          if (!take(j - 1, Pu::phase(tn, j - 1), Pu::sums(tn, j - 1), Pu::first(j - 1) < chunks)) return false;
        } else if (before >= 0) {
          if (!take(Pu::COUNT - 1, tn.phase ^ 1, Pu::COUNT == Pu::EACH ? tn.sums ^ 1 : 1, before)) return false;
        }
        if (Pu::ends(j)) scale[0] = ahead[0], scale[1] = ahead[1];
      }
      before = Pu::first(Pu::COUNT - 1) < chunks;
      Pu::stage_done(tn);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ss.empty[rg.stage]);
      rg.step(p.stages);
    }
    if (!take(Pu::COUNT - 1, tn.phase ^ 1, Pu::COUNT == Pu::EACH ? tn.sums ^ 1 : 1, before)) return false;
    // All sums of the tile meet in tensor memory, in the sets' operand
    // buffers: both boxes' and both turns'.  No set goes on before all have
    // read their share.
#pragma unroll
    for (int b = 0; b < NC / 16; ++b) {
      uint32_t u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(sum[b * 16 + i] * kQ4Unit);
      tmem_st16(operand_at(lanes, box, set, 0) + b * 16, u);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.swap_ready);
    if (!warp_wait<true>(&ss.swap_ready, swap, abort, p.err, (0x35 << 24) | which)) return false;
    tc_fence_after();
    finish_segment<KIND, 2>(
        p, ss, s, sh, c,
        [&](int bx, int at, uint32_t* u) {
          u[0] = tmem_ld1(operand_at(lanes, bx, 0, 0) + at);
          u[1] = tmem_ld1(operand_at(lanes, bx, 1, 0) + at);
        },
        [&](const uint32_t* u) { return __uint_as_float(u[0]) + __uint_as_float(u[1]); });
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ss.swap_done);
    if (!warp_wait<true>(&ss.swap_done, swap, abort, p.err, (0x36 << 24) | which)) return false;
    swap ^= 1;
    tc_fence_after();
    if (!sh.whole) count_part<false>(p, which, sh);  // swap_done: all row warps are here
    return true;
  }
};

template <Kind KIND, int G, int N16, int PARTS, typename... Args>
__device__ __forceinline__ bool rows_segment(Push<G, N16, PARTS>, Args&... args) {
  return RowsQ4<G, N16, PARTS, KIND>::segment(args...);
}

template <int G, Kind KIND>
__device__ bool rows_q4(const StreamParams& p, int which, Shared& ss, uint8_t* ring, Ring& rg, Queue& qu, Turn& tn, uint32_t& swap,
                        volatile int* abort) {
  Tiles<false> walk(p, which, ss, qu, abort);
  Segment s;
  bool ok = true;
  while (ok && walk.next(s))
    ok = with_push<G, KIND>(Columns<KIND>(p, which, ss, s).n16, p.parts, [&](auto push) {
      return rows_segment<KIND>(push, p, which, ss, ring, walk.walk, s, rg, tn, swap, abort);
    });
  return ok && walk.through && join_parts<KIND, false>(p, which, ss, abort);
}

// y[t] = its slots' rows in slot order, then the shared experts', in fp32.
__device__ void sum_rows(const StreamParams& p, const Shared& ss) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d4 = p.d / 4, R = p.T * p.k;
  const int units = p.T * d4, step = gridDim.x * kRowWarps * 32;
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

// RUNS: bf16 weights, fp32 y.
template <int G, bool LAYER, bool RUNS>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(const __grid_constant__ StreamParams p) {
  using Ge = Geo<G>;
  constexpr Kind FIRST = kGathered, SECOND = LAYER ? kRowsOfH : kRowsOfX;
  extern __shared__ uint8_t dyn[];
  Shared& ss = *reinterpret_cast<Shared*>(dyn);
  // stages on 1024-byte boundaries of shared memory (the swizzle's period)
  const uint32_t ring_at = (smem_u32(dyn) + kSharedBytes + 1023u) & ~1023u;
  uint8_t* ring = dyn + (ring_at - smem_u32(dyn));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // the same for the warp, and known to be
  if (warp == kWeightWarp) {
    if (lane < p.stages) {
      mbar_init(&ss.full_w[lane], 1);
      mbar_init(&ss.full_x[lane], 1);
      mbar_init(&ss.empty[lane], Ge::Q4 ? kRowWarps + 2 : 1);
    } else if (lane >= 16 && lane < 18) {
      const int i = lane & 1;
      for (int j = 0; j < 2; ++j) {
        mbar_init(&ss.a_ready[i][j], kRowWarps / 2);
        mbar_init(&ss.d_full[i][j], 1);
      }
      mbar_init(&ss.acc_full[i], 1);
      mbar_init(&ss.acc_empty[i], kRowWarps);
      mbar_init(&ss.rows_done[i], kRowWarps);
    } else if (lane >= 24 && lane < 24 + kTileSlots) {
      mbar_init(&ss.tile_full[lane - 24], 1);
      // readers: row warps, columns, one issuer (bf16) or two
      mbar_init(&ss.tile_empty[lane - 24], kRowWarps + 1 + (Ge::Q4 ? 2 : 1));
    } else if (lane == 20) {
      mbar_init(&ss.swap_ready, kRowWarps);
      mbar_init(&ss.swap_done, kRowWarps);
      mbar_init(&ss.out_done, 1);
      mbar_init(&ss.drained, 2);
      ss.abort = 0;
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ss.tmem, kTmemCols);
    tmem_relinquish();
  }
  if (LAYER) {
    build_work_list<Ge::Q4>(p, ss);
  } else if (tid == 0) {
    ss.nact = 1;
    ss.e[0] = ss.row0[0] = ss.blk0[1][0] = 0;
    ss.m[0] = p.T;
    ss.blk0[1][1] = ss.nblk[1] = (p.T + (1 << p.p[1].block_log2) - 1) >> p.p[1].block_log2;
    make_plan<Ge::Q4>(p, 1, ss);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  volatile int* abort = &ss.abort;
  if (warp == kWeightWarp) {
    Ring rg;
    Queue qu;
    Drain dr;
    bool ok = true;
    if (LAYER) ok = produce_weights<G, FIRST>(p, 0, ss, ring, rg, qu, dr, abort);
    if (ok) produce_weights<G, SECOND>(p, 1, ss, ring, rg, qu, dr, abort);
    dr.wait(ss.full_w);
  } else if (warp == kColumnWarp) {
    Ring rg;
    Queue qu;
    Drain dr;
    // This warp speaks for its CTA: it counts it in once the CTA's row warps
    // have left a product, and waits for the others.  (With one count and one
    // poller per warp the counter's L2 slice was so busy that the last
    // arrivals came through 8 us late.)
    auto meet = [&](int which) {
      bool ok = warp_wait<Ge::Q4>(&ss.rows_done[which], 0, abort, p.err, (0x25 << 24) | which);
      if (lane == 0) {
        // after a wait that gave up too, so that the other CTAs go on (the error word is set by then)
        if (blockIdx.x != 0 || p.drop != kDropMeeting + which) red_release_gpu_add(p.err + kCtrHidden + which, 1);
        ok = ok && wait_count(p.err + kCtrHidden + which, gridDim.x, abort, p.err, (0x26 << 24) | which);
      }
      __syncwarp();  // what lane 0 acquired, to the lane that issues the copies
      return __shfl_sync(kFull, ok, 0) != 0;
    };
    bool ok = true;
    if (LAYER) {
      ok = produce_columns<G, FIRST>(p, 0, ss, ring, rg, qu, dr, abort);
      const bool met = meet(0);    // every hidden value of every CTA,
      fence_proxy_async_global();  // for the bulk copies of this one
      ok = ok && met;
    }
    if (ok) ok = produce_columns<G, SECOND>(p, 1, ss, ring, rg, qu, dr, abort);
    if (LAYER && meet(1) && ok && lane == 0) mbar_arrive(&ss.out_done);
    dr.wait(ss.full_x);
  } else if (warp >= kMmaWarp) {
    Ring rg;
    Queue qu;
    Turn tn;
    bool ok = true;
    if constexpr (Ge::Q4) {
      const int box = warp - kMmaWarp;
      if (LAYER) ok = issue_q4<G, FIRST>(p, 0, box, ss, ring, rg, qu, tn, abort);
      if (ok) issue_q4<G, SECOND>(p, 1, box, ss, ring, rg, qu, tn, abort);
    } else if (warp == kMmaWarp) {
      if (LAYER) ok = issue_bf16<FIRST, RUNS>(p, 0, ss, ring, rg, qu, tn, abort);
      if (ok) issue_bf16<SECOND, RUNS>(p, 1, ss, ring, rg, qu, tn, abort);
    }
    __syncwarp();
    if (elect_one()) umma_commit(&ss.drained);
    __syncwarp();
    drain_wait(&ss.drained, 0);
  } else {
    Ring rg;
    Queue qu;
    Turn tn;
    [[maybe_unused]] uint32_t swap = 0;
    bool ok = true;
    if (LAYER) {
      auto through = [&](int which) {  // after a wait that gave up as well
        __syncwarp();
        if (lane == 0) mbar_arrive(&ss.rows_done[which]);
      };
      if constexpr (Ge::Q4)
        ok = rows_q4<G, FIRST>(p, 0, ss, ring, rg, qu, tn, swap, abort);
      else
        ok = rows_bf16<FIRST, RUNS>(p, 0, ss, qu, tn, abort);
      fence_proxy_async_global();  // hidden values, to other CTAs' copies
      through(0);
      if (ok) {
        if constexpr (Ge::Q4)
          ok = rows_q4<G, SECOND>(p, 1, ss, ring, rg, qu, tn, swap, abort);
        else
          ok = rows_bf16<SECOND, RUNS>(p, 1, ss, qu, tn, abort);
      }
      through(1);
      if (ok && warp_wait<Ge::Q4>(&ss.out_done, 0, abort, p.err, 0x2A << 24)) sum_rows(p, ss);
    } else {
      if constexpr (Ge::Q4)
        rows_q4<G, SECOND>(p, 1, ss, ring, rg, qu, tn, swap, abort);
      else
        rows_bf16<SECOND, RUNS>(p, 1, ss, qu, tn, abort);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(ss.tmem, kTmemCols);
  // the last CTA to pass its waits clears the counters
  if (tid == 0) ss.abort = atomicAdd(p.err + kCtrExit, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (ss.abort) {
    for (int i = tid; i < 2 * kMaxWorkers; i += kThreads) p.arrive[i] = 0;
    if (tid < kCtrEnd - kCtrHidden) p.err[kCtrHidden + tid] = 0;
  }
}

// -------------------------------------------------------------------- host
// Ranges the K blocks are cut into: one per SM of the device, whatever the
// grid, so that a capped grid gives the same bits.
int workers() { return std::min(num_sms(), kMaxWorkers); }

struct Layout {
  size_t part, arrive, h, o, total;
};
// Error region (with the counters), arrival counters, parts, hidden rows, output rows.
Layout layout(size_t rows, size_t d, size_t f) {
  Layout L{};
  size_t o = kErrRegionBytes;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.arrive = take(sizeof(int) * 2 * kMaxWorkers);
  L.part = take(sizeof(float) * kMaxWorkers * 4 * kMaxTokens * kTileRows);
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
  pr.row_step = which == 0 ? kTileRows : 2 * kTileRows;
  pr.row_tiles = ceil_div(rows, pr.row_step);
  auto box = [&](CUtensorMap* m, const DecodeWeight& w) {
    return Ge::Q4 ? map2d_any(m, w.w, 1, K / 2, mats * rows, 128, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B)
                  : map2d(m, w.w, K, mats * rows, 64, kTileRows);
  };
  bool ok = box(&pr.w0, w0);
  if (w1.w == w0.w)
    pr.w1 = pr.w0;
  else
    ok = ok && box(&pr.w1, w1);
  if constexpr (Ge::Q4) {
    auto sc = [&](CUtensorMap* m, const DecodeWeight& w) {
      return map2d_any(m, w.scales, 2, q4_scale_pitch(rows), mats * (K / G), kTileRows, Ge::GROUPS,
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

// Stages that fit beside the tables, and the launch's shared memory.  A stage
// has room for the widest tile: `cols` columns.
template <int G>
size_t ring_shape(StreamParams& p, int cols) {
  using Ge = Geo<G>;
  p.acc_cols = cols;
  const bool runs = !Ge::Q4 && p.y_type == MOE_Y_F32;
  p.acc_bufs = std::min(2, (kTmemCols - (runs ? kRunCols : 0)) / (2 * cols));
  p.run = p.acc_bufs == 2 ? kRunBlocks : kRunBlocksAlone;
  p.stage_bytes = static_cast<int>(align_up(Ge::WEIGHT_BYTES + Ge::ATOMS * cols * 128, 1024));
  const size_t fixed = kSharedBytes + 1024;
  p.stages = std::min<int>(kMaxStages, static_cast<int>((kSmemMax - fixed) / p.stage_bytes));
  return fixed + static_cast<size_t>(p.stages) * p.stage_bytes;
}

// Columns of a product's widest tile.
int columns_of(const StreamParams& p, int which, int parts) {
  return ceil_div(std::min(p.T, 1 << p.p[which].block_log2), 16) * 16 * parts;
}

template <int G, bool LAYER, bool RUNS>
int launch_kernel(StreamParams& p, size_t smem, int grid_limit, cudaStream_t s) {
  // The attribute holds for one device, and costs half a microsecond to set.
  static std::atomic<uint64_t> sized{0};  // a bit a device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (!(sized.load(std::memory_order_relaxed) & bit)) {
    if (cudaFuncSetAttribute(stream_kernel<G, LAYER, RUNS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return MOE_ERR_CUDA;
    sized.fetch_or(bit, std::memory_order_relaxed);
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
  return cudaLaunchKernelEx(&cfg, stream_kernel<G, LAYER, RUNS>, p) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
template <int G, bool LAYER>
int launch_stream(StreamParams& p, size_t smem, int grid_limit, cudaStream_t s) {
  if constexpr (G == 0)
    if (p.y_type == MOE_Y_F32) return launch_kernel<G, LAYER, true>(p, smem, grid_limit, s);
  return launch_kernel<G, LAYER, false>(p, smem, grid_limit, s);
}

void common_params(StreamParams& p, void* ws, const Layout& L, int T, void* y, int y_type) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.T = T;
  p.part = reinterpret_cast<float*>(at + L.part);
  p.arrive = reinterpret_cast<int*>(at + L.arrive);
  p.y = y;
  p.y_type = y_type;
  p.err = static_cast<int*>(ws);
  p.workers = workers();
  p.drop = g_drop;
}

template <int G>
int decode_g(const DecodeArgs& a, cudaStream_t s) {
  const moe_cfg& c = a.c;
  StreamParams p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t mats = c.E + c.n_shared;
  const uint64_t Rs = static_cast<uint64_t>(c.T) * (c.k + c.n_shared);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  const Layout L = layout(Rs, c.d_model, c.d_ff);
  common_params(p, a.ws, L, c.T, a.y, a.y_type);
  p.d = c.d_model, p.f = c.d_ff, p.E = c.E, p.k = c.k, p.S = c.n_shared, p.renorm = c.renorm;
  p.logits = a.logits, p.topk_idx = a.topk_idx, p.topk_w = a.topk_w;
  p.h = reinterpret_cast<uint16_t*>(ws + L.h);
  p.o = reinterpret_cast<float*>(ws + L.o);
  p.parts = a.y_type == MOE_Y_F32 ? 3 : 2;
  p.p[0].block_log2 = Geo<G>::block_log2(1);
  p.p[1].block_log2 = Geo<G>::block_log2(p.parts);
  if (!fill_product<G>(p.p[0], 0, a.W1, a.W3, mats, c.d_ff, c.d_model) ||
      !fill_product<G>(p.p[1], 1, a.W2, a.W2, mats, c.d_model, c.d_ff) ||
      !map2d(&p.p[0].cols, a.x, c.d_model, c.T, 64, 1) || !map2d(&p.p[1].cols, p.h, c.d_ff, p.parts * Rs, 64, 16))
    return MOE_ERR_CUDA;
  const size_t smem = ring_shape<G>(p, std::max(columns_of(p, 0, 1), columns_of(p, 1, p.parts)));
  TraceScope trace_scope(MOE_K_DECODE, s);
  return launch_stream<G, true>(p, smem, a.grid_limit, s);
}

template <int G>
int linear_g(const LinearArgs& a, cudaStream_t s) {
  StreamParams p;
  std::memset(&p, 0, sizeof(p));
  common_params(p, a.ws, layout(0, 0, 0), a.T, a.y, a.y_type);
  p.n = a.n;
  p.p[1].block_log2 = Geo<G>::block_log2(1);
  if (!fill_product<G>(p.p[1], 1, a.W, a.W, 1, a.n, a.K) || !map2d(&p.p[1].cols, a.x, a.K, a.T, 64, 16))
    return MOE_ERR_CUDA;
  const size_t smem = ring_shape<G>(p, columns_of(p, 1, 1));
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

extern "C" int moe_debug_drop_decode_count(int which) {
  if (which > moe::kDropMax) return MOE_ERR_ARG;
  moe::g_drop = which > 0 ? which : 0;
  return MOE_OK;
}
