// smla_tc_win.cu — causal MLA attention over a paged latent cache, whole or
// through a sliding window with first tokens that stay visible
// (smla_fwd_window), for bf16 rows and for E4M3 rows with one scale per cache
// block or per tensor.
//
// Mathematics.  The row (token at position p, head) sees the positions
//   V(p) = { e <= p : window == 0  or  e > p - window  or  e < sinks }
// whose block is allocated, s_e = sm_scale <q, K_e>, O = sum softmax(s)_e
// K_e[0:512], LSE = ln sum exp(s_e); no visible position gives (0, -inf).
// One pass over the keys with a running maximum (raised lazily: O is rescaled
// only when it grows by more than 2^8) and the running sum in fp32.
//
// Tile.  All heads share the key rows, and neighbouring tokens of a request
// share most of them, so a tile is 128 consecutive rows of the flattened
// (token, head) list of one request, whatever h is, and a block is 128 key
// positions.  O [128, 512] in fp32 fills one SM's TMEM by itself, so a tile
// runs on a pair of SMs as MMAs over both (cta_group::2) with M = 128: a CTA
// holds 64 rows, whose O takes 256 of its 512 TMEM columns and whose scores
// take 2 x 64.  The pair's MMAs run at the rate of two single-SM MMAs with
// M = 128 (measured: 36 QK and 16 PV steps of a block in 2210 cycles, 2176 at
// the peak rate); no partial score crosses between the SMs, in contrast to
// the sparse kernels' split over d_qk (smla_tc.cu), which can share one copy
// of a key row between QK and PV instead.
//   QK  S[128, 128] = Q . K^T      A = Q rows (64 per CTA, resident),
//                                  B = K rows: 64 of the 128 keys per CTA
//   PV  O[128, 256 n ..] += P . V  A = P rows (64 per CTA),
//                                  B = V^T: 128 of the 256 channels per CTA
//       for n = 0, 1
// A key's row is therefore read twice from L2 (as K by one CTA, as V by halves
// by both), once from HBM.
//
// Shared memory (bf16): Q 72 KB, K 72 KB, V 64 KB, P 16 KB.  K and V are one
// block deep, in rings of 3 channel groups and of 4 (channel half, key half)
// units; each part is refilled as soon as its MMAs are done, so the loads of
// block j + 1 run under the MMAs of block j.  E4M3: Q 80 KB (two terms), K 40 KB,
// V 32 KB, P 2 x 24 KB (three terms): the weights of block j + 1 are written while
// PV of block j runs (a second bf16 P in place of a V unit: 2 % slower).
//
// E4M3 rows.  Both products take the codes as they are (kind::f8f6f4, twice the
// bf16 rate for each pass).  QK: Q is the sum of two E4M3 terms after a
// power-of-two scale per row that puts its largest value in [224, 448); a bf16
// value has 8 significant bits and an E4M3 value 4, so hi = e4m3(q) and
// lo = e4m3(q - hi) give q exactly down to 2^-11 of the row's largest value
// (below, to 2^-19 of it).  The key's scale multiplies its scores in fp32.
// PV: a weight is the sum of three E5M2 terms.  E5M2 is the upper byte of f16 and
// holds 3 significant bits, so a weight rounded to 9 of f16's 11 bits is exactly
// its upper byte + that of the rest + that of what then remains (one bit more
// than bf16 keeps); the third is rounded to E5M2's grid, 2^-27 of the row's
// reference weight (keys 11 nats below the top still have their 9 bits, keys 16
// nats below are off by 3 %).  The key's scale belongs to its weight: with
// t = s + log2(scale) the running maximum is taken over t, the weights are
// 2^(t - m) = scale 2^(s - m), and the sum that divides adds weight / scale, in
// fp32 where the weights are too small for the product.  So blocks of any scales
// share one range, and nothing is converted on V's way to the tensor core.
//
// Masked positions.  A cache block of which a row of the tile sees some position
// is loaded whole: three columns of 64 rows arrive in 700 cycles as one copy, in
// 3400 as 48 gathers of four rows.  K needs no zeros: a masked score is replaced,
// its weight is 0.  V does, as 0 times NaN is NaN: rows behind the request's last
// token, which may never have been written, and blocks that are not allocated are
// read as zeros.  Any other masked position was written; should it hold an infinity
// or NaN, a row whose output is not finite although its softmax is is computed
// again from its visible positions alone (slow_rows).
//
// Scheduling.  A unit is a tile with some of its key blocks.  Many tiles: a unit
// is a tile; the grid has one cluster per tile, and a running cluster takes over
// tiles that have not started (clusterlaunchcontrol).  Few tiles: the blocks of
// all tiles, tile after tile, are cut into as many equal ranges as there are
// places for a pair; a cluster works on the tiles, or parts of tiles, in its
// range.  A part leaves a normalised fp32 partial and its LSE, and a second
// kernel merges a tile's parts in their order.  (Equal numbers of ranges per
// tile took 137 us for 32 E4M3 requests of 8 to 16 thousand keys with 128 heads,
// this 110 us.)
// Either way a cluster keeps its barriers, TMEM and loaders going, so the next
// unit's first loads and QK run under the epilogue of the last one.
//
// Warp roles: warp 0 issues QK and owns TMEM, another warp issues PV (both in
// the even CTA; two issuers, so that the waits of one are covered by the MMAs of
// the other); warps 1 and 2 load K and V; warp 3 takes units and looks up
// each block's rows (validity, scales, row ids); warps 4..11 are the softmax: four
// threads per row (TMEM lane half x column half), 32 keys each; with E4M3 rows
// warps 13..15 split Q.
// Every wait is bounded, as in the sparse kernels (tc_common.cuh).
//
// Bound and measured.  A block is 2,176 cycles of MMAs (E4M3, five passes at twice
// the rate: 2,688) and takes about 3,000: bf16 loads run at 12 TB/s from L2, K
// and V apart, through rings one block deep, all that shared memory holds.  A unit
// costs about 5 us more (lookups, first copies, epilogue).  In a captured graph: a
// prompt of 4096 tokens with 128 heads through a window of 2048, bf16, 1.19 to 1.25 ms
// in short bursts, 1.31 ms = 1.34 PFLOP/s where the power limit holds the clocks
// down; 2048 tokens with 64 heads behind 6000, E4M3, 1.28 to 1.35 and 1.40 ms = 1.29
// PFLOP/s; 64 decode tokens with 128 heads through the window, bf16, 45 us = 3.8
// TB/s; 32 of 8 to 16 thousand keys, E4M3, 107 to 110 us = 0.97 PFLOP/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "e4m3_quant.cuh"
#include "paged_batch.cuh"
#include "smla_paged.h"
#include "tc_common.cuh"
#include "tc_pair.cuh"

namespace smla {
namespace {

using namespace ptx;

constexpr int kBN = 128;                   // key positions per block
constexpr int kRows = 64;                  // tile rows per CTA
constexpr uint32_t kAtom = 8192;           // 64 rows x 128 bytes
constexpr int kKGroups = 3;                // K ring: channel groups
constexpr int kVUnits = 4;                 // V of a block: (channel half n, key half)
constexpr int kMeta = 3;                   // blocks of lookups in flight

// TMEM columns.
constexpr uint32_t kColO = 0;              // 2 x 128
constexpr uint32_t kColS = 256;            // 2 x 64
constexpr uint32_t kTmemCols = 512;

enum {
  kBarKFull = 0,                           // [3] even CTA: both CTAs' bytes
  kBarKEmpty = kBarKFull + kKGroups,       // [3] both
  kBarVFull = kBarKEmpty + kKGroups,       // [4] even CTA (a slot each)
  kBarVEmpty = kBarVFull + kVUnits,        // [4] both
  kBarSFull = kBarVEmpty + kVUnits,        // [2] both
  kBarSEmpty = kBarSFull + 2,              // [2] even CTA: 16 warps
  kBarPFull = kBarSEmpty + 2,              // [2] even CTA: 16 warps
  kBarPEmpty = kBarPFull + 2,              // [2] both
  kBarQFull = kBarPEmpty + 2,              // even CTA
  kBarQEmpty,                              // both
  kBarMFull,                               // [3] own
  kBarMEmpty = kBarMFull + kMeta,          // [3] own
  kBarTFull = kBarMEmpty + kMeta,          // [2] own: a unit's description
  kBarTEmpty = kBarTFull + 2,              // [2] own
  kBarCFull = kBarTEmpty + 2,              // [2] own: an answer of the launch control
  kBarCEmpty = kBarCFull + 2,              // [2] even CTA: both have read it
  kBarDrain = kBarCEmpty + 2,              // [2] even CTA: QK's and PV's last MMAs
  kBarQScale = kBarDrain + 2,              // own, E4M3: the Q rows' scales are written
  kNumBars
};

// The bounded waits of tc_common.cuh with everything but the first try out of
// line: the roles' loops then stay small, and they have to share one
// instruction cache (waits in line cost this kernel 1.2x).
struct PairWaiter {
  uint32_t flags;                          // shared address: abort flag, abort counter at
                                           // the start, beat
  const WinParams* p;
  __device__ __forceinline__ volatile int* shared(int i) const {
    return static_cast<volatile int*>(__cvta_shared_to_generic(flags)) + i;
  }
  __device__ __forceinline__ bool aborted() const {
    int v;
    asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(flags) : "memory");
    return v != 0;
  }
  // false: gave up (the block is aborting).  A lane whose wait came true need not
  // look at the flag.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const;
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const;
};

// A wait that runs out gives up, unless a CTA of the pair has been computing rows
// again meanwhile (slow_rows), which may take longer than any limit and says so by
// its beat.
static __device__ __noinline__ void pair_wait_slow(uint32_t bar, uint32_t parity, uint32_t flags,
                                                   const WinParams* p, bool drain) {
  const PairWaiter w{flags, p};
  Waiter slow{w.shared(0), p->status, p->abort_ctr, *w.shared(1), p->wait_limit_ns};
  if (!drain && *slow.abort) return;
  const volatile int* stop = drain ? nullptr : slow.ctr;
  int beat;
  do {
    beat = *w.shared(2);
    if (mbar_wait_bounded<false>(bar, parity, slow.limit_ns, stop, slow.ctr0)) return;
  } while (*w.shared(2) != beat && !(stop && *stop != slow.ctr0));
  slow.fail();
}
__device__ __forceinline__ bool PairWaiter::wait(uint32_t bar, uint32_t parity) const {
  if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
  pair_wait_slow(bar, parity, flags, p, false);
  return !aborted();
}
__device__ __forceinline__ void PairWaiter::drain(uint32_t bar, uint32_t parity) const {
  pair_wait_slow(bar, parity, flags, p, true);
}

// A unit as its warps need it: rows [row0, row1) of the flattened (token, head)
// list, of request r, whose last token has position p_last; positions
// [lo, p_last] and [0, sinks) are seen by some row; its key blocks are numbers
// [b0, b0 + nb) of the tile's list (block()).
struct Unit {
  int row0, row1, p_last, r;
  int lo, sinks, sink_blocks, win_block;
  int b0, nb;
  int slot;                                // of its partial; -1: the tile's only part
  int live;                                // 1 + the request's length; 0: no more units
  __device__ __forceinline__ int block(int i) const {   // i-th block's index
    return i < sink_blocks ? i : win_block + (i - sink_blocks);
  }
  // The j-th block in the order of work.  bf16: from the last, so that the slow
  // copies of the block that a request ends in come while nothing else does (a
  // prompt of 4096 tokens: 1.30 -> 1.23 ms, 64 decode tokens: 53 -> 50 us).  E4M3:
  // from the first (from the last, 32 decode tokens took 116 us, not 114).
  template <bool kFp8>
  __device__ __forceinline__ int work(int j) const {
    return block(kFp8 ? b0 + j : b0 + nb - 1 - j);
  }
};
static_assert(sizeof(Unit) == 48, "three 16-byte words");

constexpr int kWarpPv = 12;                // issues PV

template <bool kFp8>
struct Cfg {
  static constexpr int kThreads = kFp8 ? 512 : 416;
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kAtomsPerGroup = kFp8 ? 2 : 3;
  static constexpr int kMaxAtoms = kFp8 ? 5 : 9;        // 128-byte columns of a row
  // O is rescaled where a row's maximum grows by more than 2^kRaise.  E4M3 rows' weights
  // are multiplied by 1 / kBack, so that they end at 2^15, within E5M2's range: 2^4 and
  // not 2^8 leaves them four more bits below (32 decode tokens: 102.9 -> 104.5 us).
  static constexpr float kRaise = kFp8 ? 4.f : 8.f;
  static constexpr float kBack = kFp8 ? 0x1p-11f : 1.f;
  static constexpr int kPBufs = kFp8 ? 2 : 1;
  static constexpr int kQTerms = kFp8 ? 2 : 1;
  static constexpr int kPTerms = kFp8 ? 3 : 1;
  static constexpr uint32_t kVUnit = kFp8 ? kAtom : 2 * kAtom;     // 64 keys x 128 channels
  static constexpr uint32_t kPTerm = kFp8 ? kAtom : 2 * kAtom;     // 64 rows x 128 keys
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffK = kOffQ + kQTerms * kMaxAtoms * kAtom;
  static constexpr uint32_t kOffV = kOffK + kMaxAtoms * kAtom;
  static constexpr uint32_t kOffP = kOffV + kVUnits * kVUnit;
  // row maxima, fp32 [4][64]: one buffer for bf16 rows (the room that is left), else two
  static constexpr uint32_t kOffRed = kOffP + kPBufs * kPTerms * kPTerm;
  static constexpr uint32_t kOffBar = kOffRed + (kFp8 ? 2048 : 1024);
  static constexpr uint32_t kOffMask = kOffBar + 8 * (((kFp8 ? kNumBars : kBarQScale) + 1) & ~1);
                                                                      // u32 [kMeta][4]
  static constexpr uint32_t kOffUnit = kOffMask + kMeta * 16;         // Unit [2]
  static constexpr uint32_t kOffAnswer = kOffUnit + 2 * 48;           // 16 bytes [2]
  static constexpr uint32_t kOffIds = kOffAnswer + 32;                // i32 [kMeta][128] rows
  static constexpr uint32_t kOffTmem = kOffIds + kMeta * kBN * 4;
  static constexpr uint32_t kOffAbort = kOffTmem + 4;
  // E4M3: the keys' scales, each 32 keys' common scale (0: several), its log2
  // and its reciprocal, the Q rows' scales (two units')
  static constexpr uint32_t kOffScale = kFp8 ? (kOffAbort + 12 + 15) & ~15u : kOffAbort + 12;
  static constexpr uint32_t kOffSeg = kOffScale + (kFp8 ? kMeta * kBN * 4 : 0); // float4 [kMeta][4]
  static constexpr uint32_t kOffQScale = kOffSeg + (kFp8 ? kMeta * 64 : 0);
  static constexpr uint32_t kSmem = kOffQScale + (kFp8 ? 2 * kRows * 4 : 0);
  static_assert(kSmem <= 232448, "shared memory budget");
};
// The epilogue's areas in P: row sums and flags.
constexpr uint32_t kOffSums = 4096;        // float [2][4][64]
constexpr uint32_t kOffFlag = 4096 + 2048; // int [64]
// slow_rows': maxima and sums of eight warps, four rows of O
constexpr uint32_t kOffWarpSums = 0;       // float2 [8]
constexpr uint32_t kOffRows = 8192;        // float [4][512]

struct WinArgs {
  CUtensorMap row_map;   // the cache, boxes of one row x 128 bytes (gather4)
  CUtensorMap box_map;   // the cache, boxes of `box` rows x 128 bytes
  CUtensorMap k_map;     // the cache as (128-byte column, row, column index): boxes of 64 rows
  CUtensorMap v_map;     // x one K group's columns, and x two columns (bf16, whole boxes)
  CUtensorMap q_map;     // bf16 q [T * h, d_qk], boxes of 64 rows x 64 channels
  WinParams p;
  int box;               // rows per box, a power of two in 4..64; 0: gather4 alone
  int quad;              // blocks are multiples of 4 rows: 4 positions share one
  int shift;             // log2 of the block size, -1 if it is no power of two
  int wide;              // out is 32-byte aligned
  int atoms;             // 128-byte columns of a row
  int ksteps;            // 32-byte MMA steps of a row
  float scale_log2;      // sm_scale * log2(e)
};

// The tiles of a request are numbered from first_tile on.  h = 128: a tile is
// a token.  Otherwise n tokens make ceil(n h / 128) <= floor((c + n) h / 128)
// - floor(c h / 128) + 1 tiles, so floor(start h / 128) + r keeps the requests'
// numbers apart, and T h / 128 + R of them hold every tile.
__device__ __forceinline__ int64_t first_tile(const WinParams& p, int r) {
  const int64_t c = batch_start(p.b, r);
  return p.h == 128 ? c : c * p.h / 128 + r;
}

// The k-th tile of request r, whose tokens are [c0, c1) and whose length is len,
// with all of its key blocks; row1 = row0 where there is no such tile.
__device__ __forceinline__ Unit tile_unit(const WinParams& p, int r, int c0, int c1, int len,
                                          int64_t k) {
  Unit t;
  t.r = r;
  t.slot = -1;
  const int64_t r0 = (int64_t)c0 * p.h + 128 * k, r1 = min(r0 + 128, (int64_t)c1 * p.h);
  const bool used = k >= 0 && r1 > r0;
  t.row0 = used ? (int)r0 : 0;
  t.row1 = used ? (int)r1 : 0;
  t.b0 = t.nb = t.sink_blocks = t.win_block = 0;
  t.p_last = t.lo = -1;
  t.sinks = 0;
  t.live = 1 + min(len, 0x7FFFFFFE);
  if (!used) return t;
  const int tok0 = t.row0 / p.h, tok1 = (t.row1 - 1) / p.h;
  t.p_last = len - (c1 - tok1);
  if (t.p_last < 0) return t;
  const int p_first = max(len - (c1 - tok0), 0);
  t.lo = p.window ? max(p_first - (p.window - 1), 0) : 0;
  t.sinks = min(p.sinks, t.lo);
  t.win_block = t.lo / kBN;
  // (blocks past the table hold nothing, whatever a length says)
  const int end = min(t.p_last, p.table_end) / kBN + 1;
  t.sink_blocks = min(min((t.sinks + kBN - 1) / kBN, t.win_block), end);
  t.nb = t.sink_blocks + max(end - t.win_block, 0);
  return t;
}

// Unit number u where a unit is a tile: the tiles from the last, as a prompt's
// later tokens see more keys.
__device__ __forceinline__ Unit find_unit(const WinParams& p, int64_t u) {
  const int64_t tile = p.num_tiles - 1 - u;
  const int r = warp_last_request(p.b.num_reqs, tile, [&](int m) { return first_tile(p, m); });
  return tile_unit(p, r, batch_start(p.b, r), batch_start(p.b, r + 1), batch_len(p.b, r),
                   tile - first_tile(p, r));
}

// A cluster's range of the list of all tiles' blocks (a tile without one counts
// one), where it stands, and the request that it stands in.  Beginning a second
// tile costs a range about as much as 5 blocks (its Q, its first loads, another
// epilogue: 7 us with bf16 rows, 12 with E4M3), so every tile but the list's
// first counts that much more, before its blocks.
constexpr int kTileCost = 5;
struct Walk {
  int64_t pos, end, total;
  int64_t base;                            // the request's first block in the list
  int r;
  int ranges;                              // no more than there are blocks: none is empty
};
__device__ __forceinline__ int request_tiles(const WinParams& p, int c0, int c1) {
  return c1 > c0 ? (int)(((int64_t)(c1 - c0) * p.h + 127) / 128) : 0;
}
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
// x / y for x >= 0 and y > 0, in 32 bits where they hold it.
static __device__ __noinline__ int64_t divide_wide(int64_t x, int64_t y) { return x / y; }
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
  if (x < 0x7FFFFFFF && y < 0x7FFFFFFF) return (uint32_t)x / (uint32_t)y;
  return divide_wide(x, y);
}
// The w-th range.  First the list's length, then the range's place.
__device__ __forceinline__ Walk start_walk(const WinParams& p, int w) {
  const int lane = threadIdx.x & 31;
  Walk k{0, 0, 0, 0, 0, 0};
  int64_t n = 0, upto = 0, all = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int64_t acc = 0;
#pragma unroll 1
    for (int first = 0; first < p.b.num_reqs; first += 32) {
      if (pass == 0 || p.b.num_reqs > 32) {
        const int r = min(first + lane, p.b.num_reqs - 1);
        const int c0 = batch_start(p.b, r), c1 = batch_start(p.b, r + 1);
        const int len = batch_len(p.b, r);
        const int tiles = first + lane < p.b.num_reqs ? request_tiles(p, c0, c1) : 0;
        // One tile: its lane counts it.  More: the warp counts the request together.
        n = tiles == 1 ? kTileCost + max(tile_unit(p, r, c0, c1, len, 0).nb, 1) : 0;
        for (uint32_t many = __ballot_sync(0xffffffffu, tiles > 1); many; many &= many - 1) {
          const int src = __ffs(many) - 1;
          const int s0 = __shfl_sync(0xffffffffu, c0, src), s1 = __shfl_sync(0xffffffffu, c1, src);
          const int sl = __shfl_sync(0xffffffffu, len, src);
          const int st = __shfl_sync(0xffffffffu, tiles, src);
          int64_t sum = 0;
#pragma unroll 1
          for (int t = lane; t < st; t += 32)
            sum += kTileCost + max(tile_unit(p, 0, s0, s1, sl, t).nb, 1);
          sum = __shfl_sync(0xffffffffu, warp_scan(sum), 31);
          if (lane == src) n = sum;
        }
        upto = warp_scan(n);
        all = __shfl_sync(0xffffffffu, upto, 31);
      }
      if (pass == 1 && k.pos < acc + all) {
        const int src = __ffs(__ballot_sync(0xffffffffu, k.pos < acc + upto)) - 1;
        k.r = first + src;
        k.base = acc + __shfl_sync(0xffffffffu, upto - n, src);
        return k;
      }
      acc += all;
    }
    if (pass == 0) {
      k.total = acc - kTileCost;
      k.ranges = (int)min((int64_t)p.workers, k.total);
      if (w >= k.ranges) return k;
      k.pos = kTileCost + divide(k.total * w, k.ranges);
      k.end = kTileCost + divide(k.total * (w + 1), k.ranges);
    }
  }
  return k;
}
// The next part of a tile in the range; its row1 = row0 behind the last.  `note`:
// this CTA writes down which ranges hold the tile, for the merge.
__device__ __forceinline__ Unit next_part(const WinParams& p, Walk& k, int w, bool note) {
  const int lane = threadIdx.x & 31;
  Unit u{};
#pragma unroll 1
  while (k.pos < k.end && k.r < p.b.num_reqs) {
    const int c0 = batch_start(p.b, k.r), c1 = batch_start(p.b, k.r + 1);
    const int len = batch_len(p.b, k.r);
    const int tiles = request_tiles(p, c0, c1);
    // The request's tile that holds the place: number t, its blocks from t0 on.
    int t = 0;
    int64_t t0 = k.base;
#pragma unroll 1
    for (; tiles > 1 && t < tiles; t += 32) {
      const int64_t n =
          t + lane < tiles ? kTileCost + max(tile_unit(p, k.r, c0, c1, len, t + lane).nb, 1) : 0;
      const int64_t upto = warp_scan(n), all = __shfl_sync(0xffffffffu, upto, 31);
      if (k.pos < t0 + all) {
        const int src = __ffs(__ballot_sync(0xffffffffu, k.pos < t0 + upto)) - 1;
        t0 += __shfl_sync(0xffffffffu, upto - n, src);
        t += src;
        break;
      }
      t0 += all;
    }
    if (t < tiles) {
      u = tile_unit(p, k.r, c0, c1, len, t);
      const int blocks = max(u.nb, 1);
      t0 += kTileCost;                                 // its first block
      if (k.pos < t0 + blocks) {
        u.b0 = (int)max(k.pos - t0, (int64_t)0);
        const int take = (int)(min(t0 + blocks, k.end) - t0) - u.b0;
        if (take <= 0) return Unit{};                  // (the range ends before it)
        // (a range ends in at most one tile that goes on and begins in at most one
        // that went before: two partials)
        u.slot = take == blocks ? -1 : 2 * w + (u.b0 + take < blocks ? 1 : 0);
        if (u.nb > 0) u.nb = take;
        if (note && u.b0 == 0) {
          const int64_t upto = t0 + blocks - kTileCost;
          const int last = (int)divide(upto * k.ranges - 1, k.total);
          for (int g = u.row0 + lane; g < u.row1; g += 32)
            p.parts[g] = w << 19 | last << 7 | (g - u.row0);
        }
        k.pos = t0 + u.b0 + take;
        return u;
      }
      t0 += blocks;                                    // (the request's only tile: done)
    }
    k.base = t0;
    ++k.r;
    u = Unit{};
  }
  return u;
}

// Cache rows of the four positions pos .. pos + 3 (pos a multiple of 4), -1
// where no row of the tile sees the position or it has no row.
struct Rows4 {
  int id[4];
  int blk[4];
};
static __device__ __noinline__ Rows4 lookup4(const WinParams& p, const Unit& t, int pos,
                                             bool& bad) {
  Rows4 o;
  int page = -1, blk = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = pos + i;
    const bool seen = e <= t.p_last && (e >= t.lo || e < t.sinks);
    o.id[i] = -1;
    o.blk[i] = -1;
    if (seen) {
      const int pg = e / p.b.block_size;
      if (pg != page) {
        page = pg;
        blk = batch_block(p.b, t.r, pg, bad);
      }
      o.id[i] = batch_row(p.b, blk, e - pg * p.b.block_size, bad);
      if (o.id[i] >= 0) o.blk[i] = blk;
    }
  }
  return o;
}

// Slot and phase of the lookups' ring, advanced block by block.
struct MetaRing {
  int m = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++m == kMeta) {
      m = 0;
      ph ^= 1;
    }
  }
};

// A cache block's scale.  The weights need its logarithm: below 2^-64, the least that
// the append writes, it counts as that (zero too: values of at most 2^-55, scores
// next to 0), and a negative one is NaN.
__device__ __forceinline__ float block_scale(const WinParams& p, int blk) {
  const float x = ld_batch(p.k_scale + blk);
  return x < 0x1p-64f ? (x < 0.f ? NAN : 0x1p-64f) : x;
}
// A key's scale (E4M3 caches).
__device__ __forceinline__ float key_scale(const WinParams& p, int blk) {
  return p.kv_format == kE4m3Block ? block_scale(p, blk) : ld_batch(p.k_scale);
}

// 16 bytes of q, in order behind what was waited for (ld_batch).
__device__ __forceinline__ uint4 ld_q16(const uint4* at) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(at));
  return v;
}

// The unit's marked rows again, each from its visible positions in the unit's blocks
// alone, by the eight softmax warps together: each warp takes 16 keys of every block,
// two at a time, and the eight partial rows are merged in P's place.  A lane holds
// twice eight neighbouring channels of a row's 512, and two of its rope.  131,072 keys
// take 8 ms a row; meanwhile the pair's other warps wait (pair_wait_slow), for which a
// beat goes to both CTAs.
template <bool kFp8>
static __device__ __noinline__ void slow_rows(const WinParams& p, const Unit& t, uint8_t* sp,
                                              const PairWaiter w, uint32_t rank) {
  constexpr int kKeys = 2;
  const int lane = threadIdx.x & 31, sw = (threadIdx.x >> 5) - 4;
  const bool rope = p.d_qk > 512;
  // the lane's channels: ch .. + 7, ch + far .. + 7 (in one 16-byte load, or two)
  constexpr int kFar = kFp8 ? 8 : 256;
  const int ch = kFp8 ? 16 * lane : 8 * lane;
  const int* flag = reinterpret_cast<const int*>(sp + kOffFlag);
  float2* ml = reinterpret_cast<float2*>(sp + kOffWarpSums);
  float* part = reinterpret_cast<float*>(sp + kOffRows) + 512 * (sw & 3) + ch;
  const uint32_t beat = w.flags + 8, far_beat = mapa(beat, rank ^ 1u);
#pragma unroll 1
  for (int rr = 0; rr < kRows; ++rr) {
    if (!flag[rr]) continue;
    const int64_t g = (int64_t)t.row0 + 64 * (int)rank + rr;
    const int pos = t.p_last - ((t.row1 - 1) / p.h - (int)g / p.h);
    const int lo = p.window ? max(pos - (p.window - 1), 0) : 0;
    const uint16_t* qr = static_cast<const uint16_t*>(p.q) + g * p.d_qk;
    const uint4 q0 = *reinterpret_cast<const uint4*>(qr + ch);
    const uint4 q1 = *reinterpret_cast<const uint4*>(qr + ch + kFar);
    const uint32_t q[9] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w,
                           rope ? reinterpret_cast<const uint32_t*>(qr + 512)[lane] : 0u};
    float acc[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool bad = false;                                  // (the lookups have said so)
#pragma unroll 1
    for (int b = t.b0; b < t.b0 + t.nb; ++b) {
      const int e = t.block(b) * kBN + 16 * sw + (lane & 15);
      if (lane == 0) {
        const int now = (int)globaltimer_ns();
        *w.shared(2) = now;
        st_cluster_s32(far_beat, now);
      }
      if (__any_sync(0xffffffffu, w.aborted())) break;
      int row = -1;
      float scale = 1.f;
      if (e <= pos && (e >= lo || e < p.sinks)) {
        const int page = e / p.b.block_size;
        const int blk = batch_block(p.b, t.r, page, bad);
        row = batch_row(p.b, blk, e - page * p.b.block_size, bad);
        if (kFp8 && row >= 0) scale = key_scale(p, blk);
      }
      uint32_t todo = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
#pragma unroll 1
      while (todo) {
        uint32_t k[kKeys][kFp8 ? 5 : 9];               // (a row's last word: its rope)
        float s[kKeys], sc[kKeys];
        bool have[kKeys];
        int src = 0;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {              // (past the last: that key once more)
          have[c] = todo != 0;
          if (todo) src = __ffs(todo) - 1;
          todo &= todo - 1;
          const int64_t at = (int64_t)__shfl_sync(0xffffffffu, row, src) * p.d_qk;
          sc[c] = __shfl_sync(0xffffffffu, scale, src);
          if (kFp8) {
            const uint8_t* kr = static_cast<const uint8_t*>(p.kv) + at;
            const uint4 x = *reinterpret_cast<const uint4*>(kr + ch);
            k[c][0] = x.x; k[c][1] = x.y; k[c][2] = x.z; k[c][3] = x.w;
            k[c][4] = rope ? reinterpret_cast<const uint16_t*>(kr + 512)[lane] : 0u;
          } else {
            const uint16_t* kr = static_cast<const uint16_t*>(p.kv) + at;
            const uint4 x = *reinterpret_cast<const uint4*>(kr + ch);
            const uint4 y = *reinterpret_cast<const uint4*>(kr + ch + kFar);
            k[c][0] = x.x; k[c][1] = x.y; k[c][2] = x.z; k[c][3] = x.w;
            k[c][kFp8 ? 0 : 4] = y.x; k[c][kFp8 ? 0 : 5] = y.y;
            k[c][kFp8 ? 0 : 6] = y.z; k[c][kFp8 ? 0 : 7] = y.w;
            k[c][kFp8 ? 0 : 8] =
                rope ? reinterpret_cast<const uint32_t*>(kr + 512)[lane] : 0u;
          }
        }
        // The i-th pair of the lane's channels (8: the rope's).
        auto key = [&](int c, int i, float& x, float& y) {
          if (kFp8) {
            float z, u;
            e4m3x4_to_f32(i == 8 ? k[c][4] : k[c][i / 2] >> (16 * (i & 1)), x, y, z, u);
          } else {
            x = __uint_as_float(k[c][kFp8 ? 0 : i] << 16);
            y = __uint_as_float(k[c][kFp8 ? 0 : i] & 0xFFFF0000u);
          }
        };
        float top = m;
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {
          float s1 = 0.f;
          s[c] = 0.f;
#pragma unroll
          for (int i = 0; i < 9; ++i) {
            float x, y;
            key(c, i, x, y);
            s[c] = fmaf(__uint_as_float(q[i] << 16), x, s[c]);
            s1 = fmaf(__uint_as_float(q[i] & 0xFFFF0000u), y, s1);
          }
          s[c] += s1;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
          for (int c = 0; c < kKeys; ++c) s[c] += __shfl_xor_sync(0xffffffffu, s[c], o);
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {
          s[c] = have[c] ? s[c] * sc[c] * p.sm_scale : -INFINITY;
          top = fmaxf(top, s[c]);
        }
        if (top > m) {
          const float a = expf(m - top);
          l *= a;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc[i][0] *= a;
            acc[i][1] *= a;
          }
          m = top;
        }
#pragma unroll
        for (int c = 0; c < kKeys; ++c) {
          if (!have[c]) continue;
          const float e2 = s[c] == -INFINITY ? 0.f : expf(s[c] - m);
          l += e2;
          const float wt = e2 * sc[c];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float x, y;
            key(c, i, x, y);
            acc[i][0] = fmaf(wt, x, acc[i][0]);
            acc[i][1] = fmaf(wt, y, acc[i][1]);
          }
        }
      }
    }
    // The eight warps' rows: the upper four's, then with the lower four's, then in one.
    if (lane == 0) ml[sw] = make_float2(m, l);
    named_bar_sync(4, 256);
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += ml[i].x == -INFINITY ? 0.f : ml[i].y * expf(ml[i].x - top);
    // (a warp without a key: its sums are 0, or NaN where 0 met an infinity)
    const float f = (m == -INFINITY ? 1.f : expf(m - top)) / sum;
    auto at = [&](int i) {
      return reinterpret_cast<float2*>(part + (i & 4 ? kFar - 8 : 0) + 2 * i);
    };
    if (sw >= 4)
#pragma unroll
      for (int i = 0; i < 8; ++i) *at(i) = make_float2(acc[i][0] * f, acc[i][1] * f);
    named_bar_sync(4, 256);
    if (sw < 4)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 o = *at(i);
        *at(i) = make_float2(fmaf(acc[i][0], f, o.x), fmaf(acc[i][1], f, o.y));
      }
    named_bar_sync(4, 256);
    const int c = threadIdx.x - 128;                   // two channels a thread
    const float2* o = reinterpret_cast<const float2*>(sp + kOffRows) + c;
    const float x = (o[0].x + o[256].x) + (o[512].x + o[768].x);
    const float y = (o[0].y + o[256].y) + (o[512].y + o[768].y);
    if (t.slot >= 0)
      reinterpret_cast<float2*>(p.o_part +
                                ((int64_t)t.slot * 128 + 64 * (int)rank + rr) * 512)[c] =
          make_float2(x, y);
    else
      reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + g * 512)[c] =
          pack_bf16(x, y);
    named_bar_sync(4, 256);                            // (the next row's sums take their place)
  }
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<kFp8>::kThreads, 1)
smla_window_kernel(const __grid_constant__ WinArgs a) {
  using C = Cfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const WinParams& p = a.p;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t r = cluster_ctarank();

  auto bar = [&](int i) { return sb + C::kOffBar + 8u * (uint32_t)i; };
  const PairWaiter W{sb + C::kOffAbort, &p};

  // Setup, spread over the warps: barriers, TMEM, the abort flag and the tensor
  // maps; the lookups' warp meanwhile finds the first unit and its table entries.
  // The launch may come under the end of the kernel before (launch_early): nothing
  // that it could have written is read before griddepcontrol.wait, which the two
  // warps that read first execute, and the others pass the barrier behind them.
  if (tid == 32) {
    for (int i = 0; i < kKGroups; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < kVUnits; ++i) {
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSEmpty + i), 16);
      mbar_init(bar(kBarPFull + i), 16);
      mbar_init(bar(kBarPEmpty + i), 1);
    }
    mbar_init(bar(kBarQFull), kFp8 ? 6 : 1);         // E4M3: three warps of both CTAs write Q
    if (kFp8) mbar_init(bar(kBarQScale), 3);
    for (int i = 0; i < kMeta; ++i) {
      mbar_init(bar(kBarMFull + i), 1);
      mbar_init(bar(kBarMEmpty + i), 10);              // softmax, loaders
    }
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarTFull + i), 1);
      // those, the even CTA's issuers, E4M3: the warps that split Q
      mbar_init(bar(kBarTEmpty + i), 10 + (r == 0 ? 2 : 0) + (kFp8 ? 3 : 0));
      mbar_init(bar(kBarCFull + i), 1);
      mbar_init(bar(kBarCEmpty + i), 2);
    }
    mbar_init(bar(kBarDrain), 1);
    mbar_init(bar(kBarDrain + 1), 1);
    fence_mbar_init_cluster();
  }
  if (tid == 64) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    *W.shared(0) = 0;
    *W.shared(2) = 0;
    *W.shared(1) = *reinterpret_cast<volatile int*>(p.abort_ctr);
  }
  if (tid == 128) {
    tma_prefetch_map(&a.row_map);
    if (a.box && (kFp8 || a.box < 64)) tma_prefetch_map(&a.box_map);
    if (a.box == 64) tma_prefetch_map(&a.k_map);
    if (a.box == 64 && !kFp8) tma_prefetch_map(&a.v_map);
    if (!kFp8) tma_prefetch_map(&a.q_map);
  }
  if (warp == 0) {
    tmem_alloc_pair(sb + C::kOffTmem, kTmemCols);
    tmem_relinquish_pair();
  }
  Unit next{};                                         // (warp 3's)
  Walk walk{};
  bool bad = false;
  // Lane l of the lookups' warp has positions 4 l .. 4 l + 3 of a block, which
  // share a table entry where cache blocks are multiples of four rows (quad).
  struct Entry {
    int off, blk;                                      // row within the block, table entry
    uint32_t seen;                                     // bits of the four positions
  };
  const int per = a.box >> 2;                          // lanes whose rows one copy can bring
  const uint32_t mine = per ? ((1u << per) - 1u) << (lane & ~(per - 1)) : 1u << lane;
  auto entry = [&](const Unit& u, int j) {
    Entry e{0, -1, 0u};
    if (j >= u.nb) return e;
    const int pos = u.template work<kFp8>(j) * kBN + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      e.seen |= (pos + i <= u.p_last && (pos + i >= u.lo || pos + i < u.sinks) ? 1u : 0u) << i;
    // (a copy brings its rows whole where a row of the tile sees one of them)
    if (__ballot_sync(0xffffffffu, e.seen != 0) & mine) {
      const int page = a.shift >= 0 ? pos >> a.shift : pos / p.b.block_size;
      e.off = pos - page * p.b.block_size;
      e.blk = batch_block(p.b, u.r, page, bad);
    }
    return e;
  };
  Entry e0{0, -1, 0u}, e1 = e0, e2 = e0;
  if (warp == 3) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.workers > 0) {
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (the merge)
      walk = start_walk(p, (int)(blockIdx.x >> 1));
      next = next_part(p, walk, (int)(blockIdx.x >> 1), r == 0);
    } else {
      next = find_unit(p, (int64_t)(blockIdx.x >> 1));
    }
    if (a.quad) {
      e0 = entry(next, 0);
      e1 = entry(next, 1);
      e2 = entry(next, 2);
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + C::kOffTmem);
  // The even CTA's barriers, as cluster addresses.
  auto bar0 = [&](int i) { return mapa(bar(i), 0); };
  // Whether the block gave up, the same answer for the whole warp: lanes leave a
  // wait at different times, and a warp that splits here would take the
  // warp-wide instructions below apart.
  auto stopped = [&] { return __any_sync(0xffffffffu, W.aborted()) != 0; };
  // The i-th unit's description, copied by the calling warp, which then lets it
  // go; false behind the last one (or after an abort).
  auto take_unit = [&](int i, Unit& u) {
    W.wait(bar(kBarTFull + (i & 1)), (i >> 1) & 1);
    const int4* src = reinterpret_cast<const int4*>(sm + C::kOffUnit + 48 * (i & 1));
    const int4 x = src[0], y = src[1], z = src[2];
    u.row0 = x.x; u.row1 = x.y; u.p_last = x.z; u.r = x.w;
    u.lo = y.x; u.sinks = y.y; u.sink_blocks = y.z; u.win_block = y.w;
    u.b0 = z.x; u.nb = z.y; u.slot = z.z; u.live = z.w;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarTEmpty + (i & 1)));
    return __all_sync(0xffffffffu, u.live != 0 && !W.aborted()) != 0;
  };
  // The same in place, for a warp that lets it go itself, at the unit's end.
  auto peek_unit = [&](int i) {
    W.wait(bar(kBarTFull + (i & 1)), (i >> 1) & 1);
    return reinterpret_cast<const Unit*>(sm + C::kOffUnit + 48 * (i & 1));
  };
  // Whether this lane's four rows come with one copy of their box: all of the box's
  // rows are there, or all are absent, which a box before the cache's first row
  // reads as zeros.
  auto whole_box = [&](int4& id) {
    const uint32_t there = __ballot_sync(0xffffffffu, (id.x | id.y | id.z | id.w) >= 0);
    const uint32_t absent = __ballot_sync(0xffffffffu, (id.x & id.y & id.z & id.w) < 0);
    if (per == 0) return false;
    if ((absent & mine) == mine) id.x = -64;
    return (there & mine) == mine || (absent & mine) == mine;
  };
  // Blocks are counted across units (J): a barrier's n-th phase is block n's.

  // Descriptors advance by constants (16-byte units).
  if (warp == 0) {
    // ---- QK issuer (even CTA): runs up to two blocks ahead of the softmax ----
    // (Tests that stall it: no scores arrive at all.  Leaving out one block's alone
    // would let the next one's wait pass on the phase before its own.)
    if (r == 0 && !p.inject_stall) {
      const uint32_t id = kFp8 ? idesc_pair_e4m3(128, kBN) : idesc_bf16(128, kBN, false, false);
      const uint64_t dq = sdesc(sb + C::kOffQ, 16, 1024, kLayoutSw128);
      const uint64_t dk = sdesc(sb + C::kOffK, 16, 1024, kLayoutSw128);
      Unit u;
      for (int i = 0, q = 0, J = 0; take_unit(i, u); ++i) {
        if (u.nb > 0) W.wait(bar(kBarQFull), q++ & 1);
        for (int j = 0; j < u.nb; ++j, ++J) {
          if (J >= 2) W.wait(bar(kBarSEmpty + (J & 1)), ((J >> 1) - 1) & 1);
          if (stopped()) break;
          const uint32_t dS = tmem + kColS + 64 * (J & 1);
#pragma unroll 1
          for (int g = 0, c = 0; c < a.atoms; ++g) {
            W.wait(bar(kBarKFull + g), J & 1);
            __syncwarp();
            tc_fence_after();
            const int c1 = min(c + C::kAtomsPerGroup, a.atoms);
            if (elect_one()) {
#pragma unroll 1
              for (int cc = c; cc < c1; ++cc) {
                const uint64_t ad = dq + (uint32_t)cc * (kAtom >> 4);
                const uint64_t bd = dk + (uint32_t)cc * (kAtom >> 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (kFp8) {
                    // (the last atom of 576 channels is half padding)
                    if (4 * cc + i >= a.ksteps) break;
                    mma_pair_e4m3(dS, ad + 2 * i, bd + 2 * i, id, (cc | i) > 0 ? 1u : 0u);
                    mma_pair_e4m3(dS, ad + 2 * i + (C::kMaxAtoms * kAtom >> 4), bd + 2 * i, id, 1u);
                  } else {
                    mma_pair_bf16(dS, ad + 2 * i, bd + 2 * i, id, (cc | i) > 0 ? 1u : 0u);
                  }
                }
              }
              mma_commit_pair(bar(kBarKEmpty + g));
              if (c1 == a.atoms) {
                mma_commit_pair(bar(kBarSFull + (J & 1)));
                if (j == u.nb - 1) mma_commit_pair(bar(kBarQEmpty));
              }
            }
            c = c1;
            __syncwarp();
          }
        }
      }
      // Every MMA issued here has completed (also after an abort) before
      // either CTA frees its TMEM or leaves its tiles.  (Signalled to this CTA
      // alone: nothing may be on its way to the other when it leaves.)
      __syncwarp();
      if (elect_one()) mma_commit_pair(bar(kBarDrain), 1);
      __syncwarp();
      W.drain(bar(kBarDrain), 0);
    }
  } else if (warp == kWarpPv) {
    // ---- PV issuer (even CTA) ------------------------------------------------
    if (r == 0) {
      const uint32_t id = kFp8 ? idesc_pair_e5m2_e4m3(128, 256) : idesc_bf16(128, 256, false, true);
      const uint64_t dp = sdesc(sb + C::kOffP, 16, 1024, kLayoutSw128);
      const uint64_t dv = sdesc(sb + C::kOffV, kAtom, 1024, kLayoutSw128);
      Unit u;
      for (int i = 0, J = 0; take_unit(i, u); ++i) {
        for (int j = 0; j < u.nb; ++j, ++J) {
          const int pb = J % C::kPBufs;
          W.wait(bar(kBarPFull + pb), (J / C::kPBufs) & 1);
          if (stopped()) break;
          const uint64_t dpj = dp + (uint32_t)pb * (C::kPTerms * C::kPTerm >> 4);
#pragma unroll 1
          for (int v = 0; v < kVUnits; ++v) {        // v = 2 n + key half
            W.wait(bar(kBarVFull + v), J & 1);
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t dO = tmem + kColO + 128 * (v >> 1);
              const uint64_t bd = dv + (uint32_t)v * (C::kVUnit >> 4);
              const uint32_t keep = (j > 0 || (v & 1)) ? 1u : 0u;
              if (kFp8) {
                const uint64_t ad = dpj + (uint32_t)(v & 1) * 4;  // 64 keys = 64 bytes
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                  for (int x = 0; x < 3; ++x)
                    mma_pair_e4m3(dO, ad + 2 * ks + x * (C::kPTerm >> 4), bd + 256 * ks, id,
                                  (keep || ks > 0 || x > 0) ? 1u : 0u);
              } else {
                const uint64_t ad = dpj + (uint32_t)(v & 1) * (kAtom >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  mma_pair_bf16(dO, ad + 2 * ks, bd + 128 * ks, id, (keep || ks > 0) ? 1u : 0u);
              }
              mma_commit_pair(bar(kBarVEmpty + v));
              if (v == kVUnits - 1) mma_commit_pair(bar(kBarPEmpty + pb));
            }
            __syncwarp();
          }
        }
      }
      __syncwarp();
      if (elect_one()) mma_commit_pair(bar(kBarDrain + 1), 1);
      __syncwarp();
      W.drain(bar(kBarDrain + 1), 0);
    }
  } else if (warp == 1) {
    // ---- K loads: this CTA's 64 of each block's 128 keys --------------------
    const int groups = (a.atoms + C::kAtomsPerGroup - 1) / C::kAtomsPerGroup;
    int issued = 0;                                  // channel groups loaded, in order
    const int cols = 128 / C::kElem;                 // channels per atom
    const uint32_t kfull0 = bar0(kBarKFull);
    MetaRing mr;
    Unit u;
    int q = 0, J = 0;
    for (int i = 0; take_unit(i, u); ++i) {
      if (!kFp8 && u.nb > 0) {
        if (q >= 1) W.wait(bar(kBarQEmpty), (q - 1) & 1);
        if (stopped()) break;
        if (lane == 0) {
          if (r == 0) mbar_arrive_expect_tx(bar(kBarQFull), 2u * (uint32_t)a.atoms * kAtom);
#pragma unroll 1
          for (int c = 0; c < a.atoms; ++c)
            tma_load_2d_pair(sb + C::kOffQ + c * kAtom, &a.q_map, 64 * c, u.row0 + 64 * (int)r,
                             bar0(kBarQFull));
        }
        ++q;
        __syncwarp();
      }
      for (int j = 0; j < u.nb; ++j, ++J, mr.next()) {
        W.wait(bar(kBarMFull + mr.m), mr.ph);
        int4 id = reinterpret_cast<const int4*>(sm + C::kOffIds)[32 * mr.m + 16 * r + (lane & 15)];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarMEmpty + mr.m));
        // (rows of a block that no row of the tile sees come along: their scores
        // are replaced)
        const bool boxed = whole_box(id);
        const uint32_t ktile = sb + C::kOffK;
        if (a.box == 64 && __all_sync(0xffffffffu, boxed)) {  // the 64 rows as one box
          const int row = __shfl_sync(0xffffffffu, id.x, 0);  // (any lane may be elected)
          if (elect_one()) {
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
              if (J >= 1 && !W.wait(bar(kBarKEmpty + g), (J - 1) & 1)) break;
              const int c0 = g * C::kAtomsPerGroup;
              const uint32_t dst = ktile + c0 * kAtom;
              // E4M3 rows of 576 end in half a column, which the map of whole
              // columns leaves out.  bf16: a column past a row of 512 reads zeros
              // into the tile's spare atom.
              const bool half = kFp8 && c0 + 1 == a.atoms;
              if (r == 0)
                mbar_arrive_expect_tx(bar(kBarKFull + g),
                                      2u * (half ? 1u : (uint32_t)C::kAtomsPerGroup) * kAtom);
              if (half)
                tma_load_2d_pair(dst, &a.box_map, cols * c0, row, kfull0 + 8u * g);
              else
                tma_load_3d_pair(dst, &a.k_map, 0, row, c0, kfull0 + 8u * g);
              ++issued;
            }
          }
          issued = __reduce_max_sync(0xffffffffu, issued);     // (the elected lane's)
          if (stopped()) break;
          continue;
        }
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
          if (J >= 1) W.wait(bar(kBarKEmpty + g), (J - 1) & 1);
          if (stopped()) break;
          const int c0 = g * C::kAtomsPerGroup;
          // (as many columns as the other CTA's whole groups have)
          const int c1 = kFp8 ? min(c0 + C::kAtomsPerGroup, a.atoms) : c0 + C::kAtomsPerGroup;
          if (r == 0 && lane == 0)
            mbar_arrive_expect_tx(bar(kBarKFull + g), 2u * (uint32_t)(c1 - c0) * kAtom);
          __syncwarp();
          if (lane < 16 && (!boxed || (lane & (per - 1)) == 0)) {
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
              const uint32_t dst = ktile + c * kAtom + 4 * lane * 128;
              if (boxed)
                tma_load_2d_pair(dst, &a.box_map, cols * c, id.x, kfull0 + 8u * g);
              else
                tma_gather4_pair(dst, &a.row_map, cols * c, id.x, id.y, id.z, id.w,
                                 kfull0 + 8u * g);
            }
          }
          ++issued;
          __syncwarp();
        }
        if (stopped()) break;
      }
    }
    // Teardown: the last copies into each part have landed in both CTAs (the
    // even CTA's barriers count both; earlier ones were consumed).
    if (r == 0 && lane == 0) {
      if (q > 0) W.drain(bar(kBarQFull), (q - 1) & 1);
#pragma unroll 1
      for (int g = 0; g < groups && g < issued; ++g)
        W.drain(bar(kBarKFull + g), ((issued - 1 - g) / groups) & 1);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- V loads: this CTA's channels of all 128 keys -------------------------
    {
      const uint32_t vfull0 = bar0(kBarVFull);
      int issued = 0, J = 0;                         // (units loaded, in order)
      MetaRing mr;
      Unit u;
      for (int i = 0; take_unit(i, u); ++i) {
        for (int j = 0; j < u.nb; ++j, ++J, mr.next()) {
          W.wait(bar(kBarMFull + mr.m), mr.ph);
          int4 id = reinterpret_cast<const int4*>(sm + C::kOffIds)[32 * mr.m + lane];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarMEmpty + mr.m));
          // Rows behind the last token may never have been written, and a weight of
          // 0 times NaN is NaN: they are read as zeros.  (The other rows of a block
          // were written; one that is not finite costs the tile slow_rows.)
          const int up = u.live - 2 - (u.template work<kFp8>(j) * kBN + 4 * lane);
          if (up < 0) id.x = -1;
          if (up < 1) id.y = -1;
          if (up < 2) id.z = -1;
          if (up < 3) id.w = -1;
          const bool boxed = whole_box(id);
          // Two whole boxes, from one lane (bf16: a prompt 1.31 -> 1.28 ms; E4M3 rows,
          // whose V comes in half as many bytes, lose by it: 1.26 -> 1.30 ms).
          if (!kFp8 && a.box == 64 && __all_sync(0xffffffffu, boxed)) {
            const int near = __shfl_sync(0xffffffffu, id.x, 0);  // (any lane may be elected)
            const int far = __shfl_sync(0xffffffffu, id.x, 16);
            bool on = true;
            if (elect_one()) {
#pragma unroll 1
              for (int v = 0; v < kVUnits; ++v) {
                if (J >= 1 && !W.wait(bar(kBarVEmpty + v), (J - 1) & 1)) {
                  on = false;
                  break;
                }
                if (r == 0) mbar_arrive_expect_tx(bar(kBarVFull + v), 2u * C::kVUnit);
                const int ch = 256 * (v >> 1) + 128 * (int)r, row = v & 1 ? far : near;
                const uint32_t slot = sb + C::kOffV + v * C::kVUnit;
                tma_load_3d_pair(slot, &a.v_map, 0, row, ch / 64, vfull0 + 8u * v);
                ++issued;
              }
            }
            issued = __reduce_max_sync(0xffffffffu, issued);   // (the elected lane's)
            if (__any_sync(0xffffffffu, !on)) break;
            continue;
          }
          // The 16 lanes of a key half: one copy by its first lane where the half is
          // one piece of a cache block, a box per lane group, or four rows per lane.
#pragma unroll 1
          for (int v = 0; v < kVUnits; ++v) {
            if (J >= 1) W.wait(bar(kBarVEmpty + v), (J - 1) & 1);
            if (stopped()) break;
            if (r == 0 && lane == 0) mbar_arrive_expect_tx(bar(kBarVFull + v), 2u * C::kVUnit);
            __syncwarp();
            const uint32_t full_bar = vfull0 + 8u * v;
            const uint32_t slot = sb + C::kOffV + v * C::kVUnit;
            if ((lane >> 4) == (v & 1) && (!boxed || (lane & (per - 1)) == 0)) {
              const int ch = 256 * (v >> 1) + 128 * (int)r;
              const bool one = !kFp8 && boxed && per == 16;
              if (one)
                tma_load_3d_pair(slot, &a.v_map, 0, id.x, ch / 64, full_bar);
#pragma unroll 1
              for (int c = 0; !one && c < (int)(C::kVUnit / kAtom); ++c) {
                const uint32_t dst = slot + c * kAtom + 4 * (lane & 15) * 128;
                if (boxed)
                  tma_load_2d_pair(dst, &a.box_map, ch + 64 * c, id.x, full_bar);
                else
                  tma_gather4_pair(dst, &a.row_map, ch + 64 * c, id.x, id.y, id.z, id.w, full_bar);
              }
            }
            ++issued;
            __syncwarp();
          }
          if (stopped()) break;
        }
        if (stopped()) break;
      }
      if (r == 0 && lane == 0)
#pragma unroll 1
        for (int v = 0; v < kVUnits && v < issued; ++v)
          W.drain(bar(kBarVFull + v), ((issued - 1 - v) / kVUnits) & 1);
      __syncwarp();
    }
  } else if (warp == 3) {
    // ---- units, and lookups: each block's rows, validity bits and scales ------
    // This cluster's own tile comes first, then those it takes over; or the parts of
    // its range.  Both CTAs decode the same answers and read the same batch, so they
    // agree.
    // Lane l looks up positions 4 l .. 4 l + 3.  Where these share a cache block
    // (quad), the table entry of block j + 2 and the scale of block j + 1 are
    // on their way while block j is written down.
    uint32_t* words = reinterpret_cast<uint32_t*>(sm + C::kOffMask);
    const bool keyed = kFp8 && p.kv_format == kE4m3Block;   // (one scale per tensor: at the end)
    MetaRing mr;
    int J = 0;
    struct Found {
      int id[4];
      uint32_t seen;                                   // of those that have a row
      float sc;
    };
    auto found = [&](const Entry& e) {
      Found f;
      f.sc = 1.f;
      f.seen = 0;
      const int64_t row = (int64_t)e.blk * p.b.block_stride_rows + e.off;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = e.blk >= 0 && row + i < p.b.num_slots;
        bad |= e.blk >= 0 && !in && (e.seen >> i & 1u);
        f.id[i] = in ? (int)row + i : -1;
        f.seen |= in ? e.seen & 1u << i : 0u;
      }
      if (keyed && f.id[0] >= 0) f.sc = block_scale(p, e.blk);
      return f;
    };
    int i = 0;                                         // units described
    auto publish = [&](const Unit& x) {
      if (i >= 2) W.wait(bar(kBarTEmpty + (i & 1)), ((i >> 1) - 1) & 1);
      if (stopped()) return;                           // (the slot may still be in use)
      int4* dst = reinterpret_cast<int4*>(sm + C::kOffUnit + 48 * (i & 1));
      if (lane == 0) {
        dst[0] = make_int4(x.row0, x.row1, x.p_last, x.r);
        dst[1] = make_int4(x.lo, x.sinks, x.sink_blocks, x.win_block);
        dst[2] = make_int4(x.b0, x.nb, x.slot, x.live);
        mbar_arrive(bar(kBarTFull + (i & 1)));
      }
      __syncwarp();
      ++i;
    };
    bool pending = false;                              // an answer is on its way
    int n = 0;                                         // answers read
    while (!stopped()) {
      // Ask for the next tile before this one is worked on.
      const uint32_t cfull = bar(kBarCFull + (n & 1));
      const uint32_t answer = sb + C::kOffAnswer + 16 * (n & 1);
      if (p.workers == 0) {
        if (lane == 0) {
          mbar_arrive_expect_tx(cfull, 16);
          if (r == 0) {
            if (n >= 2) W.wait(bar(kBarCEmpty + (n & 1)), ((n >> 1) - 1) & 1);
            cluster_take_over(answer, cfull);
          }
        }
        pending = true;
        __syncwarp();
      }
      const Unit u = next;
      bad |= u.row1 > u.row0 && u.p_last > p.table_end;
      if (u.row1 > u.row0) publish(u);
      Found f = found(e0);
      for (int j = 0; j < u.nb; ++j, ++J, mr.next()) {
        const int m = mr.m;
        int id[4];
        uint32_t seen = 0;
        float sc[4] = {1.f, 1.f, 1.f, 1.f};
        if (a.quad) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            id[k] = f.id[k];
            sc[k] = f.sc;
          }
          seen = f.seen;
          f = found(e1);
          e1 = e2;
          e2 = entry(u, j + 3);
        } else {
          const Rows4 x = lookup4(p, u, u.template work<kFp8>(j) * kBN + 4 * lane, bad);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            id[k] = x.id[k];
            seen |= (id[k] >= 0 ? 1u : 0u) << k;
            if (keyed && id[k] >= 0) sc[k] = block_scale(p, x.blk[k]);
          }
        }
        float own = 1.f;                               // the segment's scale, 0: several
        if (keyed) {
          // (a segment: the 32 keys of eight lanes; keys that no row sees agree
          // with any scale; one that is not finite is left to the path that masks
          // every key by itself)
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (id[k] >= 0) top = fmaxf(top, sc[k]);
#pragma unroll
          for (int o = 1; o <= 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          bool same = true;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (id[k] < 0) sc[k] = top > 0.f ? top : 1.f;
            same &= sc[k] == top && top < INFINITY;
          }
          const uint32_t votes = __ballot_sync(0xffffffffu, same) >> (lane & 24);
          own = (votes & 0xFFu) == 0xFFu ? top : 0.f;
        }
        // The block's rows on their way into L2, two to three blocks before
        // their copies: a copy then waits for L2, not for HBM.
        if (a.box == 64 && (lane & 15) == 0 && id[0] >= 0 && (lane >> 4) == (int)r)
#pragma unroll 1
          for (int c = 0; c < p.d_qk * C::kElem / 128; c += C::kAtomsPerGroup)
            tma_prefetch_3d(&a.k_map, 0, id[0], c);
        if (J >= kMeta) W.wait(bar(kBarMEmpty + m), mr.ph ^ 1);
        if (stopped()) break;
        __syncwarp();
        uint32_t nib = seen << 4 * (lane & 7);
#pragma unroll
        for (int o = 1; o <= 4; o <<= 1) nib |= __shfl_xor_sync(0xffffffffu, nib, o);
        if ((lane & 7) == 0) words[4 * m + (lane >> 3)] = nib;
        reinterpret_cast<int4*>(sm + C::kOffIds)[32 * m + lane] =
            make_int4(id[0], id[1], id[2], id[3]);
        if (kFp8) {
          if ((lane & 7) == 0)
            reinterpret_cast<float4*>(sm + C::kOffSeg)[4 * m + (lane >> 3)] =
                make_float4(own, own > 0.f ? log2f(own) : 0.f, own > 0.f ? 1.f / own : 0.f, 0.f);
          reinterpret_cast<float4*>(sm + C::kOffScale)[32 * m + lane] =
              make_float4(sc[0], sc[1], sc[2], sc[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarMFull + m));
      }
      if (stopped()) break;
      if (p.workers > 0) {
        next = next_part(p, walk, (int)(blockIdx.x >> 1), r == 0);
        if (next.row1 <= next.row0) break;
      } else {
        W.wait(cfull, (n >> 1) & 1);
        if (stopped()) break;
        pending = false;
        int first;
        const bool taken = cluster_taken(answer, first);
        fence_proxy_async_smem();                        // the answer was read
        __syncwarp();
        if (lane == 0) mbar_signal_remote(bar0(kBarCEmpty + (n & 1)));
        if (!taken) break;
        next = find_unit(p, (int64_t)(first >> 1));
        ++n;
      }
      if (a.quad) {
        e0 = entry(next, 0);
        e1 = entry(next, 1);
        e2 = entry(next, 2);
      }
    }
    // (after an abort: an answer on its way still writes to shared memory)
    if (pending && lane == 0) W.drain(bar(kBarCFull + (n & 1)), (n >> 1) & 1);
    __syncwarp();
    next.live = 0;
    publish(next);
    if (bad) atomicCAS(p.status, 0, kStatusBadIndex);
    __syncwarp();
  } else if (warp < 12) {
    // ---- softmax --------------------------------------------------------------
    const int wg = (warp - 4) >> 2;
    const int tl = (warp & 3) * 32 + lane;             // TMEM lane
    const int row = tl & 63, half = tl >> 6;           // tile row, key half
    const int seg = 2 * half + wg;                     // its 32 keys of the block
    const uint32_t lane_base = ((uint32_t)(warp & 3) * 32u) << 16;
    float* red = reinterpret_cast<float*>(sm + C::kOffRed);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(sm + C::kOffMask);
    const uint32_t sempty = bar0(kBarSEmpty), pfull = bar0(kBarPFull);
    // One scale per tensor multiplies every score and the output.
    const float kscale = p.kv_format == kE4m3 ? ld_batch(p.k_scale) : 1.f;
    MetaRing mr;
    int J = 0, q = 0;                                  // blocks, units with blocks
    for (int i = 0;; ++i) {
      const Unit* t = peek_unit(i);
      // (all eight warps leave together: they share the named barriers below)
      if (named_bar_or(4, 256, !t->live || W.aborted())) break;
      int pos = -1, lo = 0;                            // the row's token sees [lo, pos], sinks
      {
        const int g = t->row0 + 64 * (int)r + row;
        if (g < t->row1) pos = t->p_last - ((t->row1 - 1) / p.h - g / p.h);
        if (p.window) lo = max(pos - (p.window - 1), 0);
      }
      const int nb = t->nb;
      // A warp whose 32 rows lie behind the tile's last only keeps step: nothing reads
      // the O that its weights, whatever is in P, make (a mixed batch with 16 heads:
      // 263 -> 258 us).
      const bool idle = t->row0 + 64 * (int)r + (row & 32) >= t->row1;
      float qs = 1.f;
      if (kFp8 && nb > 0) {
        W.wait(bar(kBarQScale), q & 1);
        qs = reinterpret_cast<const float*>(sm + C::kOffQScale)[kRows * (q & 1) + row];
        ++q;
      }
      const float scale = a.scale_log2 * qs * kscale;
      float m_run = -INFINITY;  // running max (log2 units), the same in a row's four threads
      float l_run = 0.f;       // this thread's sum of exp2(s - m_run)
      float lr_run = 0.f;      // the same sum of the bf16-rounded weights
      int blk = nb > 0 ? t->template work<kFp8>(0) : 0;
      // where the order of work leaves the sinks' blocks, or comes to them
      const int jump = kFp8 ? t->sink_blocks - t->b0 : t->b0 + nb - t->sink_blocks;
      for (int j = 0; j < nb; ++j, ++J, mr.next()) {
        const int buf = J & 1, m = mr.m;
        const int e0 = blk * kBN + 32 * seg;             // this thread's first key
        if (j + 1 == jump)
          blk = kFp8 ? t->win_block : t->sink_blocks - 1;
        else
          blk += kFp8 ? 1 : -1;
        W.wait(bar(kBarMFull + m), mr.ph);
        uint32_t see = words[4 * m + seg];
        W.wait(bar(kBarSFull + buf), (J >> 1) & 1);
        __syncwarp();
        if (idle) {
          if (lane == 0) {
            mbar_signal_remote(sempty + 8u * buf);
            mbar_arrive(bar(kBarMEmpty + m));
          }
          if (named_bar_or(4, 256, false) && !kFp8) named_bar_sync(4, 256);
          if (J >= C::kPBufs) W.wait(bar(kBarPEmpty + J % C::kPBufs), (J / C::kPBufs - 1) & 1);
          __syncwarp();
          if (lane == 0) mbar_signal_remote(pfull + 8u * (J % C::kPBufs));
          continue;
        }
        tc_fence_after();
        // The row's view of its 32 keys.
        {
          const int up = pos - e0;                       // keys 0 .. up
          uint32_t v = up >= 31 ? ~0u : up < 0 ? 0u : (2u << up) - 1u;
          const int dn = lo - e0;                        // keys dn ..
          const uint32_t win = dn <= 0 ? ~0u : dn > 31 ? 0u : ~0u << dn;
          const int sk = p.sinks - e0;                   // keys .. sk - 1
          const uint32_t snk = sk <= 0 ? 0u : sk > 31 ? ~0u : (1u << sk) - 1u;
          see &= v & (win | snk);
        }
        float s[32];
        {
          uint32_t w0[16], w1[16];
          const uint32_t col = tmem + lane_base + kColS + 64 * buf + 32 * wg;
          tmem_ld16(col, w0);
          tmem_ld16(col + 16, w1);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            s[k] = __uint_as_float(w0[k]);
            s[16 + k] = __uint_as_float(w1[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_signal_remote(sempty + 8u * buf);
        // Scores in log2 units are s * cl: where nothing is masked and the 32
        // keys share their scale they stay as the MMA left them (the factor is
        // positive and keeps their order).
        float cl = scale;
        // E4M3: the weights are 2^(t - m), t = s + log2(key's scale); `shift` is
        // that log2 and `back` the reciprocal for the 32 keys' common scale.
        float shift = 0.f, back = 1.f;
        bool several = false;
        const float* ks = reinterpret_cast<const float*>(sm + C::kOffScale) + kBN * m + 32 * seg;
        if (kFp8) {
          const float4 own = reinterpret_cast<const float4*>(sm + C::kOffSeg)[4 * m + seg];
          cl *= own.x;
          shift = own.y;
          back = own.z;
          several = !(own.x > 0.f);
          if (__builtin_expect(several, 0)) {
            cl = 1.f;
            back = 0.f;                                  // (their sums are taken below)
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = s[k] * (ks[k] * scale) + __log2f(ks[k]);
          }
        }
        if (__builtin_expect(!__all_sync(0xffffffffu, see == ~0u && cl > 0.f), 0)) {
#pragma unroll
          for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1u ? s[k] * cl : -INFINITY;
          cl = 1.f;
        }
        float hm = fmaxf(s[0], s[1]);
#pragma unroll
        for (int k = 2; k < 32; k += 2) hm = max3(hm, s[k], s[k + 1]);
        hm = fmaf(hm, cl, shift);
        // The row's reference is the largest of its four maxima: all four threads
        // take the same one.  They are read only where some row needs a new one, so
        // a single buffer is free again behind a second barrier there; two spare it.
        float* rb = red + (kFp8 ? 256 * buf : 0);
        rb[64 * seg + row] = hm;
        float alpha = 1.f;
        if (named_bar_or(4, 256, hm > m_run + C::kRaise)) {  // (true for the first finite max)
          float bm = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) bm = fmaxf(bm, rb[64 * k + row]);
          if (!kFp8) named_bar_sync(4, 256);             // (the maxima were read)
          if (bm > m_run + (C::kRaise - 1.f)) {
            alpha = ex2_approx(m_run - bm);              // 0 when m_run = -inf
            if (kFp8) {                                  // (the sums' own range is wider)
              const float half = ex2_approx(0.5f * (m_run - bm));
              l_run = l_run * half * half;
              lr_run = lr_run * half * half;
            }
            m_run = bm;
          }
        }
        // bf16: 16 pairs of weights.  E4M3: three terms of four weights a word.
        uint32_t pk[kFp8 ? 24 : 16];
        float ls = 0.f, ls1 = 0.f, lr = 0.f, lr1 = 0.f;
        const float ref = m_run == -INFINITY ? 0.f : m_run;           // (no score: weights are 0)
        const float mm = ref - shift;
        if constexpr (kFp8) {
          // The divisor, sum of weight / scale: where the 32 keys share their scale the
          // weights as the product has them, so that a key that carries the row keeps
          // its V.  The product has nothing of weights that lie far below the row's
          // reference (f16 ends at 2^-33 of it), but 1 / scale may make them most of
          // the softmax: from 2^-15 on their fp32 sum divides, from 2^-90 on (where
          // fp32 begins to end) the sum of 2^(s - m), without the scale.
          const bool low = hm < ref - 15.f;
          float bare = 0.f;
          if (__builtin_expect(several, 0)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float e = ex2_approx(s[k] - __log2f(ks[k]) - ref);
              bare += s[k] == -INFINITY ? 0.f : e;       // (masked, whatever its scale)
            }
          } else if (__builtin_expect(
                         __any_sync(0xffffffffu, hm < ref - 90.f && hm > -INFINITY), 0)) {
#pragma unroll
            for (int k = 0; k < 32; ++k) bare += ex2_approx(fmaf(s[k], cl, -ref));
          }
          // at most 2^15: within E5M2's range, whose grid is 2^-27 of a weight of 1
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& s0 = s[k + 2 * e];
              float& s1 = s[k + 2 * e + 1];
              fma2_bcast(s0, s1, cl, 15.f - C::kRaise - mm);
              const float w0 = ex2_approx(s0), w1 = ex2_approx(s1);
              add2(ls, ls1, w0, w1);
              h[e] = (pack_f16(w0, w1) + 0x00020002u) & 0xFFFCFFFCu;  // 9 significant bits
              add_f16x2_f32x2(lr, lr1, h[e]);
              s0 = w0;
              s1 = w1;
            }
#pragma unroll
            for (int x = 0; x < 3; ++x) {
              if (x == 2) {                              // what is left, to the nearest
                h[0] += 0x00800080u;
                h[1] += 0x00800080u;
              }
              pk[8 * x + k / 4] = __byte_perm(h[0], h[1], 0x7531);   // the four upper bytes
              if (x < 2) {
                h[0] = sub_f16x2(h[0], h[0] & 0xFF00FF00u);
                h[1] = sub_f16x2(h[1], h[1] & 0xFF00FF00u);
              }
            }
          }
          back *= C::kBack;
          ls = several || hm < ref - 90.f ? bare : (ls + ls1) * back;
          lr = several || low ? ls : (lr + lr1) * back;  // (9 bits: 2^-9 of a weight at most)
          l_run += ls;
          lr_run += lr;
        } else {
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            fma2_bcast(s[k], s[k + 1], cl, -mm);
            const float w0 = ex2_approx(s[k]), w1 = ex2_approx(s[k + 1]);
            add2(ls, ls1, w0, w1);
            pk[k / 2] = pack_bf16(w0, w1);
            add_bf16x2_f32x2(lr, lr1, pk[k / 2]);
          }
          l_run = l_run * alpha + (ls + ls1);
          lr_run = lr_run * alpha + (lr + lr1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarMEmpty + m));  // the lookups were read
        if (j >= 1 && __any_sync(0xffffffffu, alpha != 1.f)) {
          W.wait(bar(kBarPEmpty + (J - 1) % C::kPBufs), ((J - 1) / C::kPBufs) & 1);  // PV(j - 1)
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 128 * wg; c < 128 * wg + 128; c += 16) {
            uint32_t w[16];
            tmem_ld16(tmem + lane_base + kColO + c, w);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * alpha);
            tmem_st16(tmem + lane_base + kColO + c, w);
          }
          tmem_wait_st();
        }
        const int pb = J % C::kPBufs;
        if (J >= C::kPBufs)                              // the buffer was read
          W.wait(bar(kBarPEmpty + pb), (J / C::kPBufs - 1) & 1);
        // P row: bf16, keys 64 half + 32 wg .. + 31 as chunks 4 wg .. of atom `half`;
        // E4M3, bytes 32 seg .. + 31 of each term's row.
        uint8_t* prow = sm + C::kOffP + pb * (C::kPTerms * C::kPTerm) + row * 128;
        const uint32_t sw = (uint32_t)row & 7u;
        if constexpr (kFp8) {
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<uint4*>(prow + x * C::kPTerm +
                                        (((uint32_t)(2 * seg + c) ^ sw) << 4)) =
                  make_uint4(pk[8 * x + 4 * c], pk[8 * x + 4 * c + 1], pk[8 * x + 4 * c + 2],
                             pk[8 * x + 4 * c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(prow + half * kAtom + (((uint32_t)(4 * wg + c) ^ sw) << 4)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_signal_remote(pfull + 8u * pb);
      }

      // ---- epilogue -------------------------------------------------------------
      if (nb > 0) {
        W.wait(bar(kBarPEmpty + (J - 1) % C::kPBufs), ((J - 1) / C::kPBufs) & 1);
        __syncwarp();
        tc_fence_after();
      }
      float* sums = reinterpret_cast<float*>(sm + C::kOffP + kOffSums);
      int* flag = reinterpret_cast<int*>(sm + C::kOffP + kOffFlag);
      sums[64 * seg + row] = l_run;
      sums[256 + 64 * seg + row] = lr_run;
      if (seg == 0) flag[row] = 0;
      named_bar_sync(4, 256);
      float l = 0.f, lr = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l += sums[64 * k + row];
        lr += sums[256 + 64 * k + row];
      }
      const bool empty = l == 0.f;
      // (a sum that is not finite: NaN, whatever the weights' terms became)
      const float top = kscale * C::kBack;
      const float inv = empty ? 0.f : l < INFINITY ? __fdividef(top, lr) : NAN;
      const bool partial = t->slot >= 0;
      const int64_t g = (int64_t)t->row0 + 64 * (int)r + row;
      const bool live = g < t->row1;
      const int64_t prow_g = (int64_t)t->slot * 128 + 64 * (int)r + row;  // row of the partials
      // O columns [128 wg, + 128) are channels 256 wg + 128 half ..; a thread's
      // stores fill whole 32-byte sectors, straight from registers.
      const int ch0 = 256 * wg + 128 * half;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out);
      bool odd = false;                                  // an output that is not finite
      auto fetch = [&](int c, uint32_t (&w)[2][16]) {
        __syncwarp();
        tmem_ld16(tmem + lane_base + kColO + 128 * wg + c, w[0]);
        tmem_ld16(tmem + lane_base + kColO + 128 * wg + c + 16, w[1]);
      };
      auto put = [&](int c4, uint32_t (&wide)[2][16]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t (&w)[16] = wide[x];
          const int c = c4 + 16 * x;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float o = empty ? 0.f : __uint_as_float(w[k]) * inv;
            odd |= !(fabsf(o) < INFINITY);
            w[k] = __float_as_uint(o);
          }
          if (live && partial && !empty) {
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.o_part + prow_g * 512 + ch0 + c);
            st_global_32(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
            st_global_32(dst + 8, w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]);
          }
          if (live && !partial) {
            uint32_t b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              b[k] = pack_bf16(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
            uint32_t* dst = reinterpret_cast<uint32_t*>(out + g * 512 + ch0 + c);
            if (a.wide) {
              st_global_32(dst, b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7]);
            } else {
              reinterpret_cast<uint4*>(dst)[0] = make_uint4(b[0], b[1], b[2], b[3]);
              reinterpret_cast<uint4*>(dst)[1] = make_uint4(b[4], b[5], b[6], b[7]);
            }
          }
        }
      };
      if (!idle) {
        // (32 columns are on their way from TMEM while 32 are stored: a prompt's time
        // is 2.6 % less)
        uint32_t wa[2][16], wb[2][16];
        fetch(0, wa);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          fetch(c + 32, wb);
          put(c, wa);
          tmem_wait_ld();
          if (c == 0) fetch(64, wa);
          put(c + 32, wb);
          tmem_wait_ld();
        }
      }
      if (live && seg == 0) {
        const float v = empty ? -INFINITY : (m_run + log2f(l)) * 0.69314718055994530942f;
        if (partial)
          p.lse_part[prow_g] = v;
        else if (p.lse)
          p.lse[g] = v;
      }
      // A softmax that is not finite (a NaN or infinite visible score) is the
      // answer; a finite one with an output that is not may owe it to a masked
      // position: the row is computed again and written over.
      odd = odd && live && l < INFINITY && lr < INFINITY;
      if (odd) flag[row] = 1;
      if (__builtin_expect(named_bar_or(4, 256, odd), 0)) {  // (also orders the stores before)
        slow_rows<kFp8>(p, *t, sm + C::kOffP, W, r);
      }
      // (the next unit's first weights are signalled behind these TMEM loads)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarTEmpty + (i & 1)));
    }
    __syncwarp();
  } else if (kFp8) {
    // ---- Q rows -> two E4M3 terms under a power-of-two scale ------------------
    // Eight lanes a row; the next unit's rows are split while the last blocks of
    // the one before are still in the softmax.
    const int j8 = lane & 7, g0 = 4 * (warp - 13) + (lane >> 3);   // of 12 groups
    const uint32_t gmask = 0xFFu << (lane & 24);
    const int nch = p.d_qk / 64;
    Unit u;
    for (int i = 0, q = 0; take_unit(i, u); ++i) {
      if (u.nb <= 0) continue;
      // (a row's loads are on their way while the row before is split, the first
      // row's before the tile's shared memory is free: 100 decode tokens 117 -> 113 us)
      uint4 ahead[9];
      auto load_row = [&](int rr) {
        const int64_t gr = (int64_t)u.row0 + 64 * (int)r + rr;
        const bool have = rr < kRows && gr < u.row1;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q) + (have ? gr : u.row0) * p.d_qk) + j8;
#pragma unroll
        for (int c = 0; c < 9; ++c)
          ahead[c] = have && c < nch ? ld_q16(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      };
      load_row(g0);
      if (q >= 1) W.wait(bar(kBarQEmpty), (q - 1) & 1);
      __syncwarp();
      float* qscale = reinterpret_cast<float*>(sm + C::kOffQScale) + kRows * (q & 1);
#pragma unroll 1
      for (int rr = g0; rr < kRows; rr += 12) {
        const int64_t gr = (int64_t)u.row0 + 64 * (int)r + rr;
        if (gr - (rr & 31) >= u.row1) break;           // (rows of an idle softmax warp)
        uint4 raw[9];
#pragma unroll
        for (int c = 0; c < 9; ++c) raw[c] = ahead[c];
        load_row(rr + 12);
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 9; ++c) {
          const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = max3(amax, fabsf(__uint_as_float(w[e] << 16)),
                        fabsf(__uint_as_float(w[e] & 0xFFFF0000u)));
        }
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(gmask, amax, o));
        // 2^k with amax 2^k in [224, 448): amax = m 2^e, 1 <= m < 2, k = 8 - e
        // (m < 1.75) or 7 - e; kept within what 2^-k can hold
        const uint32_t bits = __float_as_uint(amax);
        int k = 8 - ((int)(bits >> 23) - 127) - ((bits & 0x7FFFFFu) >= 0x600000u ? 1 : 0);
        k = amax == 0.f ? 0 : min(max(k, -120), 120);
        const float up = __uint_as_float((uint32_t)(k + 127) << 23);
        if (j8 == 0)                                   // (an infinite q: NaN scores)
          qscale[rr] = amax < INFINITY ? __uint_as_float((uint32_t)(127 - k) << 23) : NAN;
#pragma unroll
        for (int c = 0; c < 10; ++c) {                 // 64-channel pieces; a tenth is padding
          if (c >= 2 * a.atoms) break;
          const uint4 v = c < 9 ? raw[c < 9 ? c : 0] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t hi[2], lw[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x[4], y0, y1, y2, y3;
            x[0] = __uint_as_float(w[2 * e] << 16) * up;
            x[1] = __uint_as_float(w[2 * e] & 0xFFFF0000u) * up;
            x[2] = __uint_as_float(w[2 * e + 1] << 16) * up;
            x[3] = __uint_as_float(w[2 * e + 1] & 0xFFFF0000u) * up;
            hi[e] = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
            e4m3x4_to_f32(hi[e], y0, y1, y2, y3);
            lw[e] = e4m3x2(x[0] - y0, x[1] - y1) | (e4m3x2(x[2] - y2, x[3] - y3) << 16);
          }
          // channel 64 c + 8 j8: atom c / 2, 16-byte chunk 4 (c % 2) + j8 / 2
          const uint32_t off = (uint32_t)(c >> 1) * kAtom + (uint32_t)rr * 128u +
                               (((4u * (c & 1) + (j8 >> 1)) ^ ((uint32_t)rr & 7u)) << 4) +
                               8u * (j8 & 1);
          *reinterpret_cast<uint2*>(sm + C::kOffQ + off) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(sm + C::kOffQ + C::kMaxAtoms * kAtom + off) =
              make_uint2(lw[0], lw[1]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kBarQScale));
        mbar_signal_remote(bar0(kBarQFull));
      }
      ++q;
    }
    __syncwarp();
  }

  // ---- teardown: both CTAs are done with each other's barriers, tiles and
  // TMEM (the even CTA drained the MMAs and the pair's copies above).  Where one
  // gave up, the two may have issued different copies (the signals of an aborted
  // issuer let the other CTA's loaders go on), whose barriers then tell nothing,
  // and a copy must not outlive the CTA that holds its barrier: a CTA that gave up
  // says so to the other, and both wait 100 us for what is in flight.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && W.aborted()) st_cluster_s32(mapa(sb + C::kOffAbort, r ^ 1u), 1);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (W.aborted()) {                                   // (the same in both CTAs)
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000u) {
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---- merge of the partials -------------------------------------------------
//   LSE = ln sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s
// One CTA per row, four channels a thread, and where a tile may have more than 16
// parts eight groups of threads that share them; the ranges first .. last hold the
// row's tile (one: it is written already), the last as its first part and the
// others as their last.  A part without a visible key has LSE_s = -inf and its
// O_s is not read.  Rows of no request are left alone.  Launched under the end of
// the kernel before (launch_early); it waits for it here.
constexpr int kMaxParts = 128;
constexpr int kMergeGroups = 8;
__global__ void __launch_bounds__(128 * kMergeGroups)
smla_window_merge_kernel(const WinParams p) {
  __shared__ float weight[kMaxParts];
  __shared__ float red[2][4];
  __shared__ float4 sums[kMergeGroups][128];
  const int tid = threadIdx.x & 127, group = threadIdx.x >> 7, groups = blockDim.x >> 7;
  const int64_t row = blockIdx.x;
  const int tok = (int)(row / p.h);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int part = p.parts[row];
  if (tok < batch_start(p.b, 0) || tok >= batch_start(p.b, p.b.num_reqs)) return;
  const int first = part >> 19, last = (part >> 7) & 0xFFF, off = part & 127;
  // (starts that do not ascend leave rows without a tile, and this word as it was)
  if (part < 0 || first >= last || last >= p.workers) return;
  const int n = last - first + 1;
  auto at = [&](int s) {
    return (int64_t)(2 * (first + s) + (first + s < last ? 1 : 0)) * 128 + off;
  };
  const float ls = tid < n ? p.lse_part[at(tid)] : -INFINITY;   // (every group alike)
  float top = ls;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (group == 0 && (tid & 31) == 0) red[0][tid >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  // (fmaxf passes over a NaN; its weight is NaN and so is the row)
  const float e = ls == -INFINITY ? 0.f : expf(ls - top);
  float z = e;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (group == 0 && (tid & 31) == 0) red[1][tid >> 5] = z;
  if (group == 0) weight[tid] = e;
  __syncthreads();
  z = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int c = tid * 4;
  for (int s0 = group; s0 < n; s0 += 8 * groups) {     // eight parts on their way at once
    float4 x[8];
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int s = s0 + i * groups;
      w[i] = s < n ? weight[s] : 0.f;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (w[i] != 0.f) x[i] = *reinterpret_cast<const float4*>(p.o_part + at(s) * 512 + c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o.x = fmaf(w[i], x[i].x, o.x);
      o.y = fmaf(w[i], x[i].y, o.y);
      o.z = fmaf(w[i], x[i].z, o.z);
      o.w = fmaf(w[i], x[i].w, o.w);
    }
  }
  if (groups > 1) {
    sums[group][tid] = o;
    __syncthreads();
    if (group > 0) return;
    for (int g = 1; g < groups; ++g) {
      const float4 x = sums[g][tid];
      o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
    }
  }
  const bool none = z == 0.f;
  const float inv = none ? 0.f : 1.f / z;
  uint2 packed = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * 512 + c) = packed;
  if (tid == 0 && p.lse) p.lse[row] = none ? -INFINITY : top + logf(z);
}

cudaError_t encode_rows(CUtensorMap* map, bool fp8, const void* base, int d, int64_t rows,
                        int box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const int es = fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// The cache as (128-byte column, row, column index): one copy brings several
// columns of 64 rows, each as a tile of its own.  The column count is that of
// whole columns.
cudaError_t encode_columns(CUtensorMap* map, bool fp8, const void* base, int d, int64_t rows,
                           int box_columns) {
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const int es = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)(128 / es), (cuuint64_t)rows, (cuuint64_t)(d * es / 128)};
  const cuuint64_t strides[2] = {(cuuint64_t)d * es, 128};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / es), 64, (cuuint32_t)box_columns};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// Launch a kernel that waits for the one before it on the stream by itself
// (griddepcontrol.wait), so that its launch and setup pass under that one's end:
// 1 to 2 us of a call, 3 of the merge.
template <class Params>
cudaError_t launch_early(void (*kernel)(Params), unsigned ctas, int threads, uint32_t smem,
                         cudaStream_t stream, const std::remove_const_t<Params>& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool kFp8>
cudaError_t launch(const WinArgs& a, unsigned ctas, cudaStream_t stream) {
  using C = Cfg<kFp8>;
  // (once per device: the attribute call costs as much as a launch)
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
    e = cudaFuncSetAttribute(smla_window_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return launch_early(smla_window_kernel<kFp8>, ctas, C::kThreads, C::kSmem, stream, a);
}

int64_t tile_numbers(int T, int h, int num_reqs) {
  return h == 128 ? T : (int64_t)T * h / 128 + num_reqs;
}

}  // namespace

// One unit per tile, or equal ranges of all tiles' blocks (WinParams::workers).
// What is known here are bounds: the tiles are taken as filled (a decode step's
// requests hold one each), the keys as max_len or the window.  A block takes about
// 1.6 us on a pair, a unit another 4; ranges cost the merge (4) and write and read
// the partials, 4 KB a row, at about 9 TB/s (L2).  Ranges are taken
// where they save a twentieth.  They need the list's length, which every cluster
// counts: up to 1024 tiles and requests.
WindowPlan make_window_plan(int T, int h, int num_reqs, int64_t max_len, int window, int sinks,
                            int num_sms) {
  WindowPlan pl{};
  pl.tiles = tile_numbers(T, h, num_reqs);
  const int64_t filled = std::max<int64_t>(std::min(num_reqs, T), ((int64_t)T * h + 127) / 128);
  int64_t keys = max_len;
  if (window) keys = std::min<int64_t>(keys, (int64_t)window + (128 + h - 1) / h);
  int64_t blocks = (keys + kBN - 1) / kBN;
  if (window && keys < max_len) blocks += 1 + (std::min<int64_t>(sinks, max_len) + kBN - 1) / kBN;
  blocks = std::max<int64_t>(blocks, 1);
  const int64_t places = std::min(std::max(num_sms / 2, 1), kMaxParts);
  const double one = (double)((filled + places - 1) / places) * (1.6 * (double)blocks + 4.0);
  const int64_t list = filled * (blocks + kTileCost) - kTileCost;
  const int64_t workers = std::min<int64_t>(places, filled * blocks);
  const double rows = (double)T * h / (double)filled;
  const double ranges = 1.6 * (double)((list + workers - 1) / workers) + 4.0 + 4.0 +
                        (double)(workers + std::min(filled, workers)) * rows * 4096.0 / 9e6;
  if (workers > 1 && std::max<int64_t>(pl.tiles, num_reqs) <= 1024 && ranges < 0.95 * one)
    pl.workers = (int)workers;
  pl.merge_groups = workers > 16 * filled ? kMergeGroups : 1;
  if (pl.workers > 0)
    pl.workspace_bytes = ((size_t)T * h * sizeof(int) + 255) / 256 * 256 +
                         (size_t)pl.workers * 2 * 128 * (512 + 1) * sizeof(float);
  return pl;
}

cudaError_t launch_window(WinParams p, cudaStream_t stream) {
  WinArgs a{};
  const bool fp8 = p.kv_format != kBf16;
  const int es = fp8 ? 1 : 2;
  p.num_tiles = tile_numbers(p.b.N, p.h, p.b.num_reqs);
  p.table_end =
      (int)std::min<int64_t>((int64_t)p.b.bt_stride * p.b.block_size, 0x7FFFFF00) - 1;
  p.sinks = std::min(p.sinks, 0x7FFFFF00);             // (more than any position)
  a.atoms = (p.d_qk * es + 127) / 128;
  a.ksteps = p.d_qk * es / 32;
  a.scale_log2 = p.sm_scale * 1.4426950408889634f;
  // Boxes: the largest power of two that divides the block (and 64); blocks of
  // other sizes than multiples of 4 take gather4 alone.
  a.box = p.b.block_size & -p.b.block_size;
  a.box = a.box > 64 ? 64 : a.box < 4 ? 0 : a.box;
  a.quad = p.b.block_size % 4 == 0;
  a.shift = -1;
  for (int k = 0; k < 31; ++k)
    if (p.b.block_size == 1 << k) a.shift = k;
  a.wide = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  cudaError_t e = encode_rows(&a.row_map, fp8, p.kv, p.d_qk, p.b.num_slots, 1);
  if (e == cudaSuccess && a.box && (fp8 || a.box < 64))
    e = encode_rows(&a.box_map, fp8, p.kv, p.d_qk, p.b.num_slots, a.box);
  if (e == cudaSuccess && a.box == 64)
    e = encode_columns(&a.k_map, fp8, p.kv, p.d_qk, p.b.num_slots, fp8 ? 2 : 3);
  if (e == cudaSuccess && a.box == 64 && !fp8)
    e = encode_columns(&a.v_map, fp8, p.kv, p.d_qk, p.b.num_slots, 2);
  if (e == cudaSuccess && !fp8)
    e = encode_rows(&a.q_map, false, p.q, p.d_qk, (int64_t)p.b.N * p.h, kRows);
  if (e != cudaSuccess) return e;
  const int64_t ctas = 2 * (p.workers > 0 ? p.workers : p.num_tiles);
  if (ctas > 0x7FFFFFFFll || (int64_t)p.b.N * p.h > 0x7FFFFFFFll)
    return cudaErrorInvalidConfiguration;
  a.p = p;
  e = fp8 ? launch<true>(a, (unsigned)ctas, stream) : launch<false>(a, (unsigned)ctas, stream);
  if (e != cudaSuccess || p.workers == 0) return e;
  return launch_early(smla_window_merge_kernel, (unsigned)(p.b.N * p.h), 128 * p.merge_groups, 0,
                      stream, p);
}

}  // namespace smla
