// smla_blocks.cu — the blocks of a paged latent cache: copied in every layer at
// once, shared by forked table rows until one of them is written, given back, and
// moved together at the start of the pool.
//
// State.  A table row lists the cache blocks of a request, refcount[b] counts the
// table entries that hold block b (0: free).  Nothing else is kept: a free block is
// found by scanning the counts, and the lowest one is taken first, so the same
// calls give the same tables whatever the order of the threads, and a scheduler on
// the host that follows the rule knows the tables without reading them.
//
//   fork      row'[c] = parent's entry for c < ceil(len / B);  ref' = ref - (entries of
//             the rows replaced) + (entries of the new rows); the last block of a row
//             that will be written (room > 0) becomes its own where others hold it;
//             then blocks for the positions [len, len + room).  Where no block is left
//             for a row's own last one, it keeps the shared one: what it has written
//             stays, and a later call finds the copy still to be made
//   free      entries of blocks that lie in [begin, end) -> -1, ref' = ref - those
//   compact   L live blocks: the k-th highest of those numbered L or more goes to the
//             k-th lowest free number below L.  With lr(b) = live blocks below b, that
//             is k = L - 1 - lr(b) for a live block and k = b - lr(b) for a free
//             place: each finds its own k, and no block is both read and written.
//
// Bound: latency for the tables (the launches of a call follow one another, each
// under the end of the one before), HBM for the rows of a pool.  Measured in a captured
// graph, on two sets of inputs in turn: 225 bf16 blocks of 64 rows in 24 layers 123 us =
// 6.4 TB/s read and written (94 % of a copy's rate), one block in 60 layers 2.5 us; eight samples
// of a prompt 10.9 us, 256 beams in 32 layers of E4M3 blocks 32.7 us (100 MB, of them 17 us
// the tables); a finished sixteenth of 64 rows 4 us, 1024 rows' windows 11.3 us; half a
// pool of 3814 blocks in 6 layers 138 us = 6.1 TB/s.
// Each pair looks at all the others for a child named again and, in one cluster, for
// writers of its last block, so many pairs cost their square: rows that go on, 1024 of 16
// columns 21 us, 4096 119 us, 16384 1.5 ms, 65536 22 ms; as many rows freed 5, 9, 43 and
// 420 us.
#include "launch.cuh"
#include "smla_blocks.h"

namespace smla {
namespace {

__device__ __forceinline__ void wait_before() {      // for the kernel before on the stream
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bad_index(int* status) { atomicCAS(status, 0, kStatusBadIndex); }

// ------------------------------------------------------------- copying --

constexpr int kCopyThreads = 256;
constexpr int kPiece = 16384;              // bytes of a block that a CTA copies at a time
constexpr int kCopyCtas = 152 * 8;         // as many as run at once

struct CopyParams {
  uint8_t* cache[kPoolLayers];
  float* scale[kPoolLayers];
  int layers, pieces;                      // pieces: CTAs that share a block
  int row_bytes, groups, block_size, block_stride_rows;
  // The moves: n of them, or *n_at.  Move i copies `rows` rows (nullptr: whole blocks)
  // of src[i] to dst[i], or to list[dst[i]], a list of *list_n blocks.
  const int32_t* src;
  const int32_t* dst;
  const int32_t* list;
  const int32_t* list_n;
  const int32_t* rows;
  const int32_t* n_at;
  int n, blocks;
  int* status;
};

// Piece by piece, 64 bytes a thread in flight.
__device__ __forceinline__ void copy_block(const CopyParams& c, int layer, int piece, int src,
                                           int dst, int rows) {
  const int tid = threadIdx.x;
  const int64_t step = (int64_t)c.block_stride_rows * c.row_bytes;
  const int64_t bytes = (int64_t)rows * c.row_bytes;
  const uint8_t* from = c.cache[layer] + src * step;
  uint8_t* to = c.cache[layer] + dst * step;
  for (int64_t at = (int64_t)piece * kPiece; at < bytes; at += (int64_t)c.pieces * kPiece) {
    const uint4* s = reinterpret_cast<const uint4*>(from + at) + tid;
    uint4* d = reinterpret_cast<uint4*>(to + at) + tid;
    const int left = (int)min((bytes - at) >> 4, (int64_t)(kPiece / 16)) - tid;
    constexpr int kLoads = kPiece / 16 / kCopyThreads;
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i * kCopyThreads < left) v[i] = s[i * kCopyThreads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i * kCopyThreads < left) d[i * kCopyThreads] = v[i];
  }
  if (piece != 0 || c.groups == 0) return;
  float* scale = c.scale[layer];
  if (c.groups < 0) {
    if (tid == 0) scale[dst] = scale[src];
    return;
  }
  const int64_t n = (int64_t)rows * c.groups;
  const float* s = scale + (int64_t)src * c.block_stride_rows * c.groups;
  float* d = scale + (int64_t)dst * c.block_stride_rows * c.groups;
  for (int64_t i = tid; i < n; i += kCopyThreads) d[i] = s[i];
}

// CTA `id` of the copying ones: a piece of a layer, for every `share`-th move.  A move is
// read while the one before it is copied (a pool of 6 layers, half free: 142 -> 138 us).
__device__ __forceinline__ void copy_moves(const CopyParams& c, int id, int share) {
  // (unsigned: the number behind the last move may pass 2^31)
  const uint32_t n = c.n_at ? *c.n_at : c.n;
  const int list_n = c.list ? *c.list_n : 0;
  const int piece = id % c.pieces, rest = id / c.pieces;
  const int layer = rest % c.layers;
  struct Move {
    int src, dst, rows;
  };
  auto read = [&](uint32_t m) {
    Move v{-1, -1, 0};
    if (m < n) {
      v.src = c.src[m];
      v.dst = c.dst[m];
      v.rows = c.rows ? c.rows[m] : c.block_size;
      if (c.list) v.dst = v.dst < list_n ? c.list[v.dst] : -1;
    }
    return v;
  };
  Move next = read(rest / c.layers);
  for (uint32_t m = rest / c.layers; m < n; m += share) {
    const Move v = next;
    next = read(m + share);
    if (v.src >= c.blocks || v.dst >= c.blocks) {
      if (piece == 0 && layer == 0 && threadIdx.x == 0) bad_index(c.status);
      continue;
    }
    if (v.src < 0 || v.dst < 0 || v.src == v.dst) continue;
    // (parts of blocks fill the first pieces alone: a CTA takes them in turn; 256 beams:
    // 34.2 -> 32.7 us)
    const int at = c.rows ? (int)((piece + m) % (uint32_t)c.pieces) : piece;
    copy_block(c, layer, at, v.src, v.dst, v.rows);
  }
}

__global__ void __launch_bounds__(kCopyThreads) smla_block_copy_kernel(
    const __grid_constant__ CopyParams c) {
  wait_before();
  allow_next();
  copy_moves(c, (int)blockIdx.x, (int)gridDim.x / (c.pieces * c.layers));
}

// The layers [first, first + kPoolLayers) of a pool.
CopyParams copy_params(const Pool& pool, int first) {
  CopyParams c{};
  c.layers = pool.layers - first < kPoolLayers ? pool.layers - first : kPoolLayers;
  for (int l = 0; l < c.layers; ++l) {
    c.cache[l] = static_cast<uint8_t*>(pool.cache[first + l]);
    c.scale[l] = pool.scale ? pool.scale[first + l] : nullptr;
  }
  c.row_bytes = pool.row_bytes;
  c.groups = pool.scale ? pool.groups : 0;
  c.block_size = pool.block_size;
  c.block_stride_rows = pool.block_stride_rows;
  const int64_t pieces = ((int64_t)pool.block_size * pool.row_bytes + kPiece - 1) / kPiece;
  c.pieces = pieces < 64 ? (int)pieces : 64;
  return c;
}
// CTAs for at most n moves.
unsigned copy_ctas(const CopyParams& c, int64_t n) {
  const int one = c.layers * c.pieces;
  int64_t share = (kCopyCtas + one - 1) / one;
  if (share > n) share = n;
  return (unsigned)(one * (share < 1 ? 1 : share));
}

// -------------------------------------------------------------- scans --

// One cluster scans the counts: its warps have neighbouring ranges of the blocks.
constexpr int kCluster = 8;
constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kCluster * kScanThreads / 32;

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range warp_range(int blocks, int warp) {
  const int64_t per = ((int64_t)blocks + kScanWarps - 1) / kScanWarps;
  const int64_t lo = per * warp;
  return {(int)min(lo, (int64_t)blocks), (int)min(lo + per, (int64_t)blocks)};
}
// Blocks of the range for which yes(ref).
template <class Yes>
__device__ __forceinline__ int count_range(const int32_t* ref, Range r, Yes yes) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 8
  for (int b = r.lo + lane; b < r.hi; b += 32) n += yes(__ldcg(ref + b)) ? 1 : 0;
  return warp_sum(n);
}
// The sum of the counts below `warp`, and of all.
__device__ __forceinline__ int2 warp_base(const int32_t* counts, int warp) {
  const int lane = threadIdx.x & 31;
  int below = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kScanWarps / 32; ++i) {
    const int w = 32 * i + lane, x = __ldcg(counts + w);
    all += x;
    below += w < warp ? x : 0;
  }
  return make_int2(warp_sum(below), warp_sum(all));
}

// --------------------------------------------------------------- tables --

constexpr int kRowThreads = 256;

// Tables and counts to their new place (n = 0: in place already).
struct Carry {
  const int32_t* from[3];
  int32_t* to[3];
  int64_t n[3];
};
__device__ __forceinline__ void carry(const Carry& p, int64_t id, int64_t threads) {
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll 4
    for (int64_t i = id; i < p.n[k]; i += threads) p.to[k][i] = p.from[k][i];
}
__global__ void __launch_bounds__(kRowThreads) smla_tables_carry_kernel(const Carry p) {
  wait_before();
  allow_next();
  carry(p, (int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}

Carry make_carry(const Tables& t) {
  Carry p{};
  auto add = [&](int k, const int32_t* from, int32_t* to, int64_t n) {
    p.from[k] = from;
    p.to[k] = to;
    p.n[k] = from && from != to ? n : 0;
  };
  add(0, t.table, t.table_out, (int64_t)t.rows * t.width);
  add(1, t.lens, t.lens_out, t.rows);
  add(2, t.ref, t.ref_out, t.blocks);
  return p;
}
int64_t most_of(const Carry& p) {
  int64_t most = p.n[0] > p.n[1] ? p.n[0] : p.n[1];
  return p.n[2] > most ? p.n[2] : most;
}
cudaError_t launch_carry(const Carry& p, cudaStream_t stream) {
  const int64_t ctas = (most_of(p) + 4 * kRowThreads - 1) / (4 * kRowThreads);
  if (ctas == 0) return cudaSuccess;
  return launch_early(smla_tables_carry_kernel, (unsigned)(ctas < 152 * 8 ? ctas : 152 * 8),
                      kRowThreads, 0, stream, p);
}

// Tables and pairs of a fork this small are handled by one cluster in one launch (a warp
// per pair), larger ones by a launch for each step that needs the one before it complete.
// The words are those of the largest array that is carried and of the children's rows.
// One cluster / a launch a step, us in a graph, rows that go on in place, four samples a
// row apart, eight new samples apart: 8 rows of 65 columns 7.6 / 8.8, 9.3 / 11.9, 9.4 /
// 11.9; 256 of 127 (65 thousand words apart) 11.5 / 11.2, 13.8 / 14.1, 10.2 / 11.8; 256 of
// 400 14.8 / 11.8, 19.2 / 15.7, 14.4 / 12.9; 512 of 127 (66 thousand words for eight) 19.4
// / 13.7, 24.1 / 17.9, 11.0 / 12.2; 1000 of 100 (101 thousand) 46 / 25, 54 / 32, 13.0 / 13.1.
constexpr int kSmallPairs = kScanWarps;
constexpr int64_t kSmallWords = 5 << 14;

// A row is worked on by a CTA, or (kWarp) by each warp of a cluster.
template <bool kWarp>
struct Team {
  static constexpr int kSize = kWarp ? 32 : kRowThreads;
  static __device__ __forceinline__ int rank() { return threadIdx.x & (kSize - 1); }
  static __device__ __forceinline__ bool any(bool x) {
    return kWarp ? __any_sync(0xffffffffu, x) : __syncthreads_or(x);
  }
};

// Whether a later element of rows[0, n) names `row` too (the team asks together).
template <bool kWarp>
__device__ __forceinline__ bool named_later(const int32_t* rows, int i, int n, int row) {
  bool again = false;
#pragma unroll 4
  for (int j = i + 1 + Team<kWarp>::rank(); j < n; j += Team<kWarp>::kSize) again |= rows[j] == row;
  return Team<kWarp>::any(again);
}

// ----------------------------------------------------------------- fork --

// What the launches of a fork hand on, in the workspace.
struct ForkSpace {
  int32_t* head;       // [4] blocks wanted, moves, free blocks
  int32_t* counts;     // [kScanWarps] free blocks of each warp's range
  int32_t* open;       // [n] the block that pair i will write into, -1: none
  int32_t* len;        // [n] the child's length, -1: the pair is passed over
  int32_t* fresh;      // [n] columns to fill behind the length
  int32_t* own;        // [n] 1: gets its own copy of `open`; and twice `fresh`
  int32_t* first;      // [n] its first place in `list`
  int32_t* src;        // [moves]
  int32_t* place;      // [moves] the destination's place in `list`
  int32_t* rows;       // [moves]
  int32_t* list;       // free blocks that are taken, lowest first
  int32_t* stage;      // [n, width] the children's rows
};
__host__ __device__ inline int64_t round4(int64_t n) { return (n + 3) / 4 * 4; }
int64_t list_size(int n, int width, int blocks) {
  const int64_t most = (int64_t)n * (width + 1);
  return most < blocks ? most : blocks;
}
ForkSpace fork_space(void* base, int n, int width, int blocks, int64_t* words) {
  int64_t at = 0;
  auto take = [&](int64_t count) {
    int32_t* p = static_cast<int32_t*>(base) + at;
    at += round4(count);
    return p;
  };
  ForkSpace s{};
  s.head = take(4);
  s.counts = take(kScanWarps);
  s.open = take(n);
  s.len = take(n);
  s.fresh = take(n);
  s.own = take(n);
  s.first = take(n);
  s.src = take(n);
  s.place = take(n);
  s.rows = take(n);
  s.list = take(list_size(n, width, blocks));
  s.stage = take((int64_t)n * width);
  *words = at;
  return s;
}

struct ForkParams {
  Tables t;
  ForkSpace s;
  const int32_t* parents;      // nullptr: the children themselves
  const int32_t* children;
  const int32_t* room;         // nullptr: none
  int32_t* missing;
  int n;
  Carry c;
};

// A pair as the later steps need it (ForkSpace).
struct Pair {
  int open, len, fresh;
};

// Pair i: the child's new row, and the counts of what it lets go and takes.  The loads of
// a step that do not need one another's answers are on their way together; `ready` is
// called before the first count changes.
template <bool kWarp, class Ready>
__device__ __forceinline__ Pair share_pair(const ForkParams& p, int i, Ready ready) {
  using Q = Team<kWarp>;
  constexpr int kAhead = 2;                            // columns of a thread read at once
  const Tables& t = p.t;
  const int tid = Q::rank();
  const int child = p.children[i];
  int parent = p.parents ? p.parents[i] : child;
  const uint32_t room = p.room ? (uint32_t)max(p.room[i], 0) : 0u;
  bool bad = child >= t.rows || parent >= t.rows;
  if (parent >= t.rows) parent = -1;
  const bool in = child >= 0 && child < t.rows;
  const int32_t* old_row = t.table + (int64_t)(in ? child : 0) * t.width;
  const int32_t* new_row = t.table + (int64_t)max(parent, 0) * t.width;
  uint32_t len = parent < 0 ? 0u : (uint32_t)max(t.lens[parent], 0);
  int was[kAhead], now[kAhead];
  auto read = [&](int c0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int c = c0 + k * Q::kSize;
      was[k] = c < t.width ? old_row[c] : -1;
      now[k] = c < t.width ? new_row[c] : -1;
    }
  };
  read(tid);
  const bool again = named_later<kWarp>(p.children, i, p.n, child);
  Pair q{-1, -1, 0};
  if (in && !again) {
    const uint32_t B = (uint32_t)t.block_size;
    if (len > (uint64_t)t.width * B) {
      len = (uint32_t)((uint64_t)t.width * B);
      bad = true;
    }
    const uint32_t part = len % B;                     // positions in the last block, 0: full
    const int have = (int)(len / B) + (part ? 1 : 0);
    const uint32_t slack = part ? B - part : 0u;
    int64_t end = have;
    if (room > slack) end += (room - slack + (B - 1)) / B;
    if (end > t.width) bad = true;
    q.len = (int)len;
    q.fresh = (int)min(end, (int64_t)t.width) - have;
    if (room > 0 && part) {
      q.open = new_row[have - 1];
      if (q.open >= t.blocks) q.open = -1;
    }
    int32_t* stage = p.s.stage + (int64_t)i * t.width;
    ready();
    for (int c0 = tid; c0 < t.width; c0 += kAhead * Q::kSize) {
      if (c0 != tid) read(c0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int c = c0 + k * Q::kSize;
        if (c >= t.width) break;
        int b = c < have ? now[k] : -1;
        if (b >= t.blocks) {
          b = -1;
          bad = true;
        }
        stage[c] = b;
        bad |= was[k] >= t.blocks;
        if (was[k] == b) continue;
        if (was[k] >= 0 && was[k] < t.blocks) atomicSub(t.ref_out + was[k], 1);
        if (b >= 0) atomicAdd(t.ref_out + b, 1);
      }
    }
  } else {
    ready();
  }
  if (tid == 0) {
    p.s.open[i] = q.open;
    p.s.len[i] = q.len;
    p.s.fresh[i] = q.fresh;
  }
  if (bad) bad_index(t.status);
  return q;
}

__global__ void __launch_bounds__(kRowThreads) smla_fork_share_kernel(const ForkParams p) {
  wait_before();
  allow_next();
  share_pair<false>(p, (int)blockIdx.x, [] {});
}

// Inclusive sum over a CTA's threads in two words of one; the total to `all`.
__device__ __forceinline__ long long cta_scan(long long x, long long* sums, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  long long w = sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  all = __shfl_sync(0xffffffffu, w, 31);
  const long long below = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  __syncthreads();                                     // (the sums' room is used again)
  return warp > 0 ? x + below : x;
}

// One cluster: which rows get a copy of their last block, and the free blocks.
// kSmall: the carrying and sharing too, a warp per pair, and each warp counts the pairs
// before its own instead of a scan over all.  What other CTAs of the cluster wrote is
// read past L1.
template <bool kSmall>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads, 1)
smla_fork_take_kernel(const ForkParams p) {
  static_assert(kScanThreads == 1024, "cta_scan: as many warps as lanes");
  wait_before();
  allow_next();
  const Tables& t = p.t;
  const ForkSpace& s = p.s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int id = (int)blockIdx.x * kScanThreads + tid, warp = id >> 5;
  __shared__ long long sums[32];
  Pair mine{-1, -1, 0};                                // pair `warp` (kSmall)
  if constexpr (kSmall) {
    carry(p.c, id, kCluster * kScanThreads);
    // (the counts have to be in place before the first of them changes)
    bool synced = p.c.n[2] == 0;
    auto ready = [&] {
      if (!synced) cluster_sync();
      synced = true;
    };
    if (warp < p.n) mine = share_pair<true>(p, warp, ready);
    ready();
    cluster_sync();
  }
  // A block that is written by some of its holders: of the writers all but the first
  // copy it; where somebody else holds it too, the first as well.
  auto pair_at = [&](int i) {
    if (kSmall && i == warp) return mine;
    return Pair{__ldcg(s.open + i), __ldcg(s.len + i), __ldcg(s.fresh + i)};
  };
  for (int i = warp; i < p.n; i += kScanWarps) {
    const Pair q = pair_at(i);
    int own = 0;
    if (q.open >= 0) {
      const int ref = __ldcg(t.ref_out + q.open);
      int writers = 0, before = 0;
#pragma unroll 8
      for (int j = lane; j < p.n; j += 32) {
        const bool same = __ldcg(s.open + j) == q.open;
        writers += same ? 1 : 0;
        before += same && j < i ? 1 : 0;
      }
      writers = warp_sum(writers);
      own = __any_sync(0xffffffffu, before > 0) || ref > writers ? 1 : 0;
    }
    if (lane == 0) s.own[i] = own | q.fresh << 1;
  }
  const Range range = warp_range(t.blocks, warp);
  const int free_here = count_range(t.ref_out, range, [](int r) { return r == 0; });
  if (lane == 0) s.counts[warp] = free_here;
  cluster_sync();
  // Each pair's place in the list of the blocks taken, and its move's number.
  const int2 base = warp_base(s.counts, warp);
  auto place = [&](int i, int cost, int at, int m) {
    s.first[i] = at;
    if (cost & 1) {
      const Pair q = pair_at(i);
      s.src[m] = q.open;
      s.place[m] = at;
      s.rows[m] = (int)((uint32_t)q.len % (uint32_t)t.block_size);
      // (a block that is copied keeps a holder: its count was above the copies made;
      // a copy that has no block is not made, and its row goes on holding this one)
      if (at < base.y) atomicSub(t.ref_out + q.open, 1);
    }
  };
  int wanted;
  if (kSmall) {
    int blocks = 0, copies = 0, at = 0, m = 0, cost = 0;
#pragma unroll 8
    for (int j = lane; j < p.n; j += 32) {
      const int x = __ldcg(s.own + j), need = (x & 1) + (x >> 1);
      blocks += need;
      copies += x & 1;
      at += j < warp ? need : 0;
      m += j < warp ? x & 1 : 0;
      if (j == warp) cost = x;
    }
    wanted = warp_sum(blocks);
    const int moves = warp_sum(copies);
    if (warp < p.n) {
      at = warp_sum(at);
      m = warp_sum(m);
      cost = warp_sum(cost);
      if (lane == 0) place(warp, cost, at, m);
    }
    if (id == 0) {
      s.head[0] = wanted;
      s.head[1] = moves;
    }
  } else {
    if (blockIdx.x == 0) {
      long long carried = 0;                           // moves << 32 | blocks
      for (int i0 = 0; i0 < p.n; i0 += kScanThreads) {
        const int i = i0 + tid;
        const int x = i < p.n ? __ldcg(s.own + i) : 0;
        const long long y = ((long long)(x & 1) << 32) + (x & 1) + (x >> 1);
        long long all;
        const long long at = carried + cta_scan(y, sums, all) - y;
        carried += all;
        if (i < p.n) place(i, x, (int)(at & 0xffffffffll), (int)(at >> 32));
      }
      if (tid == 0) {
        s.head[0] = (int)(carried & 0xffffffffll);
        s.head[1] = (int)(carried >> 32);
      }
    }
    cluster_sync();
    wanted = __ldcg(s.head);
  }
  int rank = base.x;
  for (int b0 = range.lo; b0 < range.hi && rank < wanted; b0 += 32) {
    const int b = b0 + lane;
    const bool free = b < range.hi && __ldcg(t.ref_out + b) == 0;
    const uint32_t votes = __ballot_sync(0xffffffffu, free);
    const int k = rank + __popc(votes & ((1u << lane) - 1u));
    if (free && k < wanted) {
      s.list[k] = b;
      t.ref_out[b] = 1;
    }
    rank += __popc(votes);
  }
  if (id == 0) {
    s.head[2] = base.y;
    if (p.missing) *p.missing = max(wanted - base.y, 0);
  }
}

// The children's rows, and the rows of the blocks that are copied.
struct ForkWrite {
  ForkParams f;
  CopyParams c;
  int row_ctas;
};
__global__ void __launch_bounds__(kCopyThreads) smla_fork_write_kernel(
    const __grid_constant__ ForkWrite p) {
  wait_before();
  allow_next();
  const int bid = blockIdx.x;
  if (bid >= p.row_ctas) {
    copy_moves(p.c, bid - p.row_ctas,
               ((int)gridDim.x - p.row_ctas) / (p.c.pieces * p.c.layers));
    return;
  }
  const Tables& t = p.f.t;
  const ForkSpace& s = p.f.s;
  const int i = bid, len = s.len[i];
  if (len < 0) return;
  const int child = p.f.children[i];
  const int have = (int)(((uint32_t)len + (uint32_t)(t.block_size - 1)) / (uint32_t)t.block_size);
  const int own = s.own[i] & 1, fresh = s.fresh[i], first = s.first[i];
  const int got = s.head[2];
  const int32_t* stage = s.stage + (int64_t)i * t.width;
  int32_t* row = t.table_out + (int64_t)child * t.width;
  for (int c = threadIdx.x; c < t.width; c += kCopyThreads) {
    int v = stage[c], k = -1;                          // (behind the length: -1)
    if (own && c == have - 1) k = first;
    if (c >= have && c < have + fresh) k = first + own + (c - have);
    if (k >= 0 && k < got) v = s.list[k];
    row[c] = v;
  }
  if (threadIdx.x == 0) t.lens_out[child] = len;
}

// ----------------------------------------------------------------- free --

struct FreeParams {
  Tables t;
  const int32_t* rows;
  const int32_t* begin;        // nullptr: 0
  const int32_t* end;          // nullptr: the table's end
  int n;
};
__global__ void __launch_bounds__(kRowThreads) smla_block_free_kernel(const FreeParams p) {
  wait_before();
  allow_next();
  const Tables& t = p.t;
  const int i = blockIdx.x, row = p.rows[i], tid = threadIdx.x;
  if (row < 0) return;
  if (row >= t.rows) {
    if (tid == 0) bad_index(t.status);
    return;
  }
  if (named_later<false>(p.rows, i, p.n, row)) return;
  const int64_t B = t.block_size;
  const int64_t lo = p.begin ? (max(p.begin[i], 0) + B - 1) / B : 0;
  const int64_t hi = p.end ? min(max(p.end[i], 0) / B, (int64_t)t.width) : t.width;
  int32_t* at = t.table_out + (int64_t)row * t.width;
#pragma unroll 4
  for (int c = (int)min(lo, (int64_t)t.width) + tid; c < hi; c += kRowThreads) {
    const int b = at[c];
    if (b < 0) continue;
    at[c] = -1;
    if (b < t.blocks)
      atomicSub(t.ref_out + b, 1);
    else
      bad_index(t.status);
  }
}
// -------------------------------------------------------------- compact --

struct CompactSpace {
  int32_t* head;       // [4] moves
  int32_t* counts;     // [kScanWarps] live blocks of each warp's range
  int32_t* src;        // [moves]
  int32_t* dst;        // [moves]
};
CompactSpace compact_space(void* base, int blocks, int64_t* words) {
  CompactSpace s{};
  int32_t* p = static_cast<int32_t*>(base);
  const int64_t moves = round4((int64_t)blocks / 2 + 1);
  s.head = p;
  s.counts = p + 4;
  s.src = s.counts + kScanWarps;
  s.dst = s.src + moves;
  *words = 4 + kScanWarps + 2 * moves;
  return s;
}
struct CompactParams {
  Tables t;
  CompactSpace s;
  int32_t* map;        // [blocks] the new number of a live block, -1 for a free one
  int32_t* live;       // [1] or nullptr
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScanThreads, 1)
smla_compact_plan_kernel(const CompactParams p) {
  wait_before();
  allow_next();
  const Tables& t = p.t;
  const int lane = threadIdx.x & 31;
  const int id = (int)blockIdx.x * kScanThreads + (int)threadIdx.x, warp = id >> 5;
  const Range range = warp_range(t.blocks, warp);
  const int mine = count_range(t.ref, range, [](int r) { return r > 0; });
  if (lane == 0) p.s.counts[warp] = mine;
  cluster_sync();
  const int2 base = warp_base(p.s.counts, warp);
  const int live = base.y;
  int below = base.x;                                  // live blocks below b0
  for (int b0 = range.lo; b0 < range.hi; b0 += 32) {
    const int b = b0 + lane;
    const int ref = b < range.hi ? __ldcg(t.ref + b) : 0;
    const uint32_t votes = __ballot_sync(0xffffffffu, ref > 0);
    const int lr = below + __popc(votes & ((1u << lane) - 1u));
    below += __popc(votes);
    if (b >= range.hi) continue;
    if (ref > 0) {
      if (b >= live)
        p.s.src[live - 1 - lr] = b;
      else
        p.map[b] = b;
    } else {
      p.map[b] = -1;
      if (b < live) p.s.dst[b - lr] = b;
    }
    if (b == live) p.s.head[0] = live - lr;            // as many live ones from here on
    // (places that a move writes or empties: below, when all have read their counts)
    if ((ref > 0) == (b < live)) t.ref_out[b] = ref;
  }
  if (id == 0) {
    if (live == t.blocks) p.s.head[0] = 0;
    if (p.live) *p.live = live;
  }
  cluster_sync();
  const int moves = __ldcg(p.s.head);
  for (int k = id; k < moves; k += kCluster * kScanThreads) {
    const int src = __ldcg(p.s.src + k), dst = __ldcg(p.s.dst + k);
    p.map[src] = dst;
    t.ref_out[dst] = __ldcg(t.ref + src);
    t.ref_out[src] = 0;
  }
}

struct CompactWrite {
  CompactParams f;
  CopyParams c;
  int table_ctas;
};
__global__ void __launch_bounds__(kCopyThreads) smla_compact_write_kernel(
    const __grid_constant__ CompactWrite p) {
  wait_before();
  allow_next();
  const int bid = blockIdx.x;
  if (bid >= p.table_ctas) {
    copy_moves(p.c, bid - p.table_ctas,
               ((int)gridDim.x - p.table_ctas) / (p.c.pieces * p.c.layers));
    return;
  }
  const Tables& t = p.f.t;
  const int64_t n = (int64_t)t.rows * t.width;
  const int64_t step = (int64_t)p.table_ctas * kCopyThreads;
  bool bad = false;
#pragma unroll 4
  for (int64_t i = (int64_t)bid * kCopyThreads + threadIdx.x; i < n; i += step) {
    int b = t.table[i];
    if (b >= t.blocks)
      bad = true;                                      // (left as it is)
    else
      b = b < 0 ? -1 : p.f.map[b];
    t.table_out[i] = b;
  }
  if (bad) bad_index(t.status);
}

}  // namespace

cudaError_t launch_block_copy(const Pool& pool, const int32_t* src, const int32_t* dst, int n,
                              int blocks, int* status, cudaStream_t stream) {
  for (int first = 0; first < pool.layers; first += kPoolLayers) {
    CopyParams c = copy_params(pool, first);
    c.src = src;
    c.dst = dst;
    c.n = n;
    c.blocks = blocks;
    c.status = status;
    const cudaError_t e =
        launch_early(smla_block_copy_kernel, copy_ctas(c, n), kCopyThreads, 0, stream, c);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t fork_workspace_bytes(int n, int width, int blocks) {
  int64_t words = 0;
  fork_space(nullptr, n, width, blocks, &words);
  return (size_t)words * 4;
}

cudaError_t launch_fork(const Pool& pool, const Tables& t, const int32_t* parents,
                        const int32_t* children, const int32_t* room, int n, int32_t* missing,
                        void* workspace, cudaStream_t stream) {
  const Carry carried = make_carry(t);
  if (n == 0) {
    const cudaError_t e = launch_carry(carried, stream);
    return e == cudaSuccess && missing ? cudaMemsetAsync(missing, 0, 4, stream) : e;
  }
  int64_t words = 0;
  ForkWrite w{};
  w.f = ForkParams{t, fork_space(workspace, n, t.width, t.blocks, &words), parents, children,
                   room, missing, n, carried};
  cudaError_t e = cudaSuccess;
  if (n <= kSmallPairs && most_of(carried) + (int64_t)n * t.width <= kSmallWords) {
    e = launch_early(smla_fork_take_kernel<true>, kCluster, kScanThreads, 0, stream, w.f);
  } else {
    e = launch_carry(carried, stream);
    if (e == cudaSuccess)
      e = launch_early(smla_fork_share_kernel, (unsigned)n, kRowThreads, 0, stream, w.f);
    if (e == cudaSuccess)
      e = launch_early(smla_fork_take_kernel<false>, kCluster, kScanThreads, 0, stream, w.f);
  }
  for (int first = 0; first < pool.layers && e == cudaSuccess; first += kPoolLayers) {
    w.c = copy_params(pool, first);
    w.c.src = w.f.s.src;
    w.c.dst = w.f.s.place;
    w.c.list = w.f.s.list;
    w.c.list_n = w.f.s.head + 2;
    w.c.rows = w.f.s.rows;
    w.c.n_at = w.f.s.head + 1;
    w.c.blocks = t.blocks;
    w.c.status = t.status;
    w.row_ctas = first == 0 ? n : 0;
    const unsigned ctas = room ? copy_ctas(w.c, n) : 0;
    if (w.row_ctas + ctas > 0)
      e = launch_early(smla_fork_write_kernel, (unsigned)w.row_ctas + ctas, kCopyThreads, 0,
                       stream, w);
  }
  return e;
}

cudaError_t launch_block_free(const Tables& t, const int32_t* rows, const int32_t* begin,
                              const int32_t* end, int n, cudaStream_t stream) {
  cudaError_t e = launch_carry(make_carry(t), stream);
  if (e == cudaSuccess && n > 0)
    e = launch_early(smla_block_free_kernel, (unsigned)n, kRowThreads, 0, stream,
                     FreeParams{t, rows, begin, end, n});
  return e;
}

size_t compact_workspace_bytes(int blocks) {
  int64_t words = 0;
  compact_space(nullptr, blocks, &words);
  return (size_t)words * 4;
}

cudaError_t launch_compact(const Pool& pool, const Tables& t, int32_t* map, int32_t* live,
                           void* workspace, cudaStream_t stream) {
  int64_t words = 0;
  CompactWrite w{};
  w.f = CompactParams{t, compact_space(workspace, t.blocks, &words), map, live};
  cudaError_t e =
      launch_early(smla_compact_plan_kernel, kCluster, kScanThreads, 0, stream, w.f);
  const int64_t entries = (int64_t)t.rows * t.width;
  const int64_t table_ctas = (entries + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
  for (int first = 0; first < pool.layers && e == cudaSuccess; first += kPoolLayers) {
    w.c = copy_params(pool, first);
    w.c.src = w.f.s.src;
    w.c.dst = w.f.s.dst;
    w.c.n_at = w.f.s.head;
    w.c.blocks = t.blocks;
    w.c.status = t.status;
    w.table_ctas = first == 0 ? (int)(table_ctas < 152 * 4 ? table_ctas : 152 * 4) : 0;
    e = launch_early(smla_compact_write_kernel,
                     (unsigned)w.table_ctas + copy_ctas(w.c, t.blocks / 2), kCopyThreads, 0,
                     stream, w);
  }
  return e;
}

}  // namespace smla
