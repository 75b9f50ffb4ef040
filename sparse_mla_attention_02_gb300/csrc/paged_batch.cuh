// paged_batch.cuh — a ragged batch over a paged cache as the append and the
// windowed attention take it, and the device lookups on it.
//
// Request r owns the packed tokens [query_start[r], query_start[r + 1]) and,
// with them, seq_lens[r] positions: its token i is at position
// seq_lens[r] - n_r + i.  Position e sits in cache row
// block_table[r][e / block_size] * block_stride_rows + e % block_size.
// Every value is device data, so nothing here trusts it: starts are clamped
// to [0, N], table columns and rows are checked before they are used.
#pragma once

#include "smla_paged.h"

namespace smla {

// Descriptors and scales: coherent loads, kept behind a griddepcontrol.wait that
// stands before them.  A kernel launched under the end of the one that writes them
// (the windowed attention) must not read them through the read-only path, which
// takes them for constant during its whole life.
__device__ __forceinline__ int ld_batch(const int32_t* at) {
  int v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(at));
  return v;
}
__device__ __forceinline__ float ld_batch(const float* at) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(at));
  return v;
}

__device__ __forceinline__ int batch_start(const PagedBatch& b, int r) {
  return min(max(ld_batch(b.query_start + r), 0), b.N);
}

// Length of request r (a negative one is 0, so that no position wraps round).
__device__ __forceinline__ int batch_len(const PagedBatch& b, int r) {
  return max(ld_batch(b.seq_lens + r), 0);
}

// Row of block `blk` (an entry of the table) plus `off`, or -1 when the block
// is not allocated (blk < 0) or the row lies past the cache (sets *bad).
__device__ __forceinline__ int batch_row(const PagedBatch& b, int blk, int off, bool& bad) {
  if (blk < 0) return -1;
  const int64_t row = (int64_t)blk * b.block_stride_rows + off;
  if (row >= b.num_slots) {
    bad = true;
    return -1;
  }
  return (int)row;
}

// The table's entry for column `page` of request r; -1 past the table (sets
// *bad).
__device__ __forceinline__ int batch_block(const PagedBatch& b, int r, int64_t page, bool& bad) {
  if (page >= b.bt_stride) {
    bad = true;
    return -1;
  }
  return ld_batch(b.block_table + (int64_t)r * b.bt_stride + page);
}

// The request of packed token n, or -1 behind the last request; the eight
// lanes of a group ask for the same token.  The first guess (request n, the
// decode step's answer) costs one latency; otherwise each step reads eight
// starts and keeps a ninth of the range.
__device__ __forceinline__ int batch_request(const PagedBatch& b, int n) {
  const int lane8 = threadIdx.x & 7;
  const int sh = threadIdx.x & 24;                   // the group's first lane
  const uint32_t gmask = 0xFFu << sh;
  const int guess = min(n, b.num_reqs - 1);
  if (batch_start(b, guess) <= n && n < batch_start(b, guess + 1)) return guess;
  int lo = 0, hi = b.num_reqs;
  while (hi - lo > 1) {
    const int m = lo + (int)((int64_t)(hi - lo) * (lane8 + 1) / 9);
    const uint32_t le = (__ballot_sync(gmask, batch_start(b, m) <= n) >> sh) & 0xFFu;
    const int c = __ffs(~le) - 1;                    // leading probes at or below n
    const int64_t w = hi - lo;
    const int base = lo;
    if (c > 0) lo = base + (int)(w * c / 9);
    if (c < 8) hi = base + (int)(w * (c + 1) / 9);
  }
  return batch_start(b, lo) <= n && n < batch_start(b, lo + 1) ? lo : -1;
}

// The last request r with first(r) <= u, for a non-decreasing `first`; the
// 32 lanes of a warp ask together and keep a 33rd of the range per step.
template <class First>
__device__ __forceinline__ int warp_last_request(int num_reqs, int64_t u, First first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_reqs;
  while (hi - lo > 1) {
    const int64_t w = hi - lo;
    const int base = lo;
    const int m = base + (int)(w * (lane + 1) / 33);
    const uint32_t le = __ballot_sync(0xffffffffu, first(m) <= u);
    const int c = le == 0xffffffffu ? 32 : __ffs(~le) - 1;
    if (c > 0) lo = base + (int)(w * c / 33);
    if (c < 32) hi = base + (int)(w * (c + 1) / 33);
  }
  return lo;
}

}  // namespace smla
