// smla_blocks.h — host side of the block operators on a paged cache (copying,
// forking, giving back and compacting blocks).
#pragma once

#include "smla_paged.h"

namespace smla {

// The caches of several layers, all of one layout: a block table is the same in
// every layer.  They go to a kernel by value, kPoolLayers of them a launch.
constexpr int kPoolLayers = 128;
struct Pool {
  void* const* cache;          // host arrays, one device pointer a layer
  float* const* scale;         // nullptr: no scale belongs to a block
  int layers;
  int row_bytes;
  int groups;                  // fp32 scales of a row; -1: one per block; 0: none
  int block_size, block_stride_rows;
};

// Block tables and counts, before and after (the same arrays: in place).
struct Tables {
  const int32_t* table;        // [rows, width]
  int32_t* table_out;
  const int32_t* lens;         // [rows] (fork)
  int32_t* lens_out;
  const int32_t* ref;          // [blocks] table entries that hold the block
  int32_t* ref_out;
  int rows, width, blocks;
  int block_size;
  int* status;
};

cudaError_t launch_block_copy(const Pool& pool, const int32_t* src, const int32_t* dst, int n,
                              int blocks, int* status, cudaStream_t stream);

size_t fork_workspace_bytes(int n, int width, int blocks);
cudaError_t launch_fork(const Pool& pool, const Tables& t, const int32_t* parents,
                        const int32_t* children, const int32_t* room, int n, int32_t* missing,
                        void* workspace, cudaStream_t stream);

cudaError_t launch_block_free(const Tables& t, const int32_t* rows, const int32_t* begin,
                              const int32_t* end, int n, cudaStream_t stream);

size_t compact_workspace_bytes(int blocks);
cudaError_t launch_compact(const Pool& pool, const Tables& t, int32_t* map, int32_t* live,
                           void* workspace, cudaStream_t stream);

}  // namespace smla
