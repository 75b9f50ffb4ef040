// smla_paged.h — host side of the append and the windowed attention.
#pragma once

#include "smla_internal.h"

namespace smla {

// Cache format beside those of KvFormat: E4M3 [num_slots, d_qk] with one fp32
// scale per cache block.
constexpr int kE4m3Block = 5;

// A ragged batch of N packed tokens over a paged cache (see paged_batch.cuh).
struct PagedBatch {
  const int32_t* query_start;  // [num_reqs + 1]
  const int32_t* seq_lens;     // [num_reqs]
  const int32_t* block_table;  // [num_reqs, bt_stride]
  int num_reqs, bt_stride, block_size, block_stride_rows;
  int N;                       // packed tokens
  int64_t num_slots;           // rows in the cache
};

// An append (smla_append.cu).  Strides are in elements.
struct AppendParams {
  PagedBatch b;
  const uint16_t* kv_c;        // bf16 [N, 512]
  const uint16_t* k_pe;        // bf16 [N, 64], or nullptr (d_qk 512)
  int64_t kv_c_stride, k_pe_stride;
  const float* cos_sin;        // [cos_sin_rows, 64] = cos 32 | sin 32, or nullptr (d_qk 512)
  int64_t cos_sin_rows;
  int interleaved;
  const uint16_t* q_pe;        // bf16 [N, h, 64], or nullptr
  uint16_t* q_out;
  int64_t q_tok, q_head, qo_tok, qo_head;
  int h;
  void* cache;
  float* k_scale;
  float kpe_scale;
  int* status;
  int64_t row_ctas;            // CTAs that write cache rows (set by launch_append)
};

// A windowed attention (smla_tc_win.cu).
struct WinParams {
  PagedBatch b;
  const void* q;               // bf16 [N, h, d_qk]
  const void* kv;              // [num_slots, d_qk] bf16 or E4M3
  const float* k_scale;        // E4M3: [1] or one per cache block
  void* out;                   // bf16 [N, h, 512]
  float* lse;                  // [N, h] or nullptr
  // workers > 0: the key blocks of all tiles are cut into that many ranges, and
  // tiles in parts leave partials: two per range, of up to 128 rows
  int workers;
  float* o_part;               // [2 workers, 128, 512]
  float* lse_part;             // [2 workers, 128]
  int* parts;                  // [N, h] the ranges that hold the row's tile, its row
  int merge_groups;            // thread groups of the merge
  int* status;
  int* abort_ctr;
  uint64_t wait_limit_ns;
  int inject_stall;            // see FwdParams
  int kv_format, h, d_qk;
  int window, sinks;           // window 0: every position up to the token's own
  int64_t num_tiles;           // set by launch_window
  int table_end;               // the last position a block table can hold (launch_window)
  float sm_scale;
};

struct WindowPlan {
  int64_t tiles;
  int workers, merge_groups;
  size_t workspace_bytes;
};
WindowPlan make_window_plan(int T, int h, int num_reqs, int64_t max_len, int window, int sinks,
                            int num_sms);
cudaError_t launch_window(WinParams p, cudaStream_t stream);

cudaError_t launch_append(AppendParams a, int kv_format, bool rope, cudaStream_t stream);

}  // namespace smla
