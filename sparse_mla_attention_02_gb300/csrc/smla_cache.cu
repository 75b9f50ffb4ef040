// smla_cache.cu — group-quantizing E4M3 cache write.
//
// The flashinfer_mla_sparse_sm90.py page reads E4M3 caches with one fp32
// scale per (slot, 128-channel group) (its ckv_scale_arr layout) and notes
// that the cache-write op producing that layout is missing; vLLM's
// concat_and_cache_mla (same pages) is the write for the other formats: a
// token's row [kv_c (512) | k_pe (64)] goes to the cache row at its slot.
// This kernel is that write for the group format:
//   for each written row and group g (channels [128 g, 128 g + 128)):
//     scale = amax|x| / 448 in fp32 (1 for an all-zero group),
//     code  = e4m3(x / scale), fp32 division, round to nearest even,
//             saturating at +-448 (the satfinite conversion).
// HBM-bound: per row 2 * d_qk bytes read, d_qk + 4 * G written.
//
// Eight lanes per token row, four rows per warp.  A row is 64 (d_qk 512) or
// 72 (576) chunks of 8 channels; lane j of the row's eight converts chunks
// j + 8 i, i < 8 or 9 (all of its loads issued first), so that group g is
// chunks i = 2g, 2g + 1 of all eight lanes (the rope group, i = 8, alone):
// the group max is a shuffle reduction over the eight lanes.
//
// The kernel is bound by instruction issue as much as by HBM, so the fp32
// quotients take no division: each is the IEEE quotient x / scale, reached
// by one multiply and two fused multiply-adds (Markstein's correction of
// x * RN(1/scale)), in packed f32x2 arithmetic.
#include <cuda_bf16.h>

#include "e4m3_quant.cuh"
#include "smla_internal.h"

namespace smla {
namespace {

struct CacheArgs {
  const uint16_t* kv_c;   // bf16 [N, 512]
  const uint16_t* k_pe;   // bf16 [N, d_qk - 512] or nullptr (d_qk 512)
  const int32_t* slot;    // [N]
  uint8_t* cache;         // [num_slots, d_qk]
  float* scales;          // [num_slots, G]
  int* status;
  int64_t num_slots;
  int N;
};

// kChunks = d_qk / 64: 9 (kv_c + rope) or 8 (kv_c only).
template <int kChunks>
__global__ void __launch_bounds__(256) smla_cache_write_kernel(const CacheArgs a) {
  constexpr int kD = 8 * 8 * kChunks;                // d_qk
  constexpr int kG = (kChunks + 1) / 2;              // groups
  const int j = threadIdx.x & 7;                     // lane within the row's eight
  const int n = (int)((blockIdx.x * 256u + threadIdx.x) >> 3);
  int s = n < a.N ? __ldg(a.slot + n) : -1;
  if (s >= a.num_slots) {
    if (j == 0) atomicCAS(a.status, 0, kStatusBadIndex);
    s = -1;
  }
  const bool ok = s >= 0;
  // chunk i of this lane: channel 8 (j + 8 i)
  auto src = [&](int i) {
    return i < 8 ? reinterpret_cast<const uint4*>(a.kv_c + (int64_t)n * 512) + j + 8 * i
                 : reinterpret_cast<const uint4*>(a.k_pe + (int64_t)n * 64) + j;
  };
  uint4 raw[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (ok) raw[i] = __ldg(src(i));
  }
  uint8_t* row = a.cache + (int64_t)s * kD;
  float* srow = a.scales + (int64_t)s * kG;
  uint32_t special = 0;                              // groups with a special scale
  float scale_g[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    const int i0 = 2 * g, nc = (2 * g + 1 < kChunks) ? 2 : 1;
    uint64_t xn[2][4];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < nc; ++c) unpack_neg8(raw[i0 + c], xn[c], amax);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = amax > 0.f ? amax_over_448(amax) : 1.f;
    scale_g[g] = scale;
    special |= special_scale(scale) ? 1u << g : 0u;
    const float ny = -recip_rn(scale);
    const uint64_t s2 = pack2(scale, scale), ny2 = pack2(ny, ny);
    if (ok) {
#pragma unroll
      for (int c = 0; c < nc; ++c)
        *reinterpret_cast<uint2*>(row + 8 * (j + 8 * (i0 + c))) = codes8(xn[c], s2, ny2);
      if (j == 0) srow[g] = scale;
    }
  }
  if (ok && special) {                               // rare: redo the special groups
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if (!(special >> g & 1u)) continue;
      for (int i = 2 * g; i < 2 * g + 2 && i < kChunks; ++i)
        *reinterpret_cast<uint2*>(row + 8 * (j + 8 * i)) = special_codes8(__ldg(src(i)), scale_g[g]);
    }
  }
}

}  // namespace

cudaError_t launch_cache_write(const void* kv_c, const void* k_pe, const int32_t* slot,
                               int N, int d_qk, int64_t num_slots, void* cache,
                               float* scales, int* status, cudaStream_t stream) {
  CacheArgs a{};
  a.kv_c = static_cast<const uint16_t*>(kv_c);
  a.k_pe = static_cast<const uint16_t*>(k_pe);
  a.slot = slot;
  a.cache = static_cast<uint8_t*>(cache);
  a.scales = scales;
  a.status = status;
  a.num_slots = num_slots;
  a.N = N;
  const unsigned blocks = (unsigned)(((int64_t)N * 8 + 255) / 256);
  if (d_qk == 576)
    smla_cache_write_kernel<9><<<blocks, 256, 0, stream>>>(a);
  else
    smla_cache_write_kernel<8><<<blocks, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace smla
