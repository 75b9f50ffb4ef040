// smla_append.cu — append a step's tokens to a paged latent cache, applying
// the rotary position embedding on the way: each token's row
// [kv_c (512) | rope(k_pe) (64)] goes to the cache row of its position, in
// any of the cache formats, and rope(q_pe) to the attention's query.
//
// Mathematics.  A pair (a, b) of rope channels at position p becomes
//   (a cos - b sin, b cos + a sin),  cos/sin = row p of the caller's table,
// (a, b) = channels (2i, 2i + 1) (interleaved) or (i, i + 32), in fp32 with
// every product and sum rounded on its own, so the result is the one that
// separate fp32 operations give; it is rounded once, to the format.
//
// Bound: HBM for a prefill, where the queries' rope part (256 bytes per token
// and head, in and out) is most of the traffic; latency for a decode step
// (the chain start -> length -> table entry and table row -> row).  Measured in a
// captured graph, on two sets of inputs in turn: 8192 tokens with 128 heads into bf16
// rows 48.2 us = 6.0 TB/s, 11 thousand ragged ones with 16 heads into E4M3 blocks
// 18.2 us = 4.9 TB/s (15.8 on one set, most of which stays in L2); 8192 with 16 heads
// into every format 9.5 to 10.6 us for 7.4 to 8.1 of bytes; decode steps of 64 and 128
// requests 2.8 us (bf16) and 3.9 us (E4M3 blocks, whose older rows may follow a
// growing scale).
//
// Work split.  Eight lanes hold one 64-channel vector (16 bytes a lane), four
// vectors a warp, as in smla_cache.cu.  One launch holds two kinds of CTAs:
// the first write cache rows, the others rotate queries, kHeads heads of one
// token per eight lanes so that the position lookup and the cos/sin row are
// read once for them and kHeads loads are in flight (2 heads: 61.6 us, 8: 48.9, 4: 47.7).
// Loads in flight are threads here, so every instance keeps to 64 registers, four
// CTAs an SM (three, of 80 registers: 52.1 us; five spill more, and decode takes 3.2).
#include <cuda_bf16.h>

#include "e4m3_quant.cuh"
#include "paged_batch.cuh"
#include "smla_paged.h"

namespace smla {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 8;    // 8-lane groups per CTA
constexpr int kHeads = 4;                // query heads per group

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    x[2 * p] = __uint_as_float(w[p] << 16);
    x[2 * p + 1] = __uint_as_float(w[p] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * p], x[2 * p + 1]);
    w[p] = *reinterpret_cast<uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 codes8_of(const float (&q)[8]) {
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16),
                    e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

// The cosines and sines that lane j of a group needs: pairs 4j..4j+3
// (interleaved, the first half of c and s) or 8 (j & 3) .. + 7.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ Turn load_turn(const AppendParams& a, int pos) {
  Turn t;
  const int j = threadIdx.x & 7;
  const float* row = a.cos_sin + (int64_t)pos * 64 + (a.interleaved ? 4 * j : 8 * (j & 3));
  const float4* c4 = reinterpret_cast<const float4*>(row);
  const float4* s4 = reinterpret_cast<const float4*>(row + 32);
  const float4 c0 = __ldg(c4), s0 = __ldg(s4);
  float4 c1 = c0, s1 = s0;
  if (!a.interleaved) {
    c1 = __ldg(c4 + 1);
    s1 = __ldg(s4 + 1);
  }
  t.c[0] = c0.x; t.c[1] = c0.y; t.c[2] = c0.z; t.c[3] = c0.w;
  t.c[4] = c1.x; t.c[5] = c1.y; t.c[6] = c1.z; t.c[7] = c1.w;
  t.s[0] = s0.x; t.s[1] = s0.y; t.s[2] = s0.z; t.s[3] = s0.w;
  t.s[4] = s1.x; t.s[5] = s1.y; t.s[6] = s1.z; t.s[7] = s1.w;
  return t;
}

// Lane j's eight channels 8j .. 8j + 7 of a 64-channel vector, rotated.  The
// lanes of the group call it together (the halves form's other channel of a
// pair is in lane j ^ 4).
__device__ __forceinline__ void rotate8(const uint4 raw, const Turn& t, bool interleaved,
                                        float (&y)[8]) {
  float x[8];
  unpack8(raw, x);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      y[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
    }
  } else {
    const uint32_t gmask = 0xFFu << (threadIdx.x & 24);
    uint4 o;
    o.x = __shfl_xor_sync(gmask, raw.x, 4);
    o.y = __shfl_xor_sync(gmask, raw.y, 4);
    o.z = __shfl_xor_sync(gmask, raw.z, 4);
    o.w = __shfl_xor_sync(gmask, raw.w, 4);
    float z[8];
    unpack8(o, z);
    const bool hi = threadIdx.x & 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float own = __fmul_rn(x[i], t.c[i]), other = __fmul_rn(z[i], t.s[i]);
      y[i] = hi ? __fadd_rn(own, other) : __fsub_rn(own, other);
    }
  }
}

// Position of packed token n of request r, and whether its rope row exists
// (a position past the table sets the status).
__device__ __forceinline__ int token_position(const AppendParams& a, int n, int r, bool& bad) {
  if (r < 0) return -1;
  const int pos = batch_len(a.b, r) - batch_start(a.b, r + 1) + n;
  if (pos >= 0 && a.cos_sin && pos >= a.cos_sin_rows) {
    bad = true;
    return -1;
  }
  return pos;
}

// ------------------------------------------------------------- queries --

__device__ __forceinline__ void rotate_queries(const AppendParams& a, int64_t first_group) {
  const int j = threadIdx.x & 7;
  const int64_t g = first_group + (threadIdx.x >> 3);
  const int per = (a.h + kHeads - 1) / kHeads;       // groups per token
  const int n = (int)(g / per), h0 = (int)(g % per) * kHeads;
  if (n >= a.b.N) return;
  uint4 raw[kHeads];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    if (h0 + k < a.h)
      raw[k] = *reinterpret_cast<const uint4*>(a.q_pe + n * a.q_tok + (h0 + k) * a.q_head + 8 * j);
  }
  bool bad = false;
  const int pos = token_position(a, n, batch_request(a.b, n), bad);
  if (bad && j == 0) atomicCAS(a.status, 0, kStatusBadIndex);
  if (pos < 0) return;
  const Turn t = load_turn(a, pos);
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    float y[8];
    rotate8(raw[k], t, a.interleaved, y);
    if (h0 + k < a.h)
      *reinterpret_cast<uint4*>(a.q_out + n * a.qo_tok + (h0 + k) * a.qo_head + 8 * j) = pack8(y);
  }
}

// ---------------------------------------------------------- cache rows --

__device__ __forceinline__ float group_max(float v) {
  const uint32_t gmask = 0xFFu << (threadIdx.x & 24);
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(gmask, v, o));
  return v;
}

// One token's row per eight lanes (every format but one scale per block).
template <int kFmt, bool kRope>
__device__ __forceinline__ void write_row(const AppendParams& a, int n) {
  constexpr int kD = kRope ? 576 : 512;
  const int j = threadIdx.x & 7;
  if (n >= a.b.N) return;
  // The row is read before its place is known.
  uint4 raw[8], pe = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    raw[i] = *(reinterpret_cast<const uint4*>(a.kv_c + n * a.kv_c_stride) + j + 8 * i);
  if (kRope) pe = *(reinterpret_cast<const uint4*>(a.k_pe + n * a.k_pe_stride) + j);
  bool bad = false;
  const int r = batch_request(a.b, n);
  const int pos = token_position(a, n, r, bad);
  int slot = -1;
  if (pos >= 0) {
    const int page = pos / a.b.block_size;
    slot = batch_row(a.b, batch_block(a.b, r, page, bad), pos - page * a.b.block_size, bad);
  }
  if (bad && j == 0) atomicCAS(a.status, 0, kStatusBadIndex);
  if (slot < 0) return;
  float y[8];
  if (kRope) rotate8(pe, load_turn(a, pos), a.interleaved, y);
  uint8_t* cache = static_cast<uint8_t*>(a.cache);
  if (kFmt == kBf16) {
    uint4* row = reinterpret_cast<uint4*>(cache + (int64_t)slot * (2 * kD));
#pragma unroll
    for (int i = 0; i < 8; ++i) row[j + 8 * i] = raw[i];
    if (kRope) row[64 + j] = pack8(y);
    return;
  }
  uint8_t* row = cache + (int64_t)slot * (kFmt == kDsMla ? kDsMlaRowBytes : kD);
  if (kFmt == kE4m3) {
    const float s = __ldg(a.k_scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8(raw[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] / s;
      *reinterpret_cast<uint2*>(row + 8 * (j + 8 * i)) = codes8_of(x);
    }
    if (kRope) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] / s;
      *reinterpret_cast<uint2*>(row + 512 + 8 * j) = codes8_of(y);
    }
    return;
  }
  // Group scales: amax / 448 of each 128 channels (1 for an all-zero group).
  constexpr int kG = kFmt == kE4m3Group && kRope ? 5 : 4;
  float* srow = kFmt == kDsMla ? reinterpret_cast<float*>(row + kDsMlaScaleOff)
                               : a.k_scale + (int64_t)slot * kG;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint64_t xn[2][4];
    float amax = 0.f;
    unpack_neg8(raw[2 * g], xn[0], amax);
    unpack_neg8(raw[2 * g + 1], xn[1], amax);
    amax = group_max(amax);
    const float scale = amax > 0.f ? amax_over_448(amax) : 1.f;
    const float ny = -recip_rn(scale);
    const uint64_t s2 = pack2(scale, scale), ny2 = pack2(ny, ny);
    const bool special = special_scale(scale);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      *reinterpret_cast<uint2*>(row + 8 * (j + 8 * (2 * g + c))) =
          special ? special_codes8(raw[2 * g + c], scale) : codes8(xn[c], s2, ny2);
    if (j == 0) srow[g] = scale;
  }
  if (!kRope) return;
  if (kFmt == kDsMla) {
    // (656-byte rows: 16-byte aligned at byte 528)
    *reinterpret_cast<uint4*>(row + kDsMlaRopeOff + 16 * j) = pack8(y);
    return;
  }
  float scale = a.kpe_scale;                         // kE4m3Group4Kpe
  if (kFmt == kE4m3Group) {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));
    amax = group_max(amax);
    scale = amax > 0.f ? amax / 448.f : 1.f;
    if (j == 0) srow[4] = scale;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = y[e] / scale;
  *reinterpret_cast<uint2*>(row + 512 + 8 * j) = codes8_of(y);
}

// --------------------------------------------- one scale per cache block --

// The smallest power of two s >= 2^-64 with amax <= 448 s.  448 = 1.75 * 2^8:
// with amax = m 2^e, 1 <= m < 2, that is 2^(e - 8) for m <= 1.75 and
// 2^(e - 7) otherwise.  A power of two loses nothing against a finer scale
// (E4M3 is a floating format) and makes a growing scale exact for the rows
// already there, down to E4M3's subnormals.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int k = (int)(u >> 23) - 127 - 8;
  if ((u & 0x7FFFFFu) > 0x600000u) ++k;
  if (amax == 0.f || k < -64) k = -64;
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

// The cache blocks of a request are numbered from floor(start / B) + 2 r on:
// n tokens reach at most floor(n / B) + 2 blocks, so the numbers of the
// requests do not meet, and N / B + 2 R of them hold every block.
__device__ __forceinline__ int64_t first_block_unit(const PagedBatch& b, int r) {
  return batch_start(b, r) / b.block_size + 2ll * r;
}

// One cache block per CTA: the largest |x| of the rows it receives, the
// scale, then the codes.  Older rows keep their codes unless the scale grows.
// Infinities and NaN take no part in the maximum: they become +-448 s and NaN.
// A row is read again for its codes, from L1 or L2: held in registers (128 of them,
// two CTAs an SM) it made the ragged prefill 20.8 us.

template <bool kRope>
__device__ __forceinline__ void write_block(const AppendParams& a, int64_t unit, float* red) {
  constexpr int kD = kRope ? 576 : 512;
  const PagedBatch& b = a.b;
  const int j = threadIdx.x & 7, grp = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int r = warp_last_request(b.num_reqs, unit,
                                  [&](int m) { return first_block_unit(b, m); });
  const int t0 = batch_start(b, r), t1 = batch_start(b, r + 1);
  const int len = batch_len(b, r);
  const int p0 = len - (t1 - t0);                    // position of token t0
  const int64_t page = (int64_t)max(p0, 0) / b.block_size + (unit - first_block_unit(b, r));
  const int64_t low = page * b.block_size;           // the block's first position
  // positions [pa, pb) of the block are written; [low, p0) hold older rows
  const int64_t from = max(low, (int64_t)max(p0, 0));
  int pb = (int)min(low + b.block_size, (int64_t)len);
  if (t1 <= t0 || from >= pb) return;                // (the same for every thread)
  const int pa = (int)from;
  bool bad = false;
  if (kRope && pb > a.cos_sin_rows) {                // positions without a rope row
    bad = true;
    pb = (int)min((int64_t)pb, a.cos_sin_rows);
  }
  const int blk = batch_block(b, r, page, bad);
  // (rows past the cache are not written)
  const int row0 = batch_row(b, blk, 0, bad);
  if (row0 >= 0 && row0 + (pb - 1 - low) >= b.num_slots) {
    bad = true;
    pb = (int)(low + b.num_slots - row0);
  }
  if (bad && threadIdx.x == 0) atomicCAS(a.status, 0, kStatusBadIndex);
  if (row0 < 0 || pa >= pb) return;
  const int64_t base = row0 - low;                   // cache row of position p: base + p

  // (i: rows from pa on; pa + i ends below pb, so it holds every position)
  const int rows = pb - pa;
  auto load_row = [&](int p, uint4 (&raw)[9]) {
    const int64_t n = t0 + (p - p0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      raw[i] = *(reinterpret_cast<const uint4*>(a.kv_c + n * a.kv_c_stride) + j + 8 * i);
    if (kRope) raw[8] = *(reinterpret_cast<const uint4*>(a.k_pe + n * a.k_pe_stride) + j);
  };
  auto fold = [&](const float (&x)[8], float m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = fabsf(x[e]);
      m = v < INFINITY ? fmaxf(m, v) : m;
    }
    return m;
  };
  float amax = 0.f;
  auto row_max = [&](const uint4 (&raw)[9], int p, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8(raw[i], x);
      amax = fold(x, amax);
    }
    if (kRope) {
      rotate8(raw[8], load_turn(a, p), a.interleaved, y);
      amax = fold(y, amax);
    }
  };
  for (int i = grp; i < rows; i += kGroups) {
    const int p = pa + i;
    uint4 raw[9];
    float y[8];
    load_row(p, raw);
    row_max(raw, p, y);
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[warp] = amax;
  float* scale_at = a.k_scale + blk;
  const bool kept = p0 > low;                        // older rows in the block
  const float old = kept ? *scale_at : 0.f;
  __syncthreads();                                   // (old is read before it is replaced)
  amax = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const float scale = fmaxf(block_scale(amax), old);
  const float inv = 1.f / scale;
  if (threadIdx.x == 0) *scale_at = scale;
  uint8_t* cache = static_cast<uint8_t*>(a.cache);
  auto store_row = [&](const uint4 (&raw)[9], int p, float (&y)[8]) {
    uint8_t* row = cache + (base + p) * kD;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x[8];
      unpack8(raw[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= inv;
      *reinterpret_cast<uint2*>(row + 8 * (j + 8 * i)) = codes8_of(x);
    }
    if (kRope) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= inv;
      *reinterpret_cast<uint2*>(row + 512 + 8 * j) = codes8_of(y);
    }
  };
  for (int i = grp; i < rows; i += kGroups) {
    const int p = pa + i;
    uint4 raw[9];
    float y[8];
    load_row(p, raw);
    if (kRope) rotate8(raw[8], load_turn(a, p), a.interleaved, y);
    store_row(raw, p, y);
  }
  if (kept && scale > old) {                         // older rows follow the scale
    const float ratio = old / scale;                 // (from a zero one: they stay zero)
    uint2* codes = reinterpret_cast<uint2*>(cache + (base + low) * kD);
    const int64_t n8 = (int64_t)(p0 - low) * (kD / 8);
    for (int64_t i = threadIdx.x; i < n8; i += kThreads) {
      const uint2 c = codes[i];
      float x[8];
      e4m3x4_to_f32(c.x, x[0], x[1], x[2], x[3]);
      e4m3x4_to_f32(c.y, x[4], x[5], x[6], x[7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= ratio;
      codes[i] = codes8_of(x);
    }
  }
}

template <int kFmt, bool kRope>
__global__ void __launch_bounds__(kThreads, 4) smla_append_kernel(const AppendParams a) {
  __shared__ float red[kThreads / 32];
  const int64_t bid = blockIdx.x;
  if (bid >= a.row_ctas) {
    if (kRope) rotate_queries(a, (bid - a.row_ctas) * kGroups);
  } else if (kFmt == kE4m3Block) {
    write_block<kRope>(a, bid, red);
  } else {
    write_row<kFmt, kRope>(a, (int)(bid * kGroups) + (int)(threadIdx.x >> 3));
  }
}

template <int kFmt>
cudaError_t launch_fmt(const AppendParams& a, unsigned ctas, bool rope, cudaStream_t stream) {
  constexpr bool kAlways = kFmt == kDsMla || kFmt == kE4m3Group4Kpe;   // 576-channel formats
  if (kAlways || rope)
    smla_append_kernel<kFmt, true><<<ctas, kThreads, 0, stream>>>(a);
  else if constexpr (!kAlways)
    smla_append_kernel<kFmt, false><<<ctas, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(AppendParams a, int kv_format, bool rope, cudaStream_t stream) {
  a.row_ctas = kv_format == kE4m3Block
                   ? (int64_t)a.b.N / a.b.block_size + 2ll * a.b.num_reqs
                   : ((int64_t)a.b.N + kGroups - 1) / kGroups;
  const int64_t groups = a.q_pe ? (int64_t)a.b.N * ((a.h + kHeads - 1) / kHeads) : 0;
  const int64_t ctas = a.row_ctas + (groups + kGroups - 1) / kGroups;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  switch (kv_format) {
    case kBf16: return launch_fmt<kBf16>(a, (unsigned)ctas, rope, stream);
    case kE4m3: return launch_fmt<kE4m3>(a, (unsigned)ctas, rope, stream);
    case kE4m3Group: return launch_fmt<kE4m3Group>(a, (unsigned)ctas, rope, stream);
    case kDsMla: return launch_fmt<kDsMla>(a, (unsigned)ctas, rope, stream);
    case kE4m3Group4Kpe: return launch_fmt<kE4m3Group4Kpe>(a, (unsigned)ctas, rope, stream);
    default: return launch_fmt<kE4m3Block>(a, (unsigned)ctas, rope, stream);
  }
}

}  // namespace smla
