// bfp8_attn.cuh -- what the attention kernels share: their arguments and the
// lengths of a sequence as they stand on the device.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_kvcache.cuh"

namespace bfp8 {

struct AttnArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;                   // or nullptr
  int64_t q_st, q_sh, o_st, o_sh;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  int64_t total_q;
  int64_t max_kv;               // bound of kv_lens: host bound and table width
  int32_t heads, group;         // query heads, query heads a kv head
  int32_t batch;
  int32_t max_q;
  int32_t causal;
  int32_t window;               // 0: none; at most max_kv + max_q
  int32_t few_rows;             // sequences of at most this many rows (new tokens x group) go to the kernel for few
  float scale;
  CacheView c;
  int* err;
};

// Sequence b: its rows of q and its context, clamped to the bounds, so that no
// length can lead out of a buffer.
struct SeqLens {
  int64_t row0;
  int32_t q_len;
  int32_t kv_len;
};
__device__ __forceinline__ SeqLens seq_lens(const AttnArgs& a, int b) {
  SeqLens s;
  int64_t c0 = a.cu_q[b], c1 = a.cu_q[b + 1];
  c0 = c0 < 0 ? 0 : c0 > a.total_q ? a.total_q : c0;
  c1 = c1 < c0 ? c0 : c1 > a.total_q ? a.total_q : c1;
  s.row0 = c0;
  s.q_len = static_cast<int32_t>(c1 - c0 < a.max_q ? c1 - c0 : a.max_q);
  const int64_t n = a.kv_lens[b];
  s.kv_len = static_cast<int32_t>(n < 0 ? 0 : n < a.max_kv ? n : a.max_kv);
  return s;
}

// Tokens [lo, hi) that the new token at position p sees (p >= -max_q, window <= max_kv + max_q < 2^31 - max_q).
__device__ __forceinline__ void seen_range(const AttnArgs& a, int32_t kv_len, int32_t p, int32_t& lo,
                                           int32_t& hi) {
  hi = a.causal ? p + 1 : kv_len;
  lo = a.window > 0 ? p - a.window + 1 : 0;
  if (lo < 0) lo = 0;
  if (hi > kv_len) hi = kv_len;
}

// A line of `total` units shared equally by `ctas` CTAs: where share c begins,
// and whose share unit u is in.  32-bit division (a tenth of the time) where the
// products fit.
__device__ __forceinline__ int64_t share_begin(int64_t c, int64_t total, int64_t ctas) {
  if (total < (1 << 22) && ctas < (1 << 10))
    return static_cast<uint32_t>(c) * static_cast<uint32_t>(total) / static_cast<uint32_t>(ctas);
  return c * total / ctas;
}
__device__ __forceinline__ int share_of(int64_t u, int64_t total, int64_t ctas) {
  if (total < (1 << 22) && ctas < (1 << 10))
    return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(ctas) - 1u) / static_cast<uint32_t>(total));
  return static_cast<int>(((u + 1) * ctas - 1) / total);
}

// The kernel for few rows a sequence (bfp8_attn_decode.cu): `groups` (1 to 4)
// eights of rows, `ctas` persistent CTAs, counters[ctas] zero.
// k, v: tensor maps [dim, token, head, page] of bytes, boxes of min(page_size, 128) tokens.
// behind: the launch before it in the stream is launch_attn_tile's of the same call; the two run beside each other.
int attn_decode_groups(int64_t rows);
size_t attn_decode_partial_bytes(int groups, int dim, int ctas);
cudaError_t launch_attn_decode(const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int groups, int ctas,
                               int32_t* counters, float* partials, bool behind, cudaStream_t stream);

// The kernel for more rows (bfp8_attn_tile.cu); counters[2 * ctas] zero.
size_t attn_tile_partial_bytes(int dim, int ctas);
cudaError_t launch_attn_tile(const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int ctas, int32_t* counters,
                             float* partials, cudaStream_t stream);

}  // namespace bfp8
