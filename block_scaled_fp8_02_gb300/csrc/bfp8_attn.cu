// bfp8_attn.cu -- attention of new tokens over the paged e4m3 cache: the C
// entry points, and which kernel takes which sequences.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bfp8_attn.cuh"
#include "bfp8_internal.h"

namespace bfp8 {

namespace {

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

// Rows a kv head up to which the kernel for few rows takes a sequence: what its registers hold.  16 sequences at
// 8192, 64 / 8 heads of 128: 100 us with 32 rows there, 118 with 40 in the other, whose 128-row tiles
// cost the same from 33 rows to 128.
constexpr int kFewRows = 32;

bfp8_status check_heads(int heads, int kv_heads, int dim, int max_q) {
  if (kv_heads < 1 || heads < kv_heads || heads > 65535 || heads % kv_heads != 0)
    return bad("num_heads = %d is not a multiple of num_kv_heads = %d (at most 65535)", heads, kv_heads);
  if (heads / kv_heads > 128) return bad("%d query heads a kv head (at most 128)", heads / kv_heads);
  if (dim != 64 && dim != 128) return bad("head_dim = %d (expected 64 or 128)", dim);
  if (max_q < 1 || max_q > (1 << 24)) return bad("max_q_len = %d (expected 1 .. 2^24)", max_q);
  return BFP8_OK;
}

// Rows of a sequence up to which the kernel for few rows takes it, as a count
// of eights: all sequences when even the longest is that short, else those of
// a single token (a batch of chunks and decoding sequences).
int few_groups(int group, int64_t max_q) {
  return attn_decode_groups(max_q * group <= kFewRows ? max_q * group : group);
}

bool has_many(int group, int max_q) {
  return group > kFewRows || static_cast<int64_t>(max_q) * group > 8 * few_groups(group, max_q);
}

size_t few_bytes(int group, int dim, int max_q, int sms) {
  return (attn_decode_partial_bytes(few_groups(group, max_q), dim, sms) + 255) / 256 * 256;
}

// Counter header, partial rows of the kernel for few rows, those of the other.
size_t workspace_bytes_for(int group, int dim, int max_q, int sms) {
  return kCounterHeaderBytes + few_bytes(group, dim, max_q, sms) +
         (has_many(group, max_q) ? attn_tile_partial_bytes(dim, sms) : 0);
}

}  // namespace

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_paged_attention_workspace_size(int num_heads, int num_kv_heads,
                                                           int head_dim, int max_q_len,
                                                           size_t* bytes) {
  bfp8_status st = check_heads(num_heads, num_kv_heads, head_dim, max_q_len);
  if (st != BFP8_OK) return st;
  if (!bytes) return bad("bytes is null");
  int sms = 0;
  int* err = nullptr;
  if ((st = device_for_call(&sms, &err)) != BFP8_OK) return st;
  *bytes = workspace_bytes_for(num_heads / num_kv_heads, head_dim, max_q_len, sms);
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_paged_attention(const bfp8_attention_args* p, const bfp8_kv_cache* cache,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  AttnArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  if (!p) return bad("args is null");
  // an empty call's bounds may be zero
  const bool empty = p->batch == 0 || p->total_q == 0;
  if ((st = check_heads(p->num_heads, a.c.heads, a.c.dim, empty && p->max_q_len == 0 ? 1 : p->max_q_len)) != BFP8_OK)
    return st;
  if (p->batch < 0 || p->batch > 65535 || p->total_q < 0 || p->total_q >= (int64_t{1} << 31))
    return bad("batch = %d, total_q = %lld", p->batch, (long long)p->total_q);
  if (p->max_pages < (empty ? 0 : 1) || p->ld_table < p->max_pages)
    return bad("max_pages = %d, ld_table = %lld", p->max_pages, (long long)p->ld_table);
  if (p->max_kv_len < 0 || p->max_kv_len > (int64_t{1} << 30))
    return bad("max_kv_len = %lld (expected 0 .. 2^30)", (long long)p->max_kv_len);
  if (p->max_kv_len > static_cast<int64_t>(p->max_pages) * a.c.page_size)
    return bad("max_kv_len = %lld exceeds max_pages * page_size", (long long)p->max_kv_len);
  if (!std::isfinite(p->softmax_scale)) return bad("softmax_scale is not finite");
  if (p->causal != 0 && p->causal != 1) return bad("causal = %d (expected 0 or 1)", p->causal);
  if (p->window < 0) return bad("window = %d (expected >= 0)", p->window);
  if (empty) return set_last_error(BFP8_OK, "");
  if (!p->q || !p->out || !p->block_table || !p->cu_q || !p->kv_lens)
    return bad("null pointer (q=%p out=%p block_table=%p cu_q=%p kv_lens=%p)", p->q, p->out,
               (const void*)p->block_table, (const void*)p->cu_q, (const void*)p->kv_lens);
  for (int64_t s : {p->q_stride_token, p->q_stride_head, p->out_stride_token, p->out_stride_head})
    if (s < 0) return bad("negative stride %lld", (long long)s);
  if (p->out_stride_head < a.c.dim || p->out_stride_token < a.c.dim)
    return bad("out strides must be >= head_dim");
  for (int64_t s : {p->q_stride_token, p->q_stride_head, p->out_stride_token, p->out_stride_head})
    if (s % 8) return set_last_errorf(BFP8_ERR_ALIGNMENT, "q and out strides must be multiples of 8 elements");
  if (off_align(p->q, 16) || off_align(p->out, 16) || off_align(p->lse, 4) || off_align(p->block_table, 4) ||
      off_align(p->cu_q, 4) || off_align(p->kv_lens, 4))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "q and out must be 16-byte aligned, the rest 4-byte");
  int sms = 0;
  if ((st = device_for_call(&sms, &a.err)) != BFP8_OK) {
    // a host without a device still learns of a missing workspace
    if (!workspace || workspace_bytes < kCounterHeaderBytes || off_align(workspace, 256))
      return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace missing, too small or not 256-byte aligned");
    return st;
  }
  a.group = p->num_heads / a.c.heads;
  const size_t need = workspace_bytes_for(a.group, a.c.dim, p->max_q_len, sms);
  if (!workspace || workspace_bytes < need)
    return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (off_align(workspace, 256)) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  a.q = static_cast<const __nv_bfloat16*>(p->q);
  a.out = static_cast<__nv_bfloat16*>(p->out);
  a.lse = p->lse;
  a.q_st = p->q_stride_token;
  a.q_sh = p->q_stride_head;
  a.o_st = p->out_stride_token;
  a.o_sh = p->out_stride_head;
  a.table = p->block_table;
  a.ld_table = p->ld_table;
  a.cu_q = p->cu_q;
  a.kv_lens = p->kv_lens;
  a.total_q = p->total_q;
  a.max_kv = p->max_kv_len;
  a.heads = p->num_heads;
  a.batch = p->batch;
  a.max_q = p->max_q_len;
  a.causal = p->causal;
  // A window past every distance hides nothing.  Positions begin at -max_q_len (more new tokens than context), so
  // without this p - window + 1 would leave 32 bits for the widest windows.
  a.window = p->window > p->max_kv_len + p->max_q_len ? 0 : p->window;
  a.scale = p->softmax_scale;
  const int groups = few_groups(a.group, p->max_q_len);
  a.few_rows = groups * 8;
  const uint64_t dims[4] = {static_cast<uint64_t>(a.c.dim), static_cast<uint64_t>(a.c.page_size),
                            static_cast<uint64_t>(a.c.heads), static_cast<uint64_t>(a.c.num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(a.c.st_tok), static_cast<uint64_t>(a.c.st_head),
                               static_cast<uint64_t>(a.c.st_page)};
  const uint32_t box[4] = {static_cast<uint32_t>(a.c.dim),
                           static_cast<uint32_t>(a.c.page_size < 128 ? a.c.page_size : 128), 1u, 1u};
  CUtensorMap mk, mv;
  if ((st = encode_bytes_tiled(&mk, a.c.k, 4, dims, strides, box, a.c.dim)) != BFP8_OK) return st;
  if ((st = encode_bytes_tiled(&mv, a.c.v, 4, dims, strides, box, a.c.dim)) != BFP8_OK) return st;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t* counters = static_cast<int32_t*>(workspace);
  char* partials = static_cast<char*>(workspace) + kCounterHeaderBytes;
  cudaError_t e = cudaSuccess;
  // Can a sequence be short enough for the kernel for few rows?  Not if the others at their longest leave this
  // one too many tokens (always so for a single chunk): then its launch is saved.
  const bool many = has_many(a.group, p->max_q_len);
  const bool few = a.group <= kFewRows &&
                   (!many || p->total_q <= static_cast<int64_t>(p->batch - 1) * p->max_q_len + a.few_rows / a.group);
  if (!few) a.few_rows = 0;
  if (many)
    e = launch_attn_tile(mk, mv, a, sms, counters + sms,
                         reinterpret_cast<float*>(partials + few_bytes(a.group, a.c.dim, p->max_q_len, sms)), cs);
  if (e == cudaSuccess && few)
    e = launch_attn_decode(mk, mv, a, groups, sms, counters, reinterpret_cast<float*>(partials), many, cs);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
