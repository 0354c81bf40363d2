// bfp8_attn.cu -- attention of new tokens over the paged e4m3 cache: the C
// entry points and a kernel of one warp per (token, query head).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bfp8_attn.cuh"
#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"
#include "bfp8_vec8.cuh"

namespace bfp8 {

namespace {

// One warp a row (token, head): lanes hold D / 32 elements each, one pass over
// the tokens with the running maximum and sum of the softmax.
template <int D>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z;
  const int head = blockIdx.y;
  const int kvh = head / a.group;
  const SeqLens sl = seq_lens(a, b);
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= sl.q_len) return;
  const int64_t row = sl.row0 + i;
  float q[E], o[E];
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[row * a.q_st + head * a.q_sh + lane * E + e]);
    o[e] = 0.f;
  }
  int32_t lo, hi;
  seen_range(a, sl.kv_len, sl.kv_len - sl.q_len + i, lo, hi);
  float m = -INFINITY;
  double l = 0.0;      // tens of thousands of equal weights would drift in 32 bits
  for (int32_t j = lo; j < hi; ++j) {
    const int32_t page = a.table[b * a.ld_table + (j >> a.c.page_shift)];
    if (page < 0 || page >= a.c.num_pages) {
      report_failure(a.err, kDevBadCacheIndex);
      continue;
    }
    const int32_t off = j & (a.c.page_size - 1);
    const int64_t at = page * a.c.st_page + kvh * a.c.st_head + off * a.c.st_tok + lane * E;
    const int64_t sat = page * a.c.ss_page + kvh * a.c.ss_head + off;
    float k4[4], v4[4];
    uint32_t kw, vw;
    if constexpr (E == 4) {
      kw = *reinterpret_cast<const uint32_t*>(a.c.k + at);
      vw = *reinterpret_cast<const uint32_t*>(a.c.v + at);
    } else {
      kw = *reinterpret_cast<const uint16_t*>(a.c.k + at);
      vw = *reinterpret_cast<const uint16_t*>(a.c.v + at);
    }
    e4m3x4_to_f32(kw, k4);
    e4m3x4_to_f32(vw, v4);
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k4[e], s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.c.ks[sat] * a.scale;
    const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn), pv = p * a.c.vs[sat];
    l = l * c + p;
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, pv * v4[e]);
    m = mn;
  }
  const float inv = l > 0.0 ? static_cast<float>(1.0 / l) : 0.f;
  for (int e = 0; e < E; ++e)
    a.out[row * a.o_st + head * a.o_sh + lane * E + e] = __float2bfloat16_rn(o[e] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[row * a.heads + head] = l > 0.0 ? static_cast<float>(m + log(l)) : -INFINITY;
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

bfp8_status check_heads(int heads, int kv_heads, int dim, int max_q) {
  if (kv_heads < 1 || heads < kv_heads || heads > 65535 || heads % kv_heads != 0)
    return bad("num_heads = %d is not a multiple of num_kv_heads = %d (at most 65535)", heads, kv_heads);
  if (heads / kv_heads > 128) return bad("%d query heads a kv head (at most 128)", heads / kv_heads);
  if (dim != 64 && dim != 128) return bad("head_dim = %d (expected 64 or 128)", dim);
  if (max_q < 1 || max_q > (1 << 24)) return bad("max_q_len = %d (expected 1 .. 2^24)", max_q);
  return BFP8_OK;
}

}  // namespace

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_paged_attention_workspace_size(int num_heads, int num_kv_heads,
                                                           int head_dim, int max_q_len,
                                                           size_t* bytes) {
  const bfp8_status st = check_heads(num_heads, num_kv_heads, head_dim, max_q_len);
  if (st != BFP8_OK) return st;
  if (!bytes) return bad("bytes is null");
  *bytes = kCounterHeaderBytes;
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_paged_attention(const bfp8_attention_args* p, const bfp8_kv_cache* cache,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  AttnArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  if (!p) return bad("args is null");
  if ((st = check_heads(p->num_heads, a.c.heads, a.c.dim, p->max_q_len)) != BFP8_OK) return st;
  if (p->batch < 0 || p->batch > 65535 || p->total_q < 0 || p->total_q >= (int64_t{1} << 31))
    return bad("batch = %d, total_q = %lld", p->batch, (long long)p->total_q);
  if (p->max_pages < 1 || p->ld_table < p->max_pages)
    return bad("max_pages = %d, ld_table = %lld", p->max_pages, (long long)p->ld_table);
  if (p->max_kv_len < 0 || p->max_kv_len > (int64_t{1} << 30))
    return bad("max_kv_len = %lld (expected 0 .. 2^30)", (long long)p->max_kv_len);
  if (p->max_kv_len > static_cast<int64_t>(p->max_pages) * a.c.page_size)
    return bad("max_kv_len = %lld exceeds max_pages * page_size", (long long)p->max_kv_len);
  if (!std::isfinite(p->softmax_scale)) return bad("softmax_scale is not finite");
  if (p->causal != 0 && p->causal != 1) return bad("causal = %d (expected 0 or 1)", p->causal);
  if (p->window < 0) return bad("window = %d (expected >= 0)", p->window);
  if (p->batch == 0 || p->total_q == 0) return set_last_error(BFP8_OK, "");
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
  size_t need = 0;
  if ((st = bfp8_paged_attention_workspace_size(p->num_heads, a.c.heads, a.c.dim, p->max_q_len, &need)) != BFP8_OK)
    return st;
  if (!workspace || workspace_bytes < need)
    return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (off_align(workspace, 256)) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  int sms = 0;
  if ((st = device_for_call(&sms, &a.err)) != BFP8_OK) return st;
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
  a.group = p->num_heads / a.c.heads;
  a.batch = p->batch;
  a.max_q = p->max_q_len;
  a.causal = p->causal;
  a.window = p->window;
  a.scale = p->softmax_scale;
  const dim3 grid((p->max_q_len + 7) / 8, p->num_heads, p->batch);
  if (a.c.dim == 128) attn_rows_kernel<128><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  else attn_rows_kernel<64><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
