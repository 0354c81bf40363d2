// bfp8_kvweigh.cu -- the attention weight that every cached token receives from
// the new tokens of a call, summed over them and over the query heads of a kv head.
//
//   a[h, j] = sum over query heads of kv head h, over new tokens i that see j, of exp(scale q_i . k_j - lse_i)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_attn.cuh"
#include "bfp8_attn_math.cuh"
#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kTokens = 128;
constexpr int kRows = 16;

struct WeighArgs {
  AttnArgs a;                         // lse is an input here
  float* w;
  int64_t ws_page, ws_head;
  int32_t add;
};

// A thread a token, its key in registers; rows of queries through shared memory.
template <int D>
__global__ void __launch_bounds__(kTokens) weigh_kernel(const __grid_constant__ WeighArgs p) {
  const AttnArgs& a = p.a;
  __shared__ float s_q[kRows][D];
  __shared__ float s_lse[kRows];
  const int item = static_cast<int>(blockIdx.y), b = item / a.c.heads, h = item - b * a.c.heads;
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  const SeqLens s = seq_lens(a, b);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kTokens;
  if (s.q_len == 0 || first >= s.kv_len) return;
  const int32_t j = static_cast<int32_t>(first) + tid, pos0 = s.kv_len - s.q_len;
  int32_t page = j < s.kv_len ? a.table[b * a.ld_table + (j >> a.c.page_shift)] : -1;
  const bool bad = j < s.kv_len && (page < 0 || page >= a.c.num_pages);
  if (bad) report_failure(a.err, kDevBadCacheIndex);
  const bool live = j < s.kv_len && !bad;
  if (!live) page = 0;
  const int off = j & (a.c.page_size - 1);
  float k[D];
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live) v = *reinterpret_cast<const uint4*>(a.c.k + page * a.c.st_page + h * a.c.st_head + off * a.c.st_tok + 16 * e);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_to_f32(w[i], reinterpret_cast<float(&)[4]>(k[16 * e + 4 * i]));
  }
  const float ks = live ? a.c.ks[page * a.c.ss_page + h * a.c.ss_head + off] * a.scale : 0.f;
  float sum = 0.f;
  const int64_t rows = static_cast<int64_t>(s.q_len) * a.group;
  for (int64_t r0 = 0; r0 < rows; r0 += kRows) {
    const int n = rows - r0 < kRows ? static_cast<int>(rows - r0) : kRows;
    __syncthreads();
    for (int i = tid; i < n * D; i += kTokens) {
      const int64_t r = r0 + i / D, t = r / a.group;
      s_q[i / D][i % D] = __bfloat162float(a.q[(s.row0 + t) * a.q_st + (h * a.group + r - t * a.group) * a.q_sh + i % D]);
    }
    for (int i = tid; i < n; i += kTokens) {
      const int64_t r = r0 + i, t = r / a.group;
      s_lse[i] = a.lse[(s.row0 + t) * a.heads + h * a.group + r - t * a.group];
    }
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      int32_t lo, hi;
      seen_range(a, s.kv_len, pos0 + static_cast<int32_t>((r0 + i) / a.group), lo, hi);
      if (j < lo || j >= hi) continue;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < D; ++e) x = fmaf(k[e], s_q[i][e], x);
      sum += expf(fmaf(x, ks, -s_lse[i]));
    }
  }
  if (live) {
    float* w = p.w + page * p.ws_page + h * p.ws_head + off;
    // new tokens have no sum yet
    const bool fresh = !p.add || (a.causal != 0 && j >= pos0);
    *w = fresh ? sum : *w + sum;
  }
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

}  // namespace

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_kv_cache_weigh_workspace_size(int num_heads, int num_kv_heads, int head_dim, int max_q_len,
                                                          size_t* bytes) {
  const bfp8_status st = check_heads(num_heads, num_kv_heads, head_dim, max_q_len);
  if (st != BFP8_OK) return st;
  if (!bytes) return bad("bytes is null");
  *bytes = kCounterHeaderBytes;
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_kv_cache_weigh(const bfp8_attention_args* args, const bfp8_kv_cache* cache, float* weights,
                                           int64_t weights_stride_page, int64_t weights_stride_head, int accumulate,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  WeighArgs p{};
  bfp8_status st = check_cache(cache, &p.a.c);
  if (st != BFP8_OK) return st;
  bool empty = false;
  if ((st = check_attention(args, &p.a, &empty, false)) != BFP8_OK) return st;
  if (accumulate != 0 && accumulate != 1) return bad("accumulate = %d (expected 0 or 1)", accumulate);
  if (empty) return set_last_error(BFP8_OK, "");
  if (!args->lse || !weights) return bad("null pointer (lse=%p weights=%p)", (const void*)args->lse, (const void*)weights);
  if (args->q_stride_head < p.a.c.dim || args->q_stride_token < p.a.c.dim) return bad("q strides must be >= head_dim");
  for (int64_t s : {weights_stride_page, weights_stride_head})
    if (s < p.a.c.page_size || s >= (int64_t{1} << 39)) return bad("weights stride %lld (expected >= page_size)", (long long)s);
  if (off_align(weights, 4)) return set_last_errorf(BFP8_ERR_ALIGNMENT, "weights must be 4-byte aligned");
  const int64_t items = static_cast<int64_t>(args->batch) * p.a.c.heads;
  if (items > 65535) return set_last_errorf(BFP8_ERR_UNSUPPORTED, "batch x num_kv_heads = %lld (at most 65535)", (long long)items);
  if (!workspace || workspace_bytes < kCounterHeaderBytes || off_align(workspace, 256))
    return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace missing, too small or not 256-byte aligned");
  int sms = 0;
  if ((st = device_for_call(&sms, &p.a.err)) != BFP8_OK) return st;
  p.w = weights;
  p.ws_page = weights_stride_page;
  p.ws_head = weights_stride_head;
  p.add = accumulate;
  if (p.a.max_kv == 0) return set_last_error(BFP8_OK, "");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.a.max_kv + kTokens - 1) / kTokens), static_cast<unsigned>(items));
  cfg.blockDim = dim3(kTokens);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, p.a.c.dim == 128 ? weigh_kernel<128> : weigh_kernel<64>, p);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache weigh launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
