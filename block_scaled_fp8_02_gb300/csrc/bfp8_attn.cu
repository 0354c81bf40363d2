// bfp8_attn.cu -- attention of new tokens over the paged e4m3 cache: the C
// entry points, and which kernel takes which sequences.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bfp8_attn.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"

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

// Are both parts of a call over shared prefixes computed apart, beside each other, and joined in a launch of their own?  Where the
// prefixes' takes the tile kernel and the own one the kernel for few rows: many sequences' single tokens.  64 of them, own contexts up
// to 1000 behind a prefix of 8192, 64 / 8 heads of 128: 98 us with the own part's rows waiting for the prefix's, 75 apart.  (With more
// new tokens the parts' fp32 rows would take longer to write and read than the wait; with fewer the third launch would.)
bool parts_apart(int group, int max_prefix_q, int max_q) { return has_many(group, max_prefix_q) && !has_many(group, max_q); }
// Scratch of such a call: each part's partial rows of the kernel for few rows, and those of the other, which only one takes at a time.
size_t shared_scratch_bytes(int group, int dim, int max_prefix_q, int max_q, int sms) {
  const bool tile = has_many(group, max_prefix_q) || has_many(group, max_q);
  return kCounterHeaderBytes + few_bytes(group, dim, max_prefix_q, sms) + few_bytes(group, dim, max_q, sms) +
         (tile ? attn_tile_partial_bytes(dim, sms) : 0);
}
// Behind all that: a part's rows in fp32 and their log2 sums, for each part that is not joined at once.
size_t shared_rows_bytes(int64_t total_q, int heads, int dim, bool apart) {
  return static_cast<size_t>(total_q) * heads * (dim + 1) * sizeof(float) * (apart ? 2 : 1);
}
// The new tokens, up to max_q, with which a call has the most partial rows of the kernel for few rows: those of all sequences at
// once, where more tokens leave it single ones.
int most_few_q(int group, int max_q) {
  const int q = group < kFewRows ? kFewRows / group : 1;
  return max_q < q ? max_q : q;
}

// Sequences (or prefixes), rows and context of a call, checked apart from the pointers.
bfp8_status check_context(const char* what, int batch, int max_q, int max_pages, int64_t ld_table, int64_t max_kv, int page,
                          bool empty) {
  if (batch < 0 || batch > 65535) return bad("%s: %d (expected 0 .. 65535)", what, batch);
  if (max_q < (empty ? 0 : 1) || max_q > (1 << 24)) return bad("%s: max_q_len = %d (expected 1 .. 2^24)", what, max_q);
  if (max_pages < (empty ? 0 : 1) || ld_table < max_pages)
    return bad("%s: max_pages = %d, ld_table = %lld", what, max_pages, (long long)ld_table);
  if (max_kv < 0 || max_kv > (int64_t{1} << 30)) return bad("%s: bound of lengths = %lld (expected 0 .. 2^30)", what, (long long)max_kv);
  if (max_kv > static_cast<int64_t>(max_pages) * page)
    return bad("%s: bound of lengths = %lld exceeds max_pages * page_size", what, (long long)max_kv);
  return BFP8_OK;
}

// The device, and a workspace of `need(sms)` bytes.
template <typename Need>
bfp8_status check_workspace(const void* workspace, size_t bytes, int* sms, int** err, Need need) {
  const bfp8_status st = device_for_call(sms, err);
  if (st != BFP8_OK) {
    // a host without a device still learns of a missing workspace
    if (!workspace || bytes < kCounterHeaderBytes || off_align(workspace, 256))
      return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace missing, too small or not 256-byte aligned");
    return st;
  }
  const size_t n = need(*sms);
  if (!workspace || bytes < n) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", bytes, n);
  if (off_align(workspace, 256)) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  return BFP8_OK;
}

// Tensor maps of the keys' and values' codes.
struct CacheMaps {
  CUtensorMap k, v;
};
bfp8_status encode_maps(const CacheView& c, CacheMaps* m) {
  const uint64_t dims[4] = {static_cast<uint64_t>(c.dim), static_cast<uint64_t>(c.page_size),
                            static_cast<uint64_t>(c.heads), static_cast<uint64_t>(c.num_pages)};
  const uint64_t strides[3] = {static_cast<uint64_t>(c.st_tok), static_cast<uint64_t>(c.st_head),
                               static_cast<uint64_t>(c.st_page)};
  const uint32_t box[4] = {static_cast<uint32_t>(c.dim),
                           static_cast<uint32_t>(c.page_size < 128 ? c.page_size : 128), 1u, 1u};
  const bfp8_status st = encode_bytes_tiled(&m->k, c.k, 4, dims, strides, box, c.dim);
  return st != BFP8_OK ? st : encode_bytes_tiled(&m->v, c.v, 4, dims, strides, box, c.dim);
}

// Can a sequence be short enough for the kernel for few rows?  Not if the others at their longest leave this
// one too many tokens (always so for a single chunk): then its launch is saved.
bool few_launched(const AttnArgs& a) {
  return a.group <= kFewRows && (!has_many(a.group, a.max_q) ||
                                 a.total_q <= static_cast<int64_t>(a.batch - 1) * a.max_q + 8 * few_groups(a.group, a.max_q) / a.group);
}

// SMs that the prefixes' part `b` gets where the own part `a` (by the kernel for few rows) runs beside it: by the cycles that each needs
// at its bounds (contexts of the kernel for few rows at three quarters of theirs), a block's and an item's own among them.  64 sequences, own
// contexts up to 1000 behind 8192 tokens, 64 / 8 heads of 128, by the tile kernel's SMs: 48 81 us, 64 69, 80 71, 96 78, 112 104; 79
// with the kernel for few rows behind the other, on the SMs that it leaves.  (The cycles are those of that shape, for heads of 64 too, and the
// bounds are the caller's: loose ones move the split towards its ends.)
int prefix_sms(const AttnArgs& a, const AttnArgs& b, int sms) {
  auto few = [](const AttnArgs& x) {
    return static_cast<double>(x.batch) * x.c.heads * (0.75 * static_cast<double>(x.max_kv) / 128 + 4) * 1340;
  };
  const double blocks = static_cast<double>(b.batch) * b.c.heads * ((static_cast<int64_t>(b.max_q) * b.group + 255) / 256);
  const double prefix = has_many(b.group, b.max_q) ? blocks * (static_cast<double>(b.max_kv) / 128 + 8) * 4500 : few(b);
  const int n = static_cast<int>(sms * (prefix / (prefix + few(a))));
  return n < sms / 4 ? sms / 4 : n > sms * 3 / 4 ? sms * 3 / 4 : n;
}

// Joins both parts of the rows of all sequences: a warp a (row, head).
struct JoinArgs {
  AttnArgs a;                         // the prefixes' part
  const float* own_o;                 // the own part's
  const float* own_lse2;
};
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_parts_kernel(const __grid_constant__ JoinArgs p) {
  const AttnArgs& a = p.a;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);      // token * heads + head
  const int lane = threadIdx.x & 31;
  const int64_t token = row / a.heads;
  const int head = static_cast<int>(row - token * a.heads);
  if (token >= a.total_q || token < a.cu_q[0] || token >= a.cu_q[a.batch]) return;
  using Vec = typename std::conditional<D == 128, float4, float2>::type;
  const Joined j = join_prefix(a, token, head, __ldcg(p.own_lse2 + row));
  const Vec y = __ldcg(reinterpret_cast<const Vec*>(p.own_o + row * D) + lane);
  Vec x{};
  if (j.covered) x = __ldcg(reinterpret_cast<const Vec*>(a.part_o + row * D) + lane);
  float o[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e)
    o[e] = fmaf(reinterpret_cast<const float*>(&x)[e], j.prefix, reinterpret_cast<const float*>(&y)[e] * j.own);
  __nv_bfloat16* dst = a.out + token * a.o_st + head * a.o_sh + lane * (D / 32);
  if constexpr (D == 128) st_global_v2(dst, pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0], o[1]);
  if (a.lse != nullptr && lane == 0) a.lse[row] = j.lse2 * 0.6931471805599453f;
}

cudaError_t launch_join(const JoinArgs& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.a.total_q * p.a.heads + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.a.c.dim == 128 ? join_parts_kernel<128> : join_parts_kernel<64>, p);
}

// What the kernels of one part (or all) have to themselves: counters (zero) and partial rows.
struct Scratch {
  int32_t* few_counters;
  float* few;
  int32_t* tile_counters;
  float* tile;
};

// Launches what one part (or all) takes: the kernel for many rows, that for few, or both, on `ctas` SMs.  beside: the launch before is
// of another part, and this one takes the kernel for few rows alone, which needs nothing of it (kAttnOwn: before it joins rows).
bfp8_status launch_part(const CacheMaps& m, AttnArgs a, AttnMode mode, int ctas, const Scratch& w, bool beside, cudaStream_t cs) {
  const int groups = few_groups(a.group, a.max_q);
  a.few_rows = groups * 8;
  const bool many = has_many(a.group, a.max_q), few = few_launched(a);
  if (!few) a.few_rows = 0;
  cudaError_t e = cudaSuccess;
  if (many) e = launch_attn_tile(m.k, m.v, a, mode, ctas, w.tile_counters, w.tile, cs);
  if (e == cudaSuccess && few)
    e = launch_attn_decode(m.k, m.v, a, mode, groups, ctas, w.few_counters, w.few, many ? 1 : beside ? 2 : 0, cs);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return BFP8_OK;
}

}  // namespace

bfp8_status check_heads(int heads, int kv_heads, int dim, int max_q) {
  if (kv_heads < 1 || heads < kv_heads || heads > 65535 || heads % kv_heads != 0)
    return bad("num_heads = %d is not a multiple of num_kv_heads = %d (at most 65535)", heads, kv_heads);
  if (heads / kv_heads > 128) return bad("%d query heads a kv head (at most 128)", heads / kv_heads);
  if (dim != 64 && dim != 128) return bad("head_dim = %d (expected 64 or 128)", dim);
  if (max_q < 1 || max_q > (1 << 24)) return bad("max_q_len = %d (expected 1 .. 2^24)", max_q);
  return BFP8_OK;
}

bfp8_status check_attention(const bfp8_attention_args* p, AttnArgs* a, bool* empty, bool needs_out) {
  if (!p) return bad("args is null");
  // an empty call's bounds may be zero
  *empty = p->batch == 0 || p->total_q == 0;
  bfp8_status st = check_heads(p->num_heads, a->c.heads, a->c.dim, *empty && p->max_q_len == 0 ? 1 : p->max_q_len);
  if (st != BFP8_OK) return st;
  if (p->batch < 0 || p->batch > 65535 || p->total_q < 0 || p->total_q >= (int64_t{1} << 31))
    return bad("batch = %d, total_q = %lld", p->batch, (long long)p->total_q);
  if (p->max_pages < (*empty ? 0 : 1) || p->ld_table < p->max_pages)
    return bad("max_pages = %d, ld_table = %lld", p->max_pages, (long long)p->ld_table);
  if (p->max_kv_len < 0 || p->max_kv_len > (int64_t{1} << 30))
    return bad("max_kv_len = %lld (expected 0 .. 2^30)", (long long)p->max_kv_len);
  if (p->max_kv_len > static_cast<int64_t>(p->max_pages) * a->c.page_size)
    return bad("max_kv_len = %lld exceeds max_pages * page_size", (long long)p->max_kv_len);
  if (!std::isfinite(p->softmax_scale)) return bad("softmax_scale is not finite");
  if (p->causal != 0 && p->causal != 1) return bad("causal = %d (expected 0 or 1)", p->causal);
  if (p->window < 0) return bad("window = %d (expected >= 0)", p->window);
  if (*empty) return BFP8_OK;
  if (!p->q || (needs_out && !p->out) || !p->block_table || !p->cu_q || !p->kv_lens)
    return bad("null pointer (q=%p out=%p block_table=%p cu_q=%p kv_lens=%p)", p->q, p->out,
               (const void*)p->block_table, (const void*)p->cu_q, (const void*)p->kv_lens);
  const int64_t o_st = needs_out ? p->out_stride_token : a->c.dim, o_sh = needs_out ? p->out_stride_head : a->c.dim;
  for (int64_t s : {p->q_stride_token, p->q_stride_head, o_st, o_sh})
    if (s < 0) return bad("negative stride %lld", (long long)s);
  if (o_sh < a->c.dim || o_st < a->c.dim) return bad("out strides must be >= head_dim");
  for (int64_t s : {p->q_stride_token, p->q_stride_head, o_st, o_sh})
    if (s % 8) return set_last_errorf(BFP8_ERR_ALIGNMENT, "q and out strides must be multiples of 8 elements");
  if (off_align(p->q, 16) || (needs_out && off_align(p->out, 16)) || off_align(p->lse, 4) || off_align(p->block_table, 4) ||
      off_align(p->cu_q, 4) || off_align(p->kv_lens, 4))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "q and out must be 16-byte aligned, the rest 4-byte");
  a->group = p->num_heads / a->c.heads;
  a->q = static_cast<const __nv_bfloat16*>(p->q);
  a->out = needs_out ? static_cast<__nv_bfloat16*>(p->out) : nullptr;
  a->lse = p->lse;
  a->q_st = p->q_stride_token;
  a->q_sh = p->q_stride_head;
  a->o_st = o_st;
  a->o_sh = o_sh;
  a->table = p->block_table;
  a->ld_table = p->ld_table;
  a->cu_q = p->cu_q;
  a->kv_lens = p->kv_lens;
  a->total_q = p->total_q;
  a->max_kv = p->max_kv_len;
  a->heads = p->num_heads;
  a->batch = p->batch;
  a->max_q = p->max_q_len;
  a->causal = p->causal;
  // A window past every distance hides nothing.  Positions begin at -max_q_len (more new tokens than context), so
  // without this p - window + 1 would leave 32 bits for the widest windows.
  a->window = p->window > p->max_kv_len + p->max_q_len ? 0 : p->window;
  a->scale = p->softmax_scale;
  return BFP8_OK;
}

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
  bool empty = false;
  if ((st = check_attention(p, &a, &empty, true)) != BFP8_OK) return st;
  if (empty) return set_last_error(BFP8_OK, "");
  int sms = 0;
  st = check_workspace(workspace, workspace_bytes, &sms, &a.err,
                       [&](int n) { return workspace_bytes_for(a.group, a.c.dim, a.max_q, n); });
  if (st != BFP8_OK) return st;
  CacheMaps m;
  if ((st = encode_maps(a.c, &m)) != BFP8_OK) return st;
  int32_t* counters = static_cast<int32_t*>(workspace);
  char* partials = static_cast<char*>(workspace) + kCounterHeaderBytes;
  const Scratch w{counters, reinterpret_cast<float*>(partials), counters + sms,
                  reinterpret_cast<float*>(partials + few_bytes(a.group, a.c.dim, a.max_q, sms))};
  if ((st = launch_part(m, a, kAttnWhole, sms, w, false, static_cast<cudaStream_t>(stream))) != BFP8_OK) return st;
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_shared_prefix_attention_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                                                   int max_prefix_q_len, int max_q_len, int64_t total_q,
                                                                   size_t* bytes) {
  bfp8_status st = check_heads(num_heads, num_kv_heads, head_dim, max_q_len);
  if (st == BFP8_OK) st = check_heads(num_heads, num_kv_heads, head_dim, max_prefix_q_len);
  if (st != BFP8_OK) return st;
  if (total_q < 0 || total_q >= (int64_t{1} << 31)) return bad("total_q = %lld", (long long)total_q);
  if (!bytes) return bad("bytes is null");
  int sms = 0;
  int* err = nullptr;
  if ((st = device_for_call(&sms, &err)) != BFP8_OK) return st;
  // what calls below the bounds need too
  const int group = num_heads / num_kv_heads;
  const int pq = most_few_q(group, max_prefix_q_len), q = most_few_q(group, max_q_len);
  const bool tile = has_many(group, max_prefix_q_len) || has_many(group, max_q_len);
  *bytes = kCounterHeaderBytes + few_bytes(group, head_dim, pq, sms) + few_bytes(group, head_dim, q, sms) +
           (tile ? attn_tile_partial_bytes(head_dim, sms) : 0) +
           shared_rows_bytes(total_q, num_heads, head_dim, parts_apart(group, max_prefix_q_len, max_q_len));
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_shared_prefix_attention(const bfp8_attention_args* p, const bfp8_prefix_args* f,
                                                    const bfp8_kv_cache* cache, void* workspace, size_t workspace_bytes,
                                                    void* stream) {
  AttnArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  bool empty = false;
  if ((st = check_attention(p, &a, &empty, true)) != BFP8_OK) return st;
  if (p->window != 0) return bad("window = %d: a window over a shared prefix is not supported", p->window);
  if (!f) return bad("prefix is null");
  const bool none = empty || f->prefixes == 0;
  if ((st = check_context("prefix", f->prefixes, f->max_q_len, f->max_pages, f->ld_table, f->max_len, a.c.page_size, none)) != BFP8_OK)
    return st;
  if (empty) return set_last_error(BFP8_OK, "");
  if (!none) {
    if (!f->block_table || !f->cu_q || !f->lens)
      return bad("prefix: null pointer (block_table=%p cu_q=%p lens=%p)", (const void*)f->block_table, (const void*)f->cu_q,
                 (const void*)f->lens);
    if (off_align(f->block_table, 4) || off_align(f->cu_q, 4) || off_align(f->lens, 4))
      return set_last_errorf(BFP8_ERR_ALIGNMENT, "prefix: pointers must be 4-byte aligned");
  }
  int sms = 0;
  auto scratch = [&](int n) {
    return none ? workspace_bytes_for(a.group, a.c.dim, a.max_q, n)
                : shared_scratch_bytes(a.group, a.c.dim, f->max_q_len, a.max_q, n);
  };
  const size_t rows = none ? 0 : shared_rows_bytes(a.total_q, a.heads, a.c.dim, false);
  st = check_workspace(workspace, workspace_bytes, &sms, &a.err, [&](int n) { return scratch(n) + rows; });
  if (st != BFP8_OK) return st;
  // (a workspace for more new tokens a sequence, whose parts are joined at once, need not hold both parts' rows)
  const bool apart =
      !none && parts_apart(a.group, f->max_q_len, a.max_q) && workspace_bytes >= scratch(sms) + 2 * rows;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // counters: one a CTA of either kernel for few rows, two of the other (4 * sms fit the header)
  int32_t* counters = static_cast<int32_t*>(workspace);
  char* partials = static_cast<char*>(workspace) + kCounterHeaderBytes;
  const size_t few_prefix = none ? 0 : few_bytes(a.group, a.c.dim, f->max_q_len, sms), few_own = few_bytes(a.group, a.c.dim, a.max_q, sms);
  float* const tile = reinterpret_cast<float*>(partials + few_prefix + few_own);
  const Scratch w_prefix{counters, reinterpret_cast<float*>(partials), counters + sms, tile},
      w_own{counters + 3 * sms, reinterpret_cast<float*>(partials + few_prefix), counters + sms, tile};
  CacheMaps m;
  if ((st = encode_maps(a.c, &m)) != BFP8_OK) return st;
  if (none) {
    if ((st = launch_part(m, a, kAttnWhole, sms, w_own, false, cs)) != BFP8_OK) return st;
    return set_last_error(BFP8_OK, "");
  }
  // rows of one part or both (whole rows: read and written in vectors), then their sums
  const int64_t row_floats = a.total_q * a.heads * a.c.dim;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + scratch(sms));
  a.part_lse2 = a.part_o + (apart ? 2 : 1) * row_floats;
  a.part_cu = f->cu_q;
  a.prefixes = f->prefixes;
  AttnArgs b = a;
  b.table = f->block_table;
  b.ld_table = f->ld_table;
  b.cu_q = f->cu_q;
  b.kv_lens = f->lens;
  b.max_kv = f->max_len;
  b.batch = f->prefixes;
  b.max_q = f->max_q_len;
  b.causal = 0;
  b.window = 0;
  // The own part runs beside the prefixes' where each is one launch, that of the own part for few rows: apart, or joining its rows itself
  // where the prefixes' are few too (4 sequences, up to 40 own tokens behind 500: 28.9 us one behind the other, 25.7 so).
  const bool beside = !has_many(a.group, a.max_q) && (!has_many(b.group, b.max_q) || (apart && !few_launched(b)));
  const int ctas = beside ? prefix_sms(a, b, sms) : sms;
  if ((st = launch_part(m, b, kAttnPart, ctas, w_prefix, false, cs)) != BFP8_OK) return st;
  if (!(beside && apart)) {
    if ((st = launch_part(m, a, kAttnOwn, beside ? sms - ctas : sms, w_own, beside, cs)) != BFP8_OK) return st;
    return set_last_error(BFP8_OK, "");
  }
  AttnArgs own = a;
  own.part_o = a.part_o + row_floats;
  own.part_lse2 = a.part_lse2 + a.total_q * a.heads;
  if ((st = launch_part(m, own, kAttnPart, sms - ctas, w_own, true, cs)) != BFP8_OK) return st;
  const cudaError_t e = launch_join(JoinArgs{a, own.part_o, own.part_lse2}, cs);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
