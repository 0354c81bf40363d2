// bfp8_kvevict.cu -- a sequence of the paged cache shortened to a budget: every
// kv head keeps its first and its most recent tokens and, of the others, those
// with the largest sums of attention weights; they move, in order, to the pages
// that the sequence goes on with.
//
//   kept = {j < first} + {j >= n - recent} + the (budget - first - recent) largest
//          of the rest, of equal ones those of lower position       (n > budget)
//
// Two kernels.  The first finds each (sequence, head)'s kept positions: a cluster
// of CTAs holds the sums as ordered 32-bit keys in shared memory and finds the
// key of rank `budget` by its 11, 11 and 10 bits, from histograms that the cluster's
// CTAs read from each other; then every warp writes the positions of its stretch
// behind those of the stretches before it.  The second moves the rows, 64 ranks a
// CTA at a time; in place, where a rank's source may be another rank's destination
// (never a lower one's: rank <= position), a cluster takes 512 ranks at once and
// loads them all before it stores one.
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_kvcache.cuh"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelKeys = 40960;                    // keys of a CTA that its shared memory holds; the rest is read again
constexpr int kSelMaxCluster = 8;
constexpr int kSelSmem = 2 * kBins * 4 + kSelKeys * 4;
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 64;                    // ranks of a CTA's step
constexpr int kMoveCluster = 8;

struct EvictArgs {
  CacheView c;
  float* w;
  int64_t ws_page, ws_head;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* out_table;           // the same as table: in place
  int64_t ld_out;
  const int32_t* lens;
  int32_t* new_lens;
  int32_t* kept;                      // [batch * heads, cap] positions
  int64_t cap;
  int32_t max_kv, budget, recent, first;
  int* err;
};

__device__ __forceinline__ int32_t length_of(const EvictArgs& a, int b) {
  const int32_t n = a.lens[b];
  return n < 0 ? 0 : n < a.max_kv ? n : a.max_kv;
}

// Larger sums have larger keys; a sum that is not a number counts as larger than any, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u >> 31) != 0u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  uint32_t* const hist0 = sel_smem;                         // two, by turns: another CTA may still read the last
  uint32_t* const keys = sel_smem + 2 * kBins;
  __shared__ uint32_t s_scan[kSelWarps];
  __shared__ uint32_t s_pick[2];                            // bin, ranks above it
  __shared__ uint32_t s_cnt[2];                             // this CTA's keys above the border, and at it
  __shared__ uint32_t s_warp[2][kSelWarps];
  const int C = static_cast<int>(gridDim.x);                // one cluster a (sequence, head)
  const int rank = static_cast<int>(cluster_ctarank());
  const int item = static_cast<int>(blockIdx.y), b = item / a.c.heads, h = item - b * a.c.heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int32_t n = length_of(a, b);
  if (rank == 0 && h == 0 && tid == 0) a.new_lens[b] = n < a.budget ? n : a.budget;
  if (n <= a.budget) return;                                // the whole cluster
  // this CTA's stretch, a whole number of warps' rows a warp
  const int32_t per_warp = (n + C * kSelThreads - 1) / (C * kSelThreads) * 32;
  const int32_t seg = per_warp * kSelWarps;
  const int32_t j0 = rank * seg < n ? rank * seg : n, j1 = j0 + seg < n ? j0 + seg : n;
  const int32_t* row = a.table + b * a.ld_table;
  auto page_ok = [&](int32_t page) {
    if (page >= 0 && page < a.c.num_pages) return true;
    report_failure(a.err, kDevBadCacheIndex);
    return false;
  };
  auto forced = [&](int32_t j) { return j < a.first || j >= n - a.recent; };
  auto load_key = [&](int32_t j) -> uint32_t {
    if (forced(j)) return 0xFFFFFFFFu;
    const int32_t page = __ldg(row + (j >> a.c.page_shift));
    return page_ok(page) ? key_of(a.w[page * a.ws_page + h * a.ws_head + (j & (a.c.page_size - 1))]) : 0u;
  };
  auto key_at = [&](int32_t j) { return j - j0 < kSelKeys ? keys[j - j0] : load_key(j); };
  for (int i = tid; i < 2 * kBins; i += kSelThreads) hist0[i] = 0u;
  // (eight at a time: the pages' numbers, then the sums; one by one their latencies add up: 8 CTAs for each of 8 heads'
  // 60000 tokens took 26 us with what follows)
  const int32_t held = j1 - j0 < kSelKeys ? j1 - j0 : kSelKeys;
  for (int32_t i0 = tid; i0 < held; i0 += 8 * kSelThreads) {
    int32_t page[8];
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int32_t j = j0 + i0 + e * kSelThreads;
      page[e] = i0 + e * kSelThreads < held && !forced(j) ? __ldg(row + (j >> a.c.page_shift)) : 0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int32_t j = j0 + i0 + e * kSelThreads;
      const bool there = i0 + e * kSelThreads < held && !forced(j) && page[e] >= 0 && page[e] < a.c.num_pages;
      w[e] = there ? __ldcg(a.w + page[e] * a.ws_page + h * a.ws_head + (j & (a.c.page_size - 1))) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int32_t i = i0 + e * kSelThreads;
      if (i < held) keys[i] = forced(j0 + i) ? 0xFFFFFFFFu : page_ok(page[e]) ? key_of(w[e]) : 0u;
    }
  }
  __syncthreads();
  // ---- the key of rank `budget`, from its top bits down
  uint32_t border = 0u, need = static_cast<uint32_t>(a.budget);     // ranks still to be found at or below `border`'s bits
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    uint32_t* hist = hist0 + (pass & 1) * kBins;
    for (int32_t j = j0 + tid; j < j1; j += kSelThreads) {
      const uint32_t k = key_at(j);
      if ((k & above) == border) atomicAdd(hist + ((k >> shift) & (bins - 1)), 1u);
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    // four bins a thread, the largest first, over the whole cluster
    const int top = bins - 4 - 4 * tid;
    uint32_t cnt[4] = {0u, 0u, 0u, 0u};
    if (top >= 0) {
      for (int r = 0; r < C; ++r) {
        uint32_t v[4];
        const uint32_t at = mapa_shared(smem_addr(hist + top), static_cast<uint32_t>(r));
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
#pragma unroll
        for (int e = 0; e < 4; ++e) cnt[e] += v[e];
      }
    }
    const uint32_t mine = cnt[0] + cnt[1] + cnt[2] + cnt[3];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    uint32_t before = incl - mine;
    for (int w = 0; w < warp; ++w) before += s_scan[w];
    if (before < need && need <= before + mine) {
      uint32_t at = before;
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        if (at < need && need <= at + cnt[e]) {
          s_pick[0] = static_cast<uint32_t>(top + e);
          s_pick[1] = at;
        }
        at += cnt[e];
      }
    }
    // the third pass counts where the first did: all have passed the second's barrier, nobody reads that any more
    if (pass == 1)
      for (int i = tid; i < kBins; i += kSelThreads) hist0[i] = 0u;
    __syncthreads();
    border |= s_pick[0] << shift;
    need -= s_pick[1];
    __syncthreads();
  }
  // ---- positions kept: every key above the border, and the first `need` at it
  const int32_t w0 = j0 + warp * per_warp < j1 ? j0 + warp * per_warp : j1, w1 = w0 + per_warp < j1 ? w0 + per_warp : j1;
  uint32_t gt = 0u, eq = 0u;
  for (int32_t j = w0 + lane; j < w1; j += 32) {
    const uint32_t k = key_at(j);
    gt += k > border;
    eq += k == border;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t g = 0u, e = 0u;
    for (int w = 0; w < kSelWarps; ++w) {
      g += s_warp[0][w];
      e += s_warp[1][w];
    }
    s_cnt[0] = g;
    s_cnt[1] = e;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  uint32_t g0 = 0u, e0 = 0u;                                // above and at the border, before this warp's stretch
  for (int r = 0; r < rank; ++r) {
    uint32_t g, e;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(g), "=r"(e)
                 : "r"(mapa_shared(smem_addr(s_cnt), static_cast<uint32_t>(r))) : "memory");
    g0 += g;
    e0 += e;
  }
  for (int w = 0; w < warp; ++w) {
    g0 += s_warp[0][w];
    e0 += s_warp[1][w];
  }
  int32_t* out = a.kept + item * a.cap;
  const uint32_t below = (1u << lane) - 1u;
  for (int32_t base = w0; base < w1; base += 32) {
    const int32_t j = base + lane;
    const uint32_t k = j < w1 ? key_at(j) : 0u;
    const uint32_t mg = __ballot_sync(0xffffffffu, j < w1 && k > border);
    const uint32_t me = __ballot_sync(0xffffffffu, j < w1 && k == border);
    const uint32_t eb = e0 + __popc(me & below), taken = eb < need ? eb : need;
    const bool keep = j < w1 && (k > border || (k == border && eb < need));
    if (keep) out[g0 + __popc(mg & below) + taken] = j;
    g0 += __popc(mg);
    e0 += __popc(me);
  }
  if (C > 1) cluster_sync();                                // the others may still read this CTA's counts
}

template <int D, bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kPieces = D / 16;                           // 16-byte pieces of a row's keys, and of its values
  constexpr int kStep = kMoveThreads / (2 * kPieces);       // rows that the block holds a piece a thread of
  constexpr int kUnroll = kMoveTokens / kStep;
  __shared__ int64_t s_src[kMoveTokens][3], s_dst[kMoveTokens][3];    // offsets of codes, scales and sums; -1: none
  const int item = static_cast<int>(blockIdx.y), b = item / a.c.heads, h = item - b * a.c.heads;
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  const int32_t n = length_of(a, b);
  const bool whole = n <= a.budget;
  if (kInPlace && whole) return;                            // (all of a cluster)
  const int32_t m = whole ? n : a.budget;
  const int32_t* kept = a.kept + item * a.cap;
  const int32_t step = static_cast<int32_t>(gridDim.x) * kMoveTokens;
  const int piece = tid % (2 * kPieces), r0 = tid / (2 * kPieces);
  uint8_t* const codes = (piece < kPieces ? a.c.k : a.c.v) + (piece % kPieces) * 16;
  // in place every CTA of the cluster takes part in each round's barrier
  for (int32_t i0 = 0; i0 < m; i0 += step) {
    const int32_t base = i0 + static_cast<int32_t>(blockIdx.x) * kMoveTokens;
    if (!kInPlace && base >= m) break;
    if (tid < kMoveTokens) {
      const int32_t i = base + tid;
      s_src[tid][0] = s_dst[tid][0] = -1;
      if (i < m) {
        const int32_t j = whole ? i : __ldcg(kept + i);
        if (!kInPlace || j != i) {
          const int32_t ps = a.table[b * a.ld_table + (j >> a.c.page_shift)], pd = a.out_table[b * a.ld_out + (i >> a.c.page_shift)];
          if (ps < 0 || ps >= a.c.num_pages || pd < 0 || pd >= a.c.num_pages) {
            report_failure(a.err, kDevBadCacheIndex);
          } else {
            const int32_t os = j & (a.c.page_size - 1), od = i & (a.c.page_size - 1);
            s_src[tid][0] = ps * a.c.st_page + h * a.c.st_head + os * a.c.st_tok;
            s_src[tid][1] = ps * a.c.ss_page + h * a.c.ss_head + os;
            s_src[tid][2] = ps * a.ws_page + h * a.ws_head + os;
            s_dst[tid][0] = pd * a.c.st_page + h * a.c.st_head + od * a.c.st_tok;
            s_dst[tid][1] = pd * a.c.ss_page + h * a.c.ss_head + od;
            s_dst[tid][2] = pd * a.ws_page + h * a.ws_head + od;
          }
        }
      }
    }
    __syncthreads();
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = s_src[r0 + u * kStep][0];
      if (at >= 0) x[u] = *reinterpret_cast<const uint4*>(codes + at);
    }
    float f = 0.f;
    const int what = tid / kMoveTokens, ri = tid % kMoveTokens;       // key scales, value scales, sums
    const bool scalar = what < 3 && s_src[ri][0] >= 0;
    if (scalar) f = what == 0 ? a.c.ks[s_src[ri][1]] : what == 1 ? a.c.vs[s_src[ri][1]] : a.w[s_src[ri][2]];
    if (kInPlace) cluster_sync();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = s_dst[r0 + u * kStep][0];
      if (at >= 0) *reinterpret_cast<uint4*>(codes + at) = x[u];
    }
    if (scalar) *(what == 0 ? a.c.ks + s_dst[ri][1] : what == 1 ? a.c.vs + s_dst[ri][1] : a.w + s_dst[ri][2]) = f;
    __syncthreads();
  }
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

template <typename F>
cudaError_t launch(F* f, dim3 grid, int threads, int smem, int cluster, const EvictArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

int64_t kept_cap(int64_t max_kv, int64_t budget) { return max_kv > budget ? budget : 0; }

}  // namespace

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_kv_cache_evict_workspace_size(int batch, int num_kv_heads, int64_t max_kv_len, int64_t budget,
                                                          size_t* bytes) {
  if (batch < 0 || batch > 65535 || num_kv_heads < 1 || num_kv_heads > 65535)
    return bad("batch = %d, num_kv_heads = %d", batch, num_kv_heads);
  if (max_kv_len < 0 || max_kv_len > (int64_t{1} << 30)) return bad("max_kv_len = %lld (expected 0 .. 2^30)", (long long)max_kv_len);
  if (budget < 1) return bad("budget = %lld (expected >= 1)", (long long)budget);
  if (!bytes) return bad("bytes is null");
  *bytes = kCounterHeaderBytes + static_cast<size_t>(batch) * num_kv_heads * kept_cap(max_kv_len, budget) * sizeof(int32_t);
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_kv_cache_evict(const bfp8_evict_args* p, const bfp8_kv_cache* cache, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  EvictArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  if (!p) return bad("args is null");
  if (p->batch < 0 || p->batch > 65535) return bad("batch = %d", p->batch);
  if (static_cast<int64_t>(p->batch) * a.c.heads > 65535)
    return set_last_errorf(BFP8_ERR_UNSUPPORTED, "batch x num_kv_heads = %lld (at most 65535)", (long long)p->batch * a.c.heads);
  if (p->max_kv_len < 0 || p->max_kv_len > (int64_t{1} << 30))
    return bad("max_kv_len = %lld (expected 0 .. 2^30)", (long long)p->max_kv_len);
  if (p->budget < 1 || p->recent < 0 || p->first < 0 || p->recent > p->budget || p->first > p->budget - p->recent)
    return bad("budget = %lld, recent = %lld, first = %lld (expected first + recent <= budget, budget >= 1)",
               (long long)p->budget, (long long)p->recent, (long long)p->first);
  const int64_t most = p->max_kv_len < p->budget ? p->max_kv_len : p->budget;       // tokens that a sequence keeps
  if (p->max_pages < 0 || p->ld_table < p->max_pages || p->max_kv_len > static_cast<int64_t>(p->max_pages) * a.c.page_size)
    return bad("max_pages = %d, ld_table = %lld for max_kv_len = %lld", p->max_pages, (long long)p->ld_table, (long long)p->max_kv_len);
  if (p->out_table != nullptr &&
      (p->max_out_pages < 0 || p->ld_out < p->max_out_pages || most > static_cast<int64_t>(p->max_out_pages) * a.c.page_size))
    return bad("max_out_pages = %d, ld_out = %lld for %lld kept tokens", p->max_out_pages, (long long)p->ld_out, (long long)most);
  if (p->batch == 0) return set_last_error(BFP8_OK, "");
  if (!p->kv_lens || !p->new_lens) return bad("null pointer (kv_lens=%p new_lens=%p)", (const void*)p->kv_lens, (const void*)p->new_lens);
  if (p->max_kv_len > 0 && (!p->weights || !p->block_table))
    return bad("null pointer (weights=%p block_table=%p)", (const void*)p->weights, (const void*)p->block_table);
  if (p->new_lens < p->kv_lens + p->batch && p->kv_lens < p->new_lens + p->batch) return bad("new_lens overlaps kv_lens");
  if (p->max_kv_len > 0)
    for (int64_t s : {p->weights_stride_page, p->weights_stride_head})
      if (s < a.c.page_size || s >= (int64_t{1} << 39)) return bad("weights stride %lld (expected >= page_size)", (long long)s);
  if (off_align(p->weights, 4) || off_align(p->block_table, 4) || off_align(p->out_table, 4) || off_align(p->kv_lens, 4) ||
      off_align(p->new_lens, 4))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "pointers must be 4-byte aligned");
  const size_t need =
      kCounterHeaderBytes + static_cast<size_t>(p->batch) * a.c.heads * kept_cap(p->max_kv_len, p->budget) * sizeof(int32_t);
  if (!workspace || workspace_bytes < need)
    return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (off_align(workspace, 256)) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  int sms = 0;
  if ((st = device_for_call(&sms, &a.err)) != BFP8_OK) return st;
  a.w = p->weights;
  a.ws_page = p->weights_stride_page;
  a.ws_head = p->weights_stride_head;
  a.table = p->block_table;
  a.ld_table = p->ld_table;
  const bool in_place = p->out_table == nullptr;
  a.out_table = in_place ? p->block_table : p->out_table;
  a.ld_out = in_place ? p->ld_table : p->ld_out;
  a.lens = p->kv_lens;
  a.new_lens = p->new_lens;
  a.kept = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kCounterHeaderBytes);
  a.cap = kept_cap(p->max_kv_len, p->budget);
  a.max_kv = static_cast<int32_t>(p->max_kv_len);
  a.budget = static_cast<int32_t>(p->budget < (int64_t{1} << 30) ? p->budget : (int64_t{1} << 30));
  a.recent = static_cast<int32_t>(p->recent < a.budget ? p->recent : a.budget);
  a.first = static_cast<int32_t>(p->first < a.budget ? p->first : a.budget);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int items = p->batch * a.c.heads;
  // CTAs of a (sequence, head): as many as leave each SM one and each thread a few keys
  int cluster = 1;
  while (cluster < kSelMaxCluster && items * cluster < sms && p->max_kv_len > static_cast<int64_t>(cluster) * 4 * kSelThreads) cluster *= 2;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmem);
  if (e == cudaSuccess) {
    // the keys of a stretch at its longest
    const int64_t stretch = (p->max_kv_len + cluster * kSelThreads - 1) / (cluster * kSelThreads) * kSelThreads;
    const int smem = 2 * kBins * 4 + 4 * static_cast<int>(stretch < kSelKeys ? stretch : kSelKeys);
    e = launch(evict_select_kernel, dim3(cluster, items), kSelThreads, smem, cluster, a, cs);
  }
  if (e == cudaSuccess && most > 0) {
    if (in_place) {
      if (a.cap > 0) {
        auto f = a.c.dim == 128 ? evict_move_kernel<128, true> : evict_move_kernel<64, true>;
        e = launch(f, dim3(kMoveCluster, items), kMoveThreads, 0, kMoveCluster, a, cs);
      }
    } else {
      auto f = a.c.dim == 128 ? evict_move_kernel<128, false> : evict_move_kernel<64, false>;
      const int64_t blocks = (most + kMoveTokens - 1) / kMoveTokens;
      e = launch(f, dim3(static_cast<unsigned>(blocks), items), kMoveThreads, 0, 1, a, cs);
    }
  }
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache evict launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
