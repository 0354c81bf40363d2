// bfp8_kvevict.cu -- a sequence of the paged cache shortened to a budget: every
// kv head keeps its first and its most recent tokens and, of the others, those
// with the largest sums of attention weights; they move, in order, to the pages
// that the sequence goes on with.
//
//   kept = {j < first} + {j >= n - recent} + the (budget - first - recent) largest
//          of the rest, of equal ones those of lower position       (n > budget)
//
// A cluster of CTAs (or one) a (sequence, head).  Its threads hold the sums as ordered
// 32-bit keys and find the key of rank `budget` by its 11, 11 and 10 bits, from
// histograms that are added up in the cluster's first CTA; the positions kept are written
// in order, by counts of them before each 32, and the warps move the
// rows, each 16 or 32 ranks at a time.  In place a rank's source may be
// another's destination (never a lower one's: rank <= position), so there the
// cluster loads all ranks of a round before it stores one.
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_kvcache.cuh"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kBins = 2048;
// Threads of a CTA that looks for the kept positions, and keys that each holds (a longer stretch is read anew each time).
// Many (sequence, head)s: small CTAs, four a SM (64 x 8 heads of 8000 tokens 28 us, 36 in clusters of two).  Few: large
// ones (16 x 8 heads 11 us, 19 with small ones), in clusters where their keys are too many for one (a cluster's barriers cost about
// a microsecond each, so no more CTAs than the keys need).  The choice goes by the number of (sequence, head)s alone: small CTAs read what is
// past their 8192 keys anew in each pass (64 x 8 heads to 2048 tokens, the whole call: 110 us from up to 8000, 170 from 16384, 255 from
// 32768, where the moving is much the same).
template <int T>
struct Find {
  static constexpr int kWarps = T / 32, kHold = T == 256 ? 32 : 16, kChunk = kHold * T, kCtasPerSm = T == 256 ? 4 : 1;
};
constexpr int kMaxCluster = 4;
constexpr int kMoveThreads = 256;
constexpr int kMoveTokens = 64;                    // ranks of a CTA's step (a warp moving 16 by itself, their pages asked for
                                                   // ahead: 92 us against 80 for 64 sequences' 2048 tokens, 8 heads of 128)
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

// Sum over the block's threads before this one (all call it); s_scan: a place a warp.
__device__ __forceinline__ uint32_t sum_before(uint32_t v, uint32_t* s_scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  const uint32_t other = lane < warp ? s_scan[lane] : 0u;
  const uint32_t before = __reduce_add_sync(0xffffffffu, other) + incl - v;
  __syncthreads();
  return before;
}

__device__ __forceinline__ void add_shared_cluster(uint32_t at, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void ld_shared_cluster_u2(uint32_t at, uint32_t& x, uint32_t& y) {
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(at) : "memory");
}

// Writes the positions that (sequence, head h) keeps of its n > budget tokens, in order, to `kept`.  All threads of the
// cluster's C CTAs call it.
template <int kThreads>
__device__ __forceinline__ void find_kept(const EvictArgs& a, int C, int rank, int h, int32_t n, const int32_t* row, int32_t* kept) {
  constexpr int kWarps = Find<kThreads>::kWarps, kHold = Find<kThreads>::kHold, kChunk = Find<kThreads>::kChunk;
  constexpr int kOwn = kBins / kThreads;                    // bins that a thread adds up
  constexpr int kAllBins = 2 * kBins + kBins / 2;           // of the three passes
  __shared__ __align__(16) uint32_t s_own[kAllBins], s_all[kAllBins];     // of this CTA's keys; of the cluster's (the first CTA's)
  __shared__ uint32_t s_scan[kWarps];
  __shared__ uint32_t s_pick[2];                            // bin, ranks above it
  __shared__ uint32_t s_before[2];                          // keys above the border, and at it, of the CTAs before this one
  __shared__ uint32_t s_above[kHold * kWarps], s_at[kHold * kWarps];      // ... of each 32 positions
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kCounts = kHold * kWarps;
  static_assert(kCounts <= kThreads, "a thread a count");
  // this CTA's stretch
  const int32_t seg = (n + C * 32 - 1) / (C * 32) * 32;
  const int32_t j0 = rank * seg < n ? rank * seg : n, j1 = j0 + seg < n ? j0 + seg : n;
  const uint32_t choice = static_cast<uint32_t>(n - a.recent - a.first);  // positions that are not kept in any case, from `first` on
  const float* sums = a.w + h * a.ws_head;
  uint32_t key[kHold];                                      // of positions at + e * kThreads + tid
  // (eight at a time: the pages' numbers, then the sums; one by one their latencies add up)
  auto load = [&](int32_t at) {
#pragma unroll
    for (int e0 = 0; e0 < kHold; e0 += 8) {
      if (at + e0 * kThreads >= j1) break;
      int32_t page[8];
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t j = at + (e0 + e) * kThreads + tid;
        page[e] = j < j1 && static_cast<uint32_t>(j - a.first) < choice ? __ldg(row + (j >> a.c.page_shift)) : -1;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t j = at + (e0 + e) * kThreads + tid;
        w[e] = 0.f;
        if (static_cast<uint32_t>(page[e]) < static_cast<uint32_t>(a.c.num_pages))
          w[e] = __ldcg(sums + page[e] * a.ws_page + (j & (a.c.page_size - 1)));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int32_t j = at + (e0 + e) * kThreads + tid;
        key[e0 + e] = key_of(w[e]);
        if (static_cast<uint32_t>(page[e]) >= static_cast<uint32_t>(a.c.num_pages)) {
          const bool chosen = static_cast<uint32_t>(j - a.first) < choice;       // else kept in any case
          if (chosen && j < j1) report_failure(a.err, kDevBadCacheIndex);
          key[e0 + e] = chosen ? 0u : 0xFFFFFFFFu;
        }
      }
    }
  };
  const bool once = j1 - j0 <= kChunk;
  for (int i = tid; i < kAllBins; i += kThreads) s_own[i] = s_all[i] = 0u;
  if (tid < 2) s_before[tid] = 0u;
  if (once) load(j0);
  if (C > 1) cluster_sync();
  else __syncthreads();
  // ---- the key of rank `budget`, from its top bits down
  uint32_t border = 0u, need = static_cast<uint32_t>(a.budget);     // ranks still to be found at or below `border`'s bits
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? kBins / 2 : kBins;
    const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    uint32_t *own = s_own + pass * kBins, *all = s_all + pass * kBins;
#pragma unroll 1
    for (int32_t at = j0; at < j1; at += kChunk) {
      if (!once) load(at);
#pragma unroll
      for (int e = 0; e < kHold; ++e) {
        if (at + e * kThreads >= j1) break;
        if (at + e * kThreads + tid < j1 && (key[e] & above) == border) atomicAdd(own + ((key[e] >> shift) & (bins - 1)), 1u);
      }
    }
    __syncthreads();
    // a thread's bins, the largest first; a cluster's are added up in its first CTA, where most are empty
    const int top = bins - kOwn - kOwn * tid;
    uint32_t cnt[kOwn] = {};
    if (C > 1) {
      const uint32_t sum = mapa_shared(smem_addr(all), 0u);
      for (int i = tid; i < bins; i += kThreads)
        if (own[i] != 0u) add_shared_cluster(sum + 4 * i, own[i]);
      cluster_sync();
      if (top >= 0)
#pragma unroll
        for (int e = 0; e < kOwn; e += 2) ld_shared_cluster_u2(sum + 4 * (top + e), cnt[e], cnt[e + 1]);
    } else if (top >= 0) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e) cnt[e] = own[top + e];
    }
    uint32_t mine = 0u;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) mine += cnt[e];
    const uint32_t before = sum_before(mine, s_scan);
    if (before < need && need <= before + mine) {
      uint32_t at = before;
#pragma unroll
      for (int e = kOwn - 1; e >= 0; --e) {
        if (at < need && need <= at + cnt[e]) {
          s_pick[0] = static_cast<uint32_t>(top + e);
          s_pick[1] = at;
        }
        at += cnt[e];
      }
    }
    __syncthreads();
    border |= s_pick[0] << shift;
    need -= s_pick[1];
    __syncthreads();
  }
  // ---- positions kept: every key above the border, and the first `need` at it
  uint32_t g0 = 0u, e0 = 0u;                                // above and at the border, before this CTA's stretch
  if (C > 1) {
    uint32_t gt = 0u, eq = 0u;
#pragma unroll 1
    for (int32_t at = j0; at < j1; at += kChunk) {
      if (!once) load(at);
#pragma unroll
      for (int e = 0; e < kHold; ++e) {
        if (at + e * kThreads >= j1) break;
        const bool live = at + e * kThreads + tid < j1;
        gt += live && key[e] > border;
        eq += live && key[e] == border;
      }
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    // to the CTAs behind this one
    if (lane < 2)
      for (int r = rank + 1; r < C; ++r) add_shared_cluster(mapa_shared(smem_addr(s_before + lane), static_cast<uint32_t>(r)), lane == 0 ? gt : eq);
    cluster_sync();
    g0 = s_before[0];
    e0 = s_before[1];
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
  for (int32_t at = j0; at < j1; at += kChunk) {
    if (!once) load(at);
    if (tid < kCounts) s_above[tid] = s_at[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kHold; ++e) {
      if (at + e * kThreads >= j1) break;
      const bool live = at + e * kThreads + tid < j1;
      const uint32_t mg = __ballot_sync(0xffffffffu, live && key[e] > border), me = __ballot_sync(0xffffffffu, live && key[e] == border);
      if (lane == 0) {
        s_above[e * kWarps + warp] = __popc(mg);
        s_at[e * kWarps + warp] = __popc(me);
      }
    }
    __syncthreads();
    const uint32_t ng = tid < kCounts ? s_above[tid] : 0u, ne = tid < kCounts ? s_at[tid] : 0u;
    const uint32_t bg = sum_before(ng, s_scan), be = sum_before(ne, s_scan);
    if (tid < kCounts) {
      s_above[tid] = g0 + bg;
      s_at[tid] = e0 + be;
    }
    if (tid == kThreads - 1) {                              // for the next chunk
      s_pick[0] = g0 + bg + ng;
      s_pick[1] = e0 + be + ne;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kHold; ++e) {
      if (at + e * kThreads >= j1) break;
      const int32_t j = at + e * kThreads + tid;
      const bool more = j < j1 && key[e] > border, same = j < j1 && key[e] == border;
      const uint32_t mg = __ballot_sync(0xffffffffu, more), me = __ballot_sync(0xffffffffu, same);
      const uint32_t ge = s_above[e * kWarps + warp] + __popc(mg & below), ee = s_at[e * kWarps + warp] + __popc(me & below);
      if (more || (same && ee < need)) kept[ge + (ee < need ? ee : need)] = j;
    }
    g0 = s_pick[0];
    e0 = s_pick[1];
    __syncthreads();
  }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, Find<kThreads>::kCtasPerSm) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  const int C = static_cast<int>(gridDim.x), rank = static_cast<int>(cluster_ctarank());      // a cluster a (sequence, head)
  const int item = static_cast<int>(blockIdx.y), b = item / a.c.heads, h = item - b * a.c.heads;
  griddep_launch_dependents();
  griddep_wait();
  const int32_t n = length_of(a, b);
  if (rank == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = n < a.budget ? n : a.budget;
  if (n > a.budget) find_kept<kThreads>(a, C, rank, h, n, a.table + b * a.ld_table, a.kept + item * a.cap);
}

// S blocks (blockIdx.z) take a share of every row's pieces each, and S times the ranks at a time: in place, where only a cluster's
// CTAs work on a (sequence, head) and each round waits for all of them, few items leave most SMs idle and take many rounds.
template <int D, bool kInPlace, int S>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kPieces = D / 16;                           // 16-byte pieces of a row's keys, and of its values
  constexpr int kMine = 2 * kPieces / S, kTokens = kMoveTokens * S;
  constexpr int kStep = kMoveThreads / kMine;               // rows that the block holds a piece a thread of
  constexpr int kUnroll = kTokens / kStep;
  static_assert(S == 1 ? kMoveThreads >= 3 * kTokens : kMoveThreads == kTokens && S >= 3, "a thread a scale or sum");
  __shared__ int64_t s_src[kTokens][3], s_dst[kTokens][3];    // offsets of codes, scales and sums; -1: none
  const int item = static_cast<int>(blockIdx.y), b = item / a.c.heads, h = item - b * a.c.heads;
  const int tid = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();
  const int32_t n = length_of(a, b);
  const bool whole = n <= a.budget;
  if (kInPlace && whole) return;                            // (all of a cluster)
  const int32_t m = whole ? n : a.budget;
  const int32_t* kept = a.kept + item * a.cap;
  const int32_t step = static_cast<int32_t>(gridDim.x) * kTokens;
  const int piece = static_cast<int>(blockIdx.z) * kMine + tid % kMine, r0 = tid / kMine;
  uint8_t* const codes = (piece < kPieces ? a.c.k : a.c.v) + (piece % kPieces) * 16;
  // in place every CTA of the cluster takes part in each round's barrier
  for (int32_t i0 = 0; i0 < m; i0 += step) {
    const int32_t base = i0 + static_cast<int32_t>(blockIdx.x) * kTokens;
    if (!kInPlace && base >= m) break;
    if (tid < kTokens) {
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
    const int what = S == 1 ? tid / kTokens : static_cast<int>(blockIdx.z), ri = tid % kTokens;      // key scales, value scales, sums
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

// x (and z times) blocks for each (sequence, head), the x as a cluster or not.
template <typename F>
cudaError_t launch(F* f, int x, int items, int z, bool cluster, int threads, const EvictArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(x, items, z);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(x), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster && x > 1 ? 2 : 1;
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
  // (one sequence's table may come with any stride, whose rows nobody looks for)
  const bool in_place =
      p->out_table == nullptr || (p->out_table == p->block_table && (p->batch == 1 || p->ld_out == p->ld_table));
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
  // Small CTAs where there are more (sequence, head)s than SMs, or few keys; else large ones, in clusters where the keys are more
  // than one holds and SMs are left (see Find).
  cudaError_t e;
  if (items > sms || p->max_kv_len <= 2048) {
    e = launch(evict_select_kernel<256>, 1, items, 1, false, 256, a, cs);
  } else {
    int cluster = 1;
    while (cluster < kMaxCluster && 2 * items * cluster <= sms && p->max_kv_len > static_cast<int64_t>(cluster) * Find<1024>::kChunk)
      cluster *= 2;
    e = launch(evict_select_kernel<1024>, cluster, items, 1, true, 1024, a, cs);
  }
  if (e == cudaSuccess && most > 0 && (!in_place || a.cap > 0)) {
    const int blocks = static_cast<int>((most + kMoveTokens - 1) / kMoveTokens);
    // (8 heads of 60000 tokens to 8192 in place, with the search: 53 us with one share, 32 with four; 512 items of up to 8000 to 2048: 103
    // and 136)
    const bool few = items * kMoveCluster < 2 * sms;
    if (!in_place) {
      auto f = a.c.dim == 128 ? evict_move_kernel<128, false, 1> : evict_move_kernel<64, false, 1>;
      e = launch(f, blocks, items, 1, false, kMoveThreads, a, cs);
    } else {
      auto f = a.c.dim == 128 ? (few ? evict_move_kernel<128, true, 4> : evict_move_kernel<128, true, 1>)
                              : (few ? evict_move_kernel<64, true, 4> : evict_move_kernel<64, true, 1>);
      e = launch(f, kMoveCluster, items, few ? 4 : 1, true, kMoveThreads, a, cs);
    }
  }
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache evict launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
