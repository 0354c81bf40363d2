// bfp8_kvweigh.cu -- the attention weight that every cached token receives from
// the new tokens of a call, summed over them and over the query heads of a kv
// head: the C entry points, and the kernel for few new tokens a sequence.
//
//   a[h, j] = sum over query heads of kv head h, over new tokens i that see j, of exp(scale q_i . k_j - lse_i)
//
// With at most 16 rows (new tokens x heads of a kv head) it is bound by reading
// the keys once.  The units (32 tokens of a sequence and kv head) of all
// sequences form one line; CTAs take equal shares of it and their warps turns in
// it, each by itself: a token's sum is one warp's, so that nothing is joined.
// The tokens are the 16-row operand of mma.sync.m16n8k16 (f16, fp32 sums), the
// query rows its 8 columns.  A lane reads 16 codes of a token at a time straight
// from the cache and makes f16 of them (exact); the contraction's slots hold a
// permutation of it that makes these reads whole.  Queries are scaled by a power of two
// a row (exact in f16 to 2^-37 of its largest).  The next unit's
// keys and the page numbers of the one behind it are on their way meanwhile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_attn_math.cuh"
#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_kvweigh.cuh"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kUnit = 32;                  // tokens of a unit
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kItemCost = 4;               // places of a (sequence, head) in the line besides its units
constexpr int kSeqCache = 32;              // sequences whose lengths a CTA keeps in shared memory
constexpr int kCtasPerSm = 2;

// A sequence as the scheduler sees it: tokens [t0, t1) have sums to be written.
struct SeqWork {
  int64_t row0;
  int32_t q_len, kv_len, pos0;
  int32_t t0;
  int32_t units;                           // of each kv head; 0: not this kernel's
};

__device__ __forceinline__ SeqWork seq_work(const WeighArgs& p, int b, int max_rows) {
  const SeqLens s = seq_lens(p.a, b);
  SeqWork w;
  w.row0 = s.row0;
  w.q_len = s.q_len;
  w.kv_len = s.kv_len;
  w.pos0 = s.kv_len - s.q_len;
  int32_t lo, hi;
  seen_range(p.a, s.kv_len, w.pos0, lo, hi);
  if (lo > s.kv_len) lo = s.kv_len;
  w.t0 = p.add != 0 ? lo : 0;
  w.units = 0;
  if (s.q_len > 0 && static_cast<int64_t>(s.q_len) * p.a.group <= max_rows)
    w.units = (s.kv_len + kUnit - 1) / kUnit - w.t0 / kUnit;
  return w;
}
__device__ __forceinline__ int32_t line_cost(int32_t units) { return units > 0 ? units + kItemCost : 0; }

// Inclusive sum over the block's threads (all call it).
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += part[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ void mma_f16_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where a warp is in the line.
struct Cursor {
  int b, h;
  int64_t item0;          // line position of the item's first unit
  SeqWork w;
};
// A unit on its way: its first token, and its pages (of each half; one page where a page holds both).
struct Unit {
  int b, h;
  int32_t tok;
  int32_t page[2];
  bool live;
};

template <int D, int NG>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) weigh_few_kernel(const __grid_constant__ WeighArgs p) {
  constexpr int kRows = NG * 8;
  constexpr int KC = D / 64;               // 16-byte key chunks a lane reads of a token
  const AttnArgs& a = p.a;
  __shared__ int64_t part[kWarps];
  __shared__ SeqWork seqs[kSeqCache];
  __shared__ int64_t s_before;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int H = a.c.heads;
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's share [u0, u1) of the line of units, and where it starts
  int64_t run = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const int64_t incl = block_scan(b < a.batch ? line_cost(seq_work(p, b, kRows).units) : 0, part);
    if (tid == kThreads - 1) part[0] = incl;
    __syncthreads();
    run += part[0];
    __syncthreads();
  }
  const int64_t total = run * H;
  const int64_t want = (total + kWarps - 1) / kWarps, ctas = want < gridDim.x ? want : gridDim.x;
  if (blockIdx.x >= ctas) return;
  const int64_t u0 = share_begin(blockIdx.x, total, ctas), u1 = share_begin(blockIdx.x + 1, total, ctas);
  run = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const int32_t n = b < a.batch ? line_cost(seq_work(p, b, kRows).units) : 0;
    const int64_t incl = run + block_scan(n, part);
    if (n > 0 && (incl - n) * H <= u0 && u0 < incl * H) {
      s_b = b;
      s_before = (incl - n) * H;
    }
    if (tid == kThreads - 1) part[0] = incl;
    __syncthreads();
    run = part[0];
    __syncthreads();
  }
  const int b_first = s_b;
  if (tid < kSeqCache && b_first + tid < a.batch) seqs[tid] = seq_work(p, b_first + tid, kRows);
  __syncthreads();
  auto get_seq = [&](int b) -> SeqWork { return b - b_first < kSeqCache ? seqs[b - b_first] : seq_work(p, b, kRows); };

  Cursor c;
  c.b = b_first;
  c.w = get_seq(c.b);
  c.h = static_cast<int>((u0 - s_before) / line_cost(c.w.units));
  c.item0 = s_before + static_cast<int64_t>(c.h) * line_cost(c.w.units);
  int64_t u = u0 + warp;
  // the warp's next unit, its page numbers asked for
  auto locate = [&]() {
    Unit n{};
    while (u < u1) {
      const int32_t cost = line_cost(c.w.units);
      if (u >= c.item0 + cost) {
        c.item0 += cost;
        if (++c.h == H) {
          c.h = 0;
          do {
            c.w = get_seq(++c.b);
          } while (c.w.units == 0);
        }
        continue;
      }
      const int32_t k = static_cast<int32_t>(u - c.item0);
      u += kWarps;
      if (k >= c.w.units) continue;                                  // the places behind an item
      n.b = c.b;
      n.h = c.h;
      n.tok = (c.w.t0 / kUnit + k) * kUnit;
      n.live = true;
      const int32_t* row = a.table + c.b * a.ld_table;
      n.page[0] = __ldg(row + (n.tok >> a.c.page_shift));
      n.page[1] = n.tok + 16 < c.w.kv_len ? __ldg(row + ((n.tok + 16) >> a.c.page_shift)) : n.page[0];
      break;
    }
    return n;
  };
  // its keys, their scales, and the sum that this lane will write (token 16 (t / 2) + 8 (t % 2) + g)
  struct Data {
    uint4 k[2][2][KC];
    float ks[2][2];
    float old;
  };
  auto sum_at = [&](const Unit& n) -> float* {
    const int32_t j = n.tok + 16 * (t >> 1) + 8 * (t & 1) + g;
    return p.w + n.page[t >> 1] * p.ws_page + n.h * p.ws_head + (j & (a.c.page_size - 1));
  };
  auto fetch = [&](Unit& n, Data& d) {
    if (!n.live) return;
    const SeqWork& w = get_seq(n.b);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (n.page[e] < 0 || n.page[e] >= a.c.num_pages) {
        report_failure(a.err, kDevBadCacheIndex);
        n.page[e] = -1;
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int32_t j = n.tok + 16 * e + 8 * r + g;
        const bool ok = n.page[e] >= 0 && j < w.kv_len;
        const int off = j & (a.c.page_size - 1);
        const uint8_t* src = a.c.k + (ok ? n.page[e] : 0) * a.c.st_page + n.h * a.c.st_head + off * a.c.st_tok + 16 * t;
#pragma unroll
        for (int h = 0; h < KC; ++h)
          d.k[e][r][h] = ok ? __ldg(reinterpret_cast<const uint4*>(src + 64 * h)) : make_uint4(0u, 0u, 0u, 0u);
        d.ks[e][r] = ok ? __ldg(a.c.ks + n.page[e] * a.c.ss_page + n.h * a.c.ss_head + off) : 0.f;
      }
    }
    const int32_t j = n.tok + 16 * (t >> 1) + 8 * (t & 1) + g;
    d.old = n.page[t >> 1] >= 0 && j >= w.t0 && j < w.kv_len && !begins_here(p, j, w.pos0) ? *sum_at(n) : 0.f;
  };

  // ---- the queries at hand: rows grp * 8 + g, f16 after scaling by a power of two
  uint32_t qf[NG][KC * 4][2];
  float cq[NG][2], bias[NG][2];            // of the rows 8 grp + 2 t, + 1: factor of the score, -lse in powers of two
  int32_t lo[NG][2], hi[NG][2];            // tokens that they see
  int q_b = -1, q_h = -1;
  auto queries = [&](const Unit& n, const SeqWork& w) {
    q_b = n.b;
    q_h = n.h;
    const int rows = w.q_len * a.group;
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      const int r = grp * 8 + g, i = r / a.group;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (w.row0 + i) * a.q_st + (n.h * a.group + r - i * a.group) * a.q_sh + 16 * t);
      float f[KC][16], amax = 0.f;
#pragma unroll
      for (int h = 0; h < KC; ++h) {
        uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (r < rows) {
          raw[0] = __ldg(src + 8 * h);
          raw[1] = __ldg(src + 8 * h + 1);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4& v = raw[e >> 2];
          const uint32_t x = (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
          f[h][2 * e] = __uint_as_float(x << 16);
          f[h][2 * e + 1] = __uint_as_float(x & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(f[h][2 * e]), fabsf(f[h][2 * e + 1])));
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // amax * up in [2^13, 2^14); up = 2^(13 - e), in two factors that stay in range
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      if (e < -126) e = -126;
      const int sh = 13 - e, s1 = sh / 2, s2 = sh - s1;
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + s1) << 23);
      const float f2 = __uint_as_float(static_cast<uint32_t>(127 + s2) << 23);
      const float d1 = __uint_as_float(static_cast<uint32_t>(127 - s1) << 23);
      const float d2 = __uint_as_float(static_cast<uint32_t>(127 - s2) << 23);
#pragma unroll
      for (int h = 0; h < KC; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          qf[grp][h * 4 + x][0] = pack_f16x2(f[h][4 * x] * f1 * f2, f[h][4 * x + 1] * f1 * f2);
          qf[grp][h * 4 + x][1] = pack_f16x2(f[h][4 * x + 2] * f1 * f2, f[h][4 * x + 3] * f1 * f2);
        }
      const float back = a.scale * 1.4426950408889634f * d1 * d2;
      cq[grp][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      cq[grp][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rr = grp * 8 + 2 * t + x, ii = rr / a.group;
        lo[grp][x] = hi[grp][x] = 0;
        bias[grp][x] = 0.f;
        if (rr < rows) {
          seen_range(a, w.kv_len, w.pos0 + ii, lo[grp][x], hi[grp][x]);
          bias[grp][x] = a.lse[(w.row0 + ii) * a.heads + n.h * a.group + rr - ii * a.group] * -1.4426950408889634f;
        }
      }
    }
  };

  auto compute = [&](const Unit& n, const Data& d) {
    const SeqWork& w = get_seq(n.b);
    if (n.b != q_b || n.h != q_h) queries(n, w);
    float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    float s[2][NG][KC][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int h = 0; h < KC; ++h) s[e][grp][h][0] = s[e][grp][h][1] = s[e][grp][h][2] = s[e][grp][h][3] = 0.f;
#pragma unroll
    for (int h = 0; h < KC; ++h)
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 &ka = d.k[e][0][h], &kb = d.k[e][1][h];
          const uint32_t wa = x == 0 ? ka.x : x == 1 ? ka.y : x == 2 ? ka.z : ka.w;
          const uint32_t wb = x == 0 ? kb.x : x == 1 ? kb.y : x == 2 ? kb.z : kb.w;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16(wa, a0, a2);
          e4m3x4_to_f16(wb, a1, a3);
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
            mma_f16_16x8x16(s[e][grp][h], a0, a1, a2, a3, qf[grp][h * 4 + x][0], qf[grp][h * 4 + x][1]);
        }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i >> 1, x = i & 1;
          float v = s[e][grp][0][i];
          if constexpr (KC == 2) v += s[e][grp][1][i];
          const int32_t j = n.tok + 16 * e + 8 * r + g;
          v = ex2(fmaf(v, d.ks[e][r] * cq[grp][x], bias[grp][x]));
          if (j >= lo[grp][x] && j < hi[grp][x]) sum[e][r] += v;
        }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[e][r] += __shfl_xor_sync(0xffffffffu, sum[e][r], 1);
        sum[e][r] += __shfl_xor_sync(0xffffffffu, sum[e][r], 2);
      }
    const float mine = (t >> 1) == 0 ? ((t & 1) == 0 ? sum[0][0] : sum[0][1]) : ((t & 1) == 0 ? sum[1][0] : sum[1][1]);
    const int32_t j = n.tok + 16 * (t >> 1) + 8 * (t & 1) + g;
    if (n.page[t >> 1] >= 0 && j >= w.t0 && j < w.kv_len) *sum_at(n) = d.old + mine;
  };

  Unit cur = locate();
  Data dc, dn;
  fetch(cur, dc);
  Unit nxt = locate();
  while (cur.live) {
    fetch(nxt, dn);
    const Unit after = locate();
    compute(cur, dc);
    cur = nxt;
    dc = dn;
    nxt = after;
  }
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

// Rows of a sequence up to which the kernel for few rows takes it, in eights: all sequences when even the longest is
// that short, else those of a single token.  0: none.
constexpr int kFewRows = 16;
int few_groups(int group, int64_t max_q) {
  if (group > kFewRows) return 0;
  return static_cast<int>(((max_q * group <= kFewRows ? max_q * group : group) + 7) / 8);
}
bool has_many(int group, int64_t max_q) { return max_q * group > 8 * few_groups(group, max_q); }

size_t workspace_bytes_for(int group, int max_q, int sms) {
  return kCounterHeaderBytes + (has_many(group, max_q) ? weigh_tile_partial_bytes(sms) : 0);
}

}  // namespace

cudaError_t launch_weigh_few(const WeighArgs& p, int groups, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * kCtasPerSm));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.a.c.dim == 128) return cudaLaunchKernelEx(&cfg, groups == 1 ? weigh_few_kernel<128, 1> : weigh_few_kernel<128, 2>, p);
  return cudaLaunchKernelEx(&cfg, groups == 1 ? weigh_few_kernel<64, 1> : weigh_few_kernel<64, 2>, p);
}

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_kv_cache_weigh_workspace_size(int num_heads, int num_kv_heads, int head_dim, int max_q_len,
                                                          size_t* bytes) {
  bfp8_status st = check_heads(num_heads, num_kv_heads, head_dim, max_q_len);
  if (st != BFP8_OK) return st;
  if (!bytes) return bad("bytes is null");
  int sms = 0;
  int* err = nullptr;
  if ((st = device_for_call(&sms, &err)) != BFP8_OK) return st;
  *bytes = workspace_bytes_for(num_heads / num_kv_heads, max_q_len, sms);
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
  for (int64_t s : {args->q_stride_head, args->q_stride_token, weights_stride_page, weights_stride_head})
    if (s >= (int64_t{1} << 38)) return bad("stride %lld", (long long)s);       // (what a tensor map can hold)
  if (weights_stride_page < p.a.c.page_size || weights_stride_head < p.a.c.page_size)
    return bad("weights strides must be >= page_size");
  if (off_align(weights, 4)) return set_last_errorf(BFP8_ERR_ALIGNMENT, "weights must be 4-byte aligned");
  int sms = 0;
  st = device_for_call(&sms, &p.a.err);
  const size_t need = st == BFP8_OK ? workspace_bytes_for(p.a.group, p.a.max_q, sms) : kCounterHeaderBytes;
  if (!workspace || workspace_bytes < need)
    return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  if (off_align(workspace, 256)) return set_last_errorf(BFP8_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (st != BFP8_OK) return st;
  p.w = weights;
  p.ws_page = weights_stride_page;
  p.ws_head = weights_stride_head;
  p.add = accumulate;
  if (p.a.max_kv == 0) return set_last_error(BFP8_OK, "");
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int groups = few_groups(p.a.group, p.a.max_q);
  p.a.few_rows = 8 * groups;
  const bool many = has_many(p.a.group, p.a.max_q);
  // as for the attention: can a sequence be short enough?
  const bool few = groups > 0 && (!many || p.a.total_q <= static_cast<int64_t>(p.a.batch - 1) * p.a.max_q + p.a.few_rows / p.a.group);
  if (!few) p.a.few_rows = 0;
  cudaError_t e = cudaSuccess;
  if (many) {
    const uint64_t dims[3] = {static_cast<uint64_t>(2 * p.a.c.dim), static_cast<uint64_t>(p.a.heads), static_cast<uint64_t>(p.a.total_q)};
    const uint64_t strides[2] = {static_cast<uint64_t>(2 * p.a.q_sh), static_cast<uint64_t>(2 * p.a.q_st)};
    const uint32_t box[3] = {128u, static_cast<uint32_t>(p.a.group), static_cast<uint32_t>(weigh_tile_tokens(p.a.group, p.a.max_q))};
    CUtensorMap mq;
    if ((st = encode_bytes_tiled(&mq, p.a.q, 3, dims, strides, box, 128)) != BFP8_OK) return st;
    e = launch_weigh_tile(mq, p, sms, static_cast<int32_t*>(workspace),
                          reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterHeaderBytes), cs);
  }
  if (e == cudaSuccess && few) e = launch_weigh_few(p, groups, sms, cs);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache weigh launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
