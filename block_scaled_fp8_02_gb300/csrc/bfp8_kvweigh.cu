// bfp8_kvweigh.cu -- the attention weight that every cached token receives from
// the new tokens of a call, summed over them and over the query heads of a kv
// head: the C entry points, and the kernel for few new tokens a sequence.
//
//   a[h, j] = sum over query heads of kv head h, over new tokens i that see j, of exp(scale q_i . k_j - lse_i)
//
// With at most 16 rows (new tokens x heads of a kv head) it is bound by reading
// the keys once.  The units (32 tokens of a sequence and kv head, 16 where a page has no more) of all
// sequences form one line; CTAs take equal shares of it and their warps turns in
// it, each by itself: a token's sum is one warp's, so that nothing is joined.
// The tokens are the 16-row operand of mma.sync.m16n8k16 (f16, fp32 sums), the
// query rows its 8 columns.  A lane reads 16 codes of a token at a time and makes
// f16 of them (exact); the contraction's slots hold a permutation of it that makes these
// reads whole.  Queries are scaled by a power of two a row (exact in f16 to 2^-37
// of its largest).  Units come by asynchronous copies, each lane into places that
// it alone reads, so that a warp has several on their way, waits for nobody else and
// holds none in registers (a unit on its way in registers: 127 us for 64 sequences of up
// to 8000 tokens, 64 / 8 heads of 128).
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kItemCost = 8;               // places of a (sequence, head) in the line besides its units
constexpr int kCtasPerSm = 2;

// A sequence as the scheduler sees it: tokens [t0, t1) have sums to be written.
struct SeqWork {
  int64_t row0;
  int32_t q_len, kv_len, pos0;
  int32_t t0;
  int32_t units;                           // of each kv head; 0: not this kernel's
};

template <int U>
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
    w.units = (s.kv_len + U - 1) / U - w.t0 / U;
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

template <int D, int U>
struct FewCfg {
  static constexpr int kHalves = U / 16;                           // a unit's 16 tokens, of an MMA
  static constexpr int kKeys = U * D;
  static constexpr int kStages = D == 128 ? (U == 32 ? 3 : 5) : (U == 32 ? 5 : 8);      // units of a warp on their way
  static constexpr int kOffKs = kKeys;                             // scales of tokens g and g + 8 of each half and lane
  static constexpr int kOffOld = kOffKs + kHalves * 2 * 32 * 4;    // the sum so far of the token that the lane writes
  static constexpr int kStage = kOffOld + 32 * 4;
  static constexpr int kSmem = kWarps * kStages * kStage;
  static_assert(kCtasPerSm * (kSmem + 2560) <= 228 * 1024, "shared memory of the CTAs of a SM");
};

// 16 or 4 bytes into shared memory, zeros in place of a source that is not there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where a warp is in the line: an item, and what does not change within it.
struct Cursor {
  int b, h;
  int64_t item0;          // line position of the item's first unit
  int32_t units, t0, kv_len, pos0;
  int32_t k, end;         // the warp's next unit of it; those of it in the share
  const uint8_t* keys;    // of this lane, in page 0
  const float* scales;
  const float* sums;
};
// A unit: its first token and its page; b < 0: none.
struct Unit {
  int b, h;
  int32_t tok, page;
};

template <int D, int NG, int U>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) weigh_few_kernel(const __grid_constant__ WeighArgs p) {
  using C = FewCfg<D, U>;
  constexpr int NH = C::kHalves;
  constexpr int kRows = NG * 8;
  constexpr int KC = D / 64;               // 16-byte key chunks a lane reads of a token
  const AttnArgs& a = p.a;
  extern __shared__ __align__(16) uint8_t few_smem[];
  __shared__ int64_t part[kWarps];
  __shared__ Unit units[kWarps][C::kStages];
  __shared__ int64_t s_before;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int H = a.c.heads;
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's share [u0, u1) of the line of units, and where it starts
  int64_t run = 0, incl0 = 0;
  int32_t n0 = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    n0 = b < a.batch ? line_cost(seq_work<U>(p, b, kRows).units) : 0;
    incl0 = block_scan(n0, part);
    if (tid == kThreads - 1) part[0] = incl0;
    __syncthreads();
    run += part[0];
    __syncthreads();
  }
  const int64_t total = run * H;
  const int64_t want = (total + kWarps - 1) / kWarps, ctas = want < gridDim.x ? want : gridDim.x;
  if (blockIdx.x >= ctas) return;
  const int64_t u0 = share_begin(blockIdx.x, total, ctas), u1 = share_begin(blockIdx.x + 1, total, ctas);
  auto find = [&](int b, int64_t incl, int32_t n) {
    if (n > 0 && (incl - n) * H <= u0 && u0 < incl * H) {
      s_b = b;
      s_before = (incl - n) * H;
    }
  };
  if (a.batch <= kThreads) {
    find(tid, incl0, n0);
  } else {
    run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      const int b = b0 + tid;
      const int32_t n = b < a.batch ? line_cost(seq_work<U>(p, b, kRows).units) : 0;
      const int64_t incl = run + block_scan(n, part);
      find(b, incl, n);
      if (tid == kThreads - 1) part[0] = incl;
      __syncthreads();
      run = part[0];
      __syncthreads();
    }
  }
  __syncthreads();

  // the token whose sum this lane writes (units of 16: lanes t = 0 and 1)
  const int out = g + 8 * t;
  Cursor c{};
  auto enter_head = [&]() {
    c.end = static_cast<int32_t>(c.item0 + c.units < u1 ? c.units : u1 - c.item0);
    c.keys = a.c.k + c.h * a.c.st_head + g * a.c.st_tok + 16 * t;
    c.scales = a.c.ks + c.h * a.c.ss_head + g;
    c.sums = p.w + c.h * p.ws_head + out;
  };
  auto enter = [&](int b) {
    const SeqWork w = seq_work<U>(p, b, kRows);
    c.b = b;
    c.units = w.units;
    c.t0 = w.t0;
    c.kv_len = w.kv_len;
    c.pos0 = w.pos0;
  };
  enter(s_b);
  c.h = static_cast<int>((u0 - s_before) / line_cost(c.units));
  c.item0 = s_before + static_cast<int64_t>(c.h) * line_cost(c.units);
  c.k = static_cast<int32_t>(u0 - c.item0) + warp;
  enter_head();
  // the warp's next unit, its page's number asked for
  auto locate = [&]() {
    Unit n;
    n.b = -1;
    n.h = n.tok = n.page = 0;
    while (c.k >= c.end) {
      const int32_t cost = line_cost(c.units);
      if (c.item0 + cost >= u1) return n;
      while (c.k < cost) c.k += kWarps;                              // the places behind the item
      c.k -= cost;
      c.item0 += cost;
      if (++c.h == H) {
        c.h = 0;
        do {
          enter(c.b + 1);
        } while (c.units == 0);
      }
      enter_head();
    }
    n.b = c.b;
    n.h = c.h;
    n.tok = (c.t0 / U + c.k) * U;
    n.page = __ldg(a.table + c.b * a.ld_table + (n.tok >> a.c.page_shift));
    c.k += kWarps;
    return n;
  };
  uint8_t* const ring = few_smem + warp * (C::kStages * C::kStage);
  const uint32_t ring_at = smem_addr(ring);
  // starts the copies of the unit located last: keys, their scales, the sum to be added to
  auto fetch = [&](Unit& n, int slot) {
    if (n.b >= 0) {
      if (n.page < 0 || n.page >= a.c.num_pages) {
        if (lane == 0) report_failure(a.err, kDevBadCacheIndex);
        n.page = -1;
      }
      const bool there = n.page >= 0;
      const int64_t page = there ? n.page : 0;
      const int off = n.tok & (a.c.page_size - 1);
      const uint8_t* keys = c.keys + page * a.c.st_page + off * a.c.st_tok;
      const float* scales = c.scales + page * a.c.ss_page + off;
      const uint32_t at = ring_at + slot * C::kStage;
      // (a whole unit, which most are, needs none of the comparisons)
      const bool all = there && n.tok + U <= c.kv_len;
#pragma unroll
      for (int r = 0; r < 2 * NH; ++r) {                             // tokens 8 r + g
        const bool live = all || (there && n.tok + 8 * r + g < c.kv_len);
#pragma unroll
        for (int h = 0; h < KC; ++h) copy16(at + ((r * KC + h) * 32 + lane) * 16, keys + 8 * r * a.c.st_tok + 64 * h, live);
        copy4(at + C::kOffKs + (r * 32 + lane) * 4, scales + 8 * r, live);
      }
      const int32_t j = n.tok + out;
      if (t < 2 * NH)
        copy4(at + C::kOffOld + lane * 4, c.sums + page * p.ws_page + off, there && j < c.kv_len && !begins_here(p, j, c.pos0));
    }
    if (lane == 0) units[warp][slot] = n;
    copies_end();
  };

  // ---- the queries at hand: rows grp * 8 + g, f16 after scaling by a power of two
  uint32_t qf[NG][KC * 4][2];
  float cq[NG][2], bias[NG][2];            // of the rows 8 grp + 2 t, + 1: factor of the score, -lse in powers of two
  int32_t lo[NG][2], hi[NG][2];            // tokens that they see
  int q_b = -1, q_h = -1;
  int32_t q_t0 = 0, q_end = 0;             // the tokens of the sequence whose sums are written
  int32_t all_lo = 0, all_hi = 0;          // those that all kRows rows see
  auto queries = [&](const Unit& n) {
    q_b = n.b;
    q_h = n.h;
    const SeqWork w = seq_work<U>(p, n.b, kRows);
    q_t0 = w.t0;
    q_end = w.kv_len;
    const int rows = w.q_len * a.group;
    {
      int32_t x;
      seen_range(a, w.kv_len, w.pos0 + w.q_len - 1, all_lo, x);
      seen_range(a, w.kv_len, w.pos0, x, all_hi);
      if (rows < kRows) all_hi = 0;
    }
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

  auto compute = [&](const Unit& n, int slot) {
    if (n.b != q_b || n.h != q_h) queries(n);
    const uint8_t* at = ring + slot * C::kStage;
    const float* sc = reinterpret_cast<const float*>(at + C::kOffKs) + lane;
    float s[NH][NG][KC][4];
#pragma unroll
    for (int e = 0; e < NH; ++e)
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int h = 0; h < KC; ++h) s[e][grp][h][0] = s[e][grp][h][1] = s[e][grp][h][2] = s[e][grp][h][3] = 0.f;
#pragma unroll
    for (int h = 0; h < KC; ++h)
#pragma unroll
      for (int e = 0; e < NH; ++e) {
        const uint4 ka = *reinterpret_cast<const uint4*>(at + ((2 * e * KC + h) * 32 + lane) * 16),
                    kb = *reinterpret_cast<const uint4*>(at + (((2 * e + 1) * KC + h) * 32 + lane) * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t wa = x == 0 ? ka.x : x == 1 ? ka.y : x == 2 ? ka.z : ka.w;
          const uint32_t wb = x == 0 ? kb.x : x == 1 ? kb.y : x == 2 ? kb.z : kb.w;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16(wa, a0, a2);
          e4m3x4_to_f16(wb, a1, a3);
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
            mma_f16_16x8x16(s[e][grp][h], a0, a1, a2, a3, qf[grp][h * 4 + x][0], qf[grp][h * 4 + x][1]);
        }
      }
    const bool all = n.tok >= all_lo && n.tok + U <= all_hi;
    float sum[2 * NH];                                               // of tokens 8 r + g
#pragma unroll
    for (int r = 0; r < 2 * NH; ++r) {
      const float ks = sc[32 * r];
      const int32_t j = n.tok + 8 * r + g;
      sum[r] = 0.f;
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int i = 2 * (r & 1) + x;
          float v = s[r >> 1][grp][0][i];
          if constexpr (KC == 2) v += s[r >> 1][grp][1][i];
          v = ex2(fmaf(v, ks * cq[grp][x], bias[grp][x]));
          if (!all && (j < lo[grp][x] || j >= hi[grp][x])) v = 0.f;
          sum[r] += v;
        }
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    const int32_t j = n.tok + out;
    float mine = t == 0 ? sum[0] : sum[1];
    if constexpr (NH == 2) mine = t < 2 ? mine : t == 2 ? sum[2] : sum[3];
    if (t < 2 * NH && n.page >= 0 && j >= q_t0 && j < q_end)
      p.w[n.page * p.ws_page + n.h * p.ws_head + (j & (a.c.page_size - 1))] = reinterpret_cast<const float*>(at + C::kOffOld)[lane] + mine;
  };

  // a unit's page number is asked for a turn before its copies start
  Unit next = locate();
  int slot = 0;
  for (int i = 0; i < C::kStages - 1; ++i) {
    fetch(next, i);
    next = locate();
  }
  while (true) {
    copies_wait<C::kStages - 2>();
    __syncwarp();                                                    // lane 0's note of the unit, and the slot read last
    const Unit n = units[warp][slot];
    if (n.b < 0) break;
    const int free = slot == 0 ? C::kStages - 1 : slot - 1;
    fetch(next, free);
    next = locate();
    compute(n, slot);
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
  }
  copies_wait<0>();
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

namespace {

template <int D, int NG, int U>
cudaError_t launch_few(const WeighArgs& p, int ctas, cudaStream_t stream) {
  using C = FewCfg<D, U>;
  cudaError_t e = cudaFuncSetAttribute(weigh_few_kernel<D, NG, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * kCtasPerSm));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_few_kernel<D, NG, U>, p);
}

template <int U>
cudaError_t launch_few_of(const WeighArgs& p, int groups, int ctas, cudaStream_t stream) {
  if (p.a.c.dim == 128) return groups == 1 ? launch_few<128, 1, U>(p, ctas, stream) : launch_few<128, 2, U>(p, ctas, stream);
  return groups == 1 ? launch_few<64, 1, U>(p, ctas, stream) : launch_few<64, 2, U>(p, ctas, stream);
}

}  // namespace

// (64 sequences of up to 8000 tokens on pages of 64, 64 / 8 heads of 128: 67.8 us in units of 16, 64.6 in units of 32)
cudaError_t launch_weigh_few(const WeighArgs& p, int groups, int ctas, cudaStream_t stream) {
  return p.a.c.page_size >= 32 ? launch_few_of<32>(p, groups, ctas, stream) : launch_few_of<16>(p, groups, ctas, stream);
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
