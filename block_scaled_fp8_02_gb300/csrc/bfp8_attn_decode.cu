// bfp8_attn_decode.cu -- attention of few new tokens a sequence (at most 32
// rows of query heads a kv head) over the paged e4m3 cache: bound by reading
// the cache once.
//
// Work is (sequence, kv head) items of 128-token units, all items' units in one
// line; the persistent CTAs (one a SM) take equal shares of that line, so that
// ragged contexts and single long ones load every SM alike.  Ending an item costs
// a CTA the time of kItemCost units, which lie behind its units in the line.  A CTA computes its
// share from the lengths on the device.  An item cut by a share's border leaves
// fp32 partial outputs in the workspace; the last CTA of it to arrive adds them
// in CTA order (deterministic).
//
// A producer warp streams units through TMA (tensor-map boxes of one page and
// head, 128-byte swizzle, and the pages' scales by bulk copies) into a ring.
// Teams of four warps take units in turn (or, past 16 rows, share the rows), 32 tokens a warp; each warp keeps its
// own running maximum, sum and output.  The tokens are the 16-row operand of
// mma.sync.m16n8k16 (f16, fp32 sums) and the query rows its 8 columns:
//   S^T [16 tokens x 8 rows] = K Q^T,    O^T [D x 8 rows] += V^T P^T.
// The e4m3 codes become f16 in registers (exact, one conversion a pair).  Slots
// of the contraction may hold any permutation of it as long as both operands
// agree, so every fragment is plain 16-byte shared loads: K's lanes read
// neighbouring elements as the contraction slots, V's lanes read four tokens'
// 16 bytes and interleave them by byte permutes; no transposes but the 8 x 8
// movmatrix that turns P^T into the second product's operand.  Token slot g
// holds token g/2 + 4 (g % 2) (D = 128), which keeps both reads free of bank
// conflicts under the swizzle.
//
// Scales: scores x (in powers of two) are multiplied by the key's scale in
// fp32.  A value's scale joins its weight: the second product's f16 operand is
// 2^(x + log2 vs - mv + 7) with mv a running maximum of x + log2 vs, so that it
// keeps 11 bits down to 2^-21 of the largest weighted value whatever the spread
// of the scales; the sum of the weights 2^(x - m) is kept apart, in fp32.
// Queries are scaled by a power of two a row (exact in f16).  m and mv may lag
// by up to 8; they and the accumulators move only when a score passes that (a
// warp vote).
//
// Measured, 64 query over 8 kv heads of 128: 64 sequences of up to 8192 tokens
// (558 MB of cache) 106 us, 5.3 TB/s or 0.78 of the measured copy rate; one of
// 32768 tokens 21.9 us (25 to 29 with the host's call, back to back), of which 10.2 would be the cache's reading and the rest
// is the launch, the first units' latency and the joining of the parts.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "bfp8_attn.cuh"
#include "bfp8_attn_math.cuh"
#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kUnit = 128;                 // tokens of a unit
constexpr int kItemCost = 4;               // (measured: query, joining the warps, output 5000 cycles; a unit 1340)
constexpr int kSeqCache = 32;              // sequences whose lengths a CTA keeps in shared memory
constexpr float kNoMax = -3.0e38f;         // running maximum before any token
constexpr float kLag = 8.f;                // how far scores may exceed the running maximum
constexpr float kLift = 7.f;               // weighted values are 2^(x + log2 vs - mv + kLift) <= 2^15

template <int D, int NG, int RT>
struct DecCfg {
  static constexpr int kCodes = kUnit * D;                 // K or V of a unit
  static constexpr int kStageBytes = 2 * kCodes;
  static constexpr int kScaleFloats = 2 * kUnit;
  static constexpr int kStages = D == 128 ? 6 : 12;
  // Consumers: teams of four warps, 32 tokens a warp, as two chains of 16.  Up to 16 rows (NG eights of
  // them in a warp) the teams take units in turn (RT = 1); more rows than a warp's registers hold are shared out
  // and RT teams work on every unit (one warp with 32 rows spilled: 16 sequences of 4 tokens at 8192,
  // 64 / 8 heads of 128, took 167 us against 103 then, 100 now).  The last warpgroup's first warp produces; registers are handed to the consumers
  // (launch: 128 or 168 a thread).
  static constexpr int kWarps = NG == 1 ? 12 : 8;
  static constexpr int kGroups = kWarps / 4;
  static constexpr int kThreads = (kWarps + 4) * 32;
  static constexpr int kRegs = NG == 1 ? 152 : 224, kRegsProducer = 56;
  // a slot always belongs to the same team, which waits for each of its phases in turn: a wait by parity
  // cannot tell a phase from the one two further on
  static_assert(kStages % kGroups == 0 && (RT == 1 || RT == kGroups), "slots belong to teams, or to all");
  static constexpr int kParts = RT == 1 ? kWarps : 4;      // warps whose parts make up a row
  static constexpr int kPitch = D + 4;                     // floats of a row of partials
  static constexpr int kJoin = 4;                          // rows whose warps' parts are joined at once
  static constexpr int kOffScale = kStages * kStageBytes;
  static constexpr int kOffRed = kOffScale + kStages * kScaleFloats * 4;
  static constexpr int kOffMl = kOffRed + kWarps * kJoin * kPitch * 4;
  static constexpr int kOffSeq = kOffMl + kWarps * kJoin * 3 * 4;
  static constexpr int kOffBar = kOffSeq + kSeqCache * 32;
  static constexpr int kSmem = kOffBar + 2 * kStages * 8 + 64 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// A sequence as the scheduler sees it.
struct SeqWork {
  int32_t units;       // of each kv head; 0: not this kernel's
  int32_t t0, t1;      // tokens some row sees: [t0, t1)
  int32_t q_len;
  int32_t pos0;        // position of the first new token
  int32_t kv_len;
  int64_t row0;
};

__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, int b, int max_rows) {
  const SeqLens s = seq_lens(a, b);
  SeqWork w;
  w.row0 = s.row0;
  w.q_len = s.q_len;
  w.kv_len = s.kv_len;
  w.pos0 = s.kv_len - s.q_len;
  int32_t lo, hi, lo2;
  seen_range(a, s.kv_len, w.pos0, lo, hi);                          // the first row's start
  seen_range(a, s.kv_len, w.pos0 + s.q_len - 1, lo2, hi);           // the last row's end
  w.t0 = lo;
  w.t1 = hi;
  w.units = 0;
  if (s.q_len > 0 && static_cast<int64_t>(s.q_len) * a.group <= max_rows)
    w.units = hi > lo ? (hi + kUnit - 1) / kUnit - lo / kUnit : 1;
  return w;
}

// Length of an item in the line.
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
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Largest over the lanes that share lane % 4.
__device__ __forceinline__ float max_over_g(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum_over_g(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Token a slot holds, and byte offset of a 16-byte chunk in a unit's rows.
template <int D>
__device__ __forceinline__ int slot_token(int g) {
  return D == 128 ? (g >> 1) + 4 * (g & 1) : g;
}
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int row, int c) {
  if constexpr (D == 128) return static_cast<uint32_t>(row * 128 + ((c ^ (row & 7)) << 4));
  else return static_cast<uint32_t>(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

struct DecodeArgs {
  AttnArgs a;
  int32_t* counters;          // one a CTA, zero between calls
  float* partials;            // two slots a CTA: NG * 8 rows of D floats, then their log2 sums
  unsigned long long wait_limit;
  int32_t behind;             // launched right behind the other kernel, for the same call
};

template <int D, int NG, int RT>
__global__ void __launch_bounds__((DecCfg<D, NG, RT>::kThreads), 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ DecodeArgs p) {
  using C = DecCfg<D, NG, RT>;
  constexpr int kRows = NG * 8 * RT;
  const AttnArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset: the compiler has to see that this is shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  auto bar_full = [&](int s) { return sbase + static_cast<uint32_t>(C::kOffBar + 8 * s); };
  auto bar_empty = [&](int s) { return sbase + static_cast<uint32_t>(C::kOffBar + 8 * (C::kStages + s)); };
  SeqWork* seqs = reinterpret_cast<SeqWork*>(smem + C::kOffSeq);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.c.heads;
  __shared__ uint32_t s_spoilt[2];            // rows to become NaN, of the item at hand and the next

  if (tid == 0) {
    s_spoilt[0] = s_spoilt[1] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 4 * RT);
    }
    fence_barrier_init();
  }
  griddep_launch_dependents();
  // Behind the other kernel this one starts once all of its CTAs have passed their wait, on what SMs it leaves,
  // needs nothing of it and only must not be done before it.
  if (!p.behind) griddep_wait();

  // ---- this CTA's share [u0, u1) of the line of units, and where it starts
  __shared__ int64_t part[C::kThreads / 32];
  __shared__ int64_t s_before;
  __shared__ int s_b;
  int64_t run = 0, incl0 = 0;
  SeqWork mine{};                                      // sequence tid of the last chunk of them
  for (int b0 = 0; b0 < a.batch; b0 += C::kThreads) {
    const int b = b0 + tid;
    mine.units = 0;
    if (b < a.batch) mine = seq_work(a, b, kRows);
    incl0 = block_scan(line_cost(mine.units), part);
    if (tid == C::kThreads - 1) part[0] = incl0;
    __syncthreads();
    run += part[0];
    __syncthreads();
  }
  const int64_t total = run * H;
  const int64_t ctas = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= ctas) {                            // whole CTA: nothing is in flight yet
    if (p.behind) griddep_wait();
    return;
  }
  const int64_t u0 = share_begin(blockIdx.x, total, ctas), u1 = share_begin(blockIdx.x + 1, total, ctas);
  auto locate = [&](int b, int64_t incl, int32_t n) {
    if (n > 0 && (incl - n) * H <= u0 && u0 < incl * H) {
      s_b = b;
      s_before = (incl - n) * H;
    }
  };
  if (a.batch <= C::kThreads) {                        // the lengths are in registers
    locate(tid, incl0, line_cost(mine.units));
    __syncthreads();
    if (tid >= s_b && tid < a.batch && tid - s_b < kSeqCache) seqs[tid - s_b] = mine;
  } else {
    run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += C::kThreads) {
      const int b = b0 + tid;
      const int32_t n = b < a.batch ? line_cost(seq_work(a, b, kRows).units) : 0;
      const int64_t incl = run + block_scan(n, part);
      locate(b, incl, n);
      if (tid == C::kThreads - 1) part[0] = incl;
      __syncthreads();
      run = part[0];
      __syncthreads();
    }
    if (tid < kSeqCache && s_b + tid < a.batch) seqs[tid] = seq_work(a, s_b + tid, kRows);
  }
  __syncthreads();
  const int b_first = s_b;
  auto get_seq = [&](int b) -> SeqWork {
    return b - b_first < kSeqCache ? seqs[b - b_first] : seq_work(a, b, kRows);
  };
  // cursor over the share: item (b, h), its units [k0, k1) here, its place in the line
  struct Cursor {
    int b, h;
    int64_t item0;          // line position of the item's first unit
    int32_t k0, k1;
    SeqWork w;
  };
  auto clip = [&](Cursor& c) {                  // false: only the item's end lies in the share
    c.k0 = static_cast<int32_t>(u0 > c.item0 ? u0 - c.item0 : 0);
    c.k1 = static_cast<int32_t>(c.item0 + c.w.units < u1 ? c.w.units : u1 - c.item0);
    return c.k0 < c.k1;
  };
  auto next = [&](Cursor& c) -> bool {          // false: the share is done
    do {
      c.item0 += line_cost(c.w.units);
      if (c.item0 >= u1) return false;
      if (++c.h == H) {
        c.h = 0;
        do {
          c.w = get_seq(++c.b);
        } while (c.w.units == 0);
      }
    } while (!clip(c));
    return true;
  };
  auto start = [&](Cursor& c) -> bool {
    c.b = b_first;
    c.w = get_seq(c.b);
    c.h = static_cast<int>((u0 - s_before) / line_cost(c.w.units));
    c.item0 = s_before + static_cast<int64_t>(c.h) * line_cost(c.w.units);
    return clip(c) || next(c);
  };

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------ producer
    setmaxnreg_dec<C::kRegsProducer>();
    if (warp > C::kWarps) return;
    const int page = a.c.page_size, shift = a.c.page_shift;
    const int ppu = page >= kUnit ? 1 : kUnit / page;            // boxes of a unit
    const int box = page >= kUnit ? kUnit : page;                // tokens of a box
    const uint32_t box_bytes = static_cast<uint32_t>(2 * box * D + 2 * box * 4);
    uint32_t q = 0;
    bool ok = true;
    Cursor c;
    for (bool more = start(c); more && ok; more = next(c)) {
      const int32_t ub = c.w.t0 / kUnit;
      const int32_t* row = a.table + c.b * a.ld_table;
      // table entries of 32 boxes at a time, one a lane
      int32_t cached = -1, entry = 0;
      for (int32_t k = c.k0; k < c.k1 && ok; ++k, ++q) {
        const int32_t tok = (ub + k) * kUnit;
        const int32_t first = tok / box;                         // box numbers of this unit
        if (first / 32 != cached) {
          cached = first / 32;
          const int64_t t = (static_cast<int64_t>(cached) * 32 + lane) * box;
          entry = 0;
          if (t < c.w.t1 && t + box > c.w.t0) {
            entry = __ldg(row + (t >> shift));
            if (entry < 0 || entry >= a.c.num_pages) {
              report_failure(a.err, kDevBadCacheIndex);
              entry = 0;
            }
          }
        }
        const int slot = static_cast<int>(q % C::kStages);
        int free = 1;                                            // one lane waits for the warp
        if (lane == 0)
          free = mbar_wait_bounded(bar_empty(slot), static_cast<uint32_t>((q / C::kStages) & 1) ^ 1u, p.wait_limit);
        if (!__shfl_sync(0xffffffffu, free, 0)) {
          if (lane == 0) report_failure(a.err, kDevTimeoutProducer);
          ok = false;
          break;
        }
        // boxes that hold tokens some row sees
        const int32_t t = tok + lane * box;
        const bool live = lane < ppu && t < c.w.t1 && t + box > c.w.t0;
        const int n = __popc(__ballot_sync(0xffffffffu, live));
        if (lane == 0) mbar_arrive_expect_tx(bar_full(slot), n * box_bytes);
        const int32_t pg = __shfl_sync(0xffffffffu, entry, (first + lane) & 31);
        __syncwarp();
        if (live) {
          const int off = t & (page - 1);
          const uint32_t kd = sbase + static_cast<uint32_t>(slot * C::kStageBytes + lane * box * D);
          tma_load_4d(kd, &tmK, bar_full(slot), 0, off, c.h, pg);
          tma_load_4d(kd + C::kCodes, &tmV, bar_full(slot), 0, off, c.h, pg);
          const int64_t so = pg * a.c.ss_page + c.h * a.c.ss_head + off;
          const uint32_t sd = sbase + static_cast<uint32_t>(C::kOffScale + slot * C::kScaleFloats * 4 + lane * box * 4);
          bulk_load(sd, a.c.ks + so, box * 4, bar_full(slot));
          bulk_load(sd + kUnit * 4, a.c.vs + so, box * 4, bar_full(slot));
        }
      }
    }
    // no copy may still be landing in shared memory when the CTA exits
    for (uint32_t i = q > C::kStages ? q - C::kStages : 0; i < q; ++i)
      if (!mbar_wait_bounded(bar_full(static_cast<int>(i % C::kStages)), static_cast<uint32_t>((i / C::kStages) & 1),
                             p.wait_limit)) {
        if (lane == 0) report_failure(a.err, kDevTimeoutTail);
        break;
      }
    return;
  }

  // ------------------------------------------------------------- consumers
  setmaxnreg_inc<C::kRegs>();
  const int team = warp >> 2, wq = warp & 3;         // units team, team + kGroups .. ; 32 tokens of each
  const int row0 = RT == 1 ? 0 : team * 8 * NG;      // first row of this team
  const int g = lane >> 2, t = lane & 3;
  const int pg = slot_token<D>(g);
  // value chunk and tokens of this lane
  const int v_tok[4] = {slot_token<D>(2 * t), slot_token<D>(2 * t + 1), slot_token<D>(2 * t) + 8,
                        slot_token<D>(2 * t + 1) + 8};
  constexpr int KC = D / 64;                 // 16-byte key chunks a lane reads of a token
  constexpr int DT = D / 16;                 // 16-element tiles of the output
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);
  float* red_m = reinterpret_cast<float*>(smem + C::kOffMl);
  float* red_l = red_m + C::kWarps * C::kJoin;
  float* red_v = red_l + C::kWarps * C::kJoin;
  __shared__ int s_last;
  bool ok = true;
  uint32_t q = 0, item = 0;
  // the rows row0 + grp * 8 + g of an item's queries, this lane's elements; fetched while the item before ends
  uint4 raw[NG][KC][2];
  auto fetch = [&](const Cursor& c) {
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      const int r = row0 + grp * 8 + g, i = r / a.group;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (c.w.row0 + i) * a.q_st +
                                                        (c.h * a.group + r - i * a.group) * a.q_sh + 16 * t);
#pragma unroll
      for (int h = 0; h < KC; ++h) {
        raw[grp][h][0] = raw[grp][h][1] = make_uint4(0u, 0u, 0u, 0u);
        if (r < c.w.q_len * a.group) {
          raw[grp][h][0] = __ldg(src + 8 * h);
          raw[grp][h][1] = __ldg(src + 8 * h + 1);
        }
      }
    }
  };
  Cursor c;
  bool more = start(c);
  if (more) fetch(c);
  while (more) {
    const SeqWork w = c.w;
    const int rows = w.q_len * a.group;
    // ---- queries: rows row0 + grp * 8 + g, f16 after scaling by a power of two
    uint32_t qf[NG][KC * 4][2];
    float cq[NG][2];
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      float amax = 0.f;
      float f[KC][16];
#pragma unroll
      for (int h = 0; h < KC; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4& u = raw[grp][h][i >> 2];
          const uint32_t x = (i & 3) == 0 ? u.x : (i & 3) == 1 ? u.y : (i & 3) == 2 ? u.z : u.w;
          f[h][2 * i] = __uint_as_float(x << 16);
          f[h][2 * i + 1] = __uint_as_float(x & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(f[h][2 * i]), fabsf(f[h][2 * i + 1])));
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
        for (int i = 0; i < 4; ++i) {
          qf[grp][h * 4 + i][0] = pack_f16x2(f[h][4 * i] * f1 * f2, f[h][4 * i + 1] * f1 * f2);
          qf[grp][h * 4 + i][1] = pack_f16x2(f[h][4 * i + 2] * f1 * f2, f[h][4 * i + 3] * f1 * f2);
        }
      // (an infinite query: every score a NaN, also where all products happen to be of one sign)
      const float back = e > 127 ? __uint_as_float(0x7FFFFFFFu) : a.scale * 1.4426950408889634f * d1 * d2;
      cq[grp][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      cq[grp][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
    // tokens every row sees: no mask between them
    int32_t full_lo, full_hi, x_lo, x_hi;
    seen_range(a, w.kv_len, w.pos0 + w.q_len - 1, full_lo, x_hi);
    seen_range(a, w.kv_len, w.pos0, x_lo, full_hi);

    float acc[NG][DT][4];
    float m[NG][2], mv[NG][2], l[NG][2];
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      m[grp][0] = m[grp][1] = mv[grp][0] = mv[grp][1] = kNoMax;
      l[grp][0] = l[grp][1] = 0.f;
#pragma unroll
      for (int j = 0; j < DT; ++j) acc[grp][j][0] = acc[grp][j][1] = acc[grp][j][2] = acc[grp][j][3] = 0.f;
    }
    const int32_t ub = w.t0 / kUnit;
    // this warp's 32 tokens of a unit as NU times 16, whose chains of dependent steps overlap
    // (tokens that every row sees have a copy of their own, without the masks: 16 sequences of 3 tokens at 8192, 64 / 8
    // heads of 128, 88 us against 96 in one; 16 of 4 102 against 103.5; batches of one token 105 against 107)
    auto process = [&](int32_t k, auto masked) {
      constexpr bool edge = decltype(masked)::value;
      constexpr int NU = 2;
      int32_t base[NU];
      const uint8_t *kst[NU], *vst[NU];
      float ks[NU][2], lv[NU][2];
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int slot = static_cast<int>(q % C::kStages), at = wq * 32 + 16 * u;
        base[u] = (ub + k) * kUnit + at;
        kst[u] = smem + slot * C::kStageBytes + at * D;
        vst[u] = kst[u] + C::kCodes;
        const float* sc = reinterpret_cast<const float*>(smem + C::kOffScale) + slot * C::kScaleFloats + at;
        ks[u][0] = sc[pg];
        ks[u][1] = sc[pg + 8];
        lv[u][0] = lg2(sc[kUnit + pg]);
        lv[u][1] = lg2(sc[kUnit + pg + 8]);
      }
      // ---- scores
      float s[NU][NG][4];
      {
        float part[NU][NG][KC][4];
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int h = 0; h < KC; ++h)
              part[u][grp][h][0] = part[u][grp][h][1] = part[u][grp][h][2] = part[u][grp][h][3] = 0.f;
#pragma unroll
        for (int h = 0; h < KC; ++h) {
          uint4 ka[NU], kb[NU];
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            ka[u] = *reinterpret_cast<const uint4*>(kst[u] + chunk_off<D>(pg, t + 4 * h));
            kb[u] = *reinterpret_cast<const uint4*>(kst[u] + chunk_off<D>(pg + 8, t + 4 * h));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
              const uint32_t wa = i == 0 ? ka[u].x : i == 1 ? ka[u].y : i == 2 ? ka[u].z : ka[u].w;
              const uint32_t wb = i == 0 ? kb[u].x : i == 1 ? kb[u].y : i == 2 ? kb[u].z : kb[u].w;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(wa, a0, a2);
              e4m3x4_to_f16(wb, a1, a3);
#pragma unroll
              for (int grp = 0; grp < NG; ++grp)
                mma_f16_16x8x16(part[u][grp][h], a0, a1, a2, a3, qf[grp][h * 4 + i][0], qf[grp][h * 4 + i][1]);
            }
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = part[u][grp][0][i];
              if constexpr (KC == 2) v += part[u][grp][1][i];
              s[u][grp][i] = v * ks[u][i >> 1] * cq[grp][i & 1];
            }
      }
      if constexpr (edge) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int32_t j0 = base[u] + pg;
          if (j0 < w.t0 || j0 >= w.t1) lv[u][0] = 0.f;              // whatever an unused place holds
          if (j0 + 8 < w.t0 || j0 + 8 >= w.t1) lv[u][1] = 0.f;
#pragma unroll
          for (int grp = 0; grp < NG; ++grp)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = row0 + grp * 8 + 2 * t + e;
              int32_t lo, hi;
              seen_range(a, w.kv_len, w.pos0 + r / a.group, lo, hi);
              if (j0 < lo || j0 >= hi) s[u][grp][e] = -INFINITY;
              if (j0 + 8 < lo || j0 + 8 >= hi) s[u][grp][2 + e] = -INFINITY;
            }
        }
      }
      // ---- move the references when a score passes its limit
      float top[NG][2], topv[NG][2];
      bool need = false;
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[grp][e] = topv[grp][e] = -INFINITY;
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            top[grp][e] = fmaxf(top[grp][e], fmaxf(s[u][grp][e], s[u][grp][2 + e]));
            topv[grp][e] = fmaxf(topv[grp][e], fmaxf(s[u][grp][e] + lv[u][0], s[u][grp][2 + e] + lv[u][1]));
          }
          need |= top[grp][e] > m[grp][e] + kLag || topv[grp][e] > mv[grp][e] + kLag;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          float fe[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[grp][e], max_over_g(top[grp][e]));
            const float vn = fmaxf(mv[grp][e], max_over_g(topv[grp][e]));
            l[grp][e] *= ex2(m[grp][e] - mn);
            fe[e] = ex2(mv[grp][e] - vn);
            m[grp][e] = mn;
            mv[grp][e] = vn;
          }
#pragma unroll
          for (int j = 0; j < DT; ++j) {
            acc[grp][j][0] *= fe[0];
            acc[grp][j][1] *= fe[1];
            acc[grp][j][2] *= fe[0];
            acc[grp][j][3] *= fe[1];
          }
        }
      }
      // ---- weights, and the second product's operand
      uint32_t pb[NU][NG][2];
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        const float b0 = mv[grp][0] - kLift, b1 = mv[grp][1] - kLift;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          l0 += ex2(s[u][grp][0] - m[grp][0]) + ex2(s[u][grp][2] - m[grp][0]);
          l1 += ex2(s[u][grp][1] - m[grp][1]) + ex2(s[u][grp][3] - m[grp][1]);
          pb[u][grp][0] =
              transpose8x8(pack_f16x2(ex2(s[u][grp][0] + (lv[u][0] - b0)), ex2(s[u][grp][1] + (lv[u][0] - b1))));
          pb[u][grp][1] =
              transpose8x8(pack_f16x2(ex2(s[u][grp][2] + (lv[u][1] - b0)), ex2(s[u][grp][3] + (lv[u][1] - b1))));
        }
        l[grp][0] += l0;
        l[grp][1] += l1;
      }
      // ---- values: bytes of four tokens interleaved into token pairs
      constexpr int VW = D / 32;                               // words of a token that a lane takes
      uint32_t vw[NU][4][VW];
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vst[u] + chunk_off<D>(v_tok[i], pg));
            vw[u][i][0] = x.x;
            vw[u][i][1] = x.y;
            vw[u][i][2] = x.z;
            vw[u][i][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vst[u] + chunk_off<D>(v_tok[i], g >> 1) + 8 * (g & 1));
            vw[u][i][0] = x.x;
            vw[u][i][1] = x.y;
          }
          if (edge && (base[u] + v_tok[i] < w.t0 || base[u] + v_tok[i] >= w.t1)) {
#pragma unroll
            for (int e = 0; e < VW; ++e) vw[u][i][e] = 0u;
          }
        }
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < VW; ++i)
#pragma unroll
          for (int hlf = 0; hlf < 2; ++hlf) {
            const uint32_t sel = hlf ? 0x7362u : 0x5140u;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(__byte_perm(vw[u][0][i], vw[u][1][i], sel), a0, a1);
            e4m3x4_to_f16(__byte_perm(vw[u][2][i], vw[u][3][i], sel), a2, a3);
#pragma unroll
            for (int grp = 0; grp < NG; ++grp)
              mma_f16_16x8x16(acc[grp][2 * i + hlf], a0, a1, a2, a3, pb[u][grp][0], pb[u][grp][1]);
          }
    };
    // A value that is not finite must not reach rows that do not see its token, not even with a weight of zero.  Among
    // tokens that only some rows see (this warp's from .. to) it is taken out of the stage, and the rows that see it
    // are noted: they become NaN when the parts are joined.  (Teams that share a unit may each find it.)
    auto take_out = [&](int slot, int32_t first, int32_t from, int32_t to) {
      constexpr int kLanes = D / 16;                           // of a token
#pragma unroll 1
      for (int32_t j = from + lane / kLanes; j < to; j += 32 / kLanes) {
        uint4* x = reinterpret_cast<uint4*>(smem + slot * C::kStageBytes + C::kCodes + chunk_off<D>(j - first, lane % kLanes));
        float* vs = reinterpret_cast<float*>(smem + C::kOffScale) + slot * C::kScaleFloats + kUnit + (j - first);
        const uint4 w4 = *x;
        const bool scale = *vs >= 0.f && *vs < INFINITY;
        if ((nan_codes(w4.x) | nan_codes(w4.y) | nan_codes(w4.z) | nan_codes(w4.w)) != 0u || !scale) {
          *x = make_uint4(without_nan_codes(w4.x), without_nan_codes(w4.y), without_nan_codes(w4.z), without_nan_codes(w4.w));
          if (!scale) *vs = 0.f;
          fence_proxy_async_smem();                            // (the stage's next contents come by TMA)
          for (int r = 0; r < rows; ++r) {
            int32_t lo, hi;
            seen_range(a, w.kv_len, w.pos0 + r / a.group, lo, hi);
            if (j >= lo && j < hi) atomicOr(&s_spoilt[item & 1], 1u << r);
          }
        }
      }
      __syncwarp();
    };
    for (int32_t k = c.k0; k < c.k1; ++k, ++q) {
      if (RT == 1 && static_cast<int>(q % C::kGroups) != team) continue;
      const int slot = static_cast<int>(q % C::kStages);
      if (ok) {
        const bool in = mbar_wait_bounded(bar_full(slot), (q / C::kStages) & 1u, p.wait_limit);
        ok = __all_sync(0xffffffffu, in);
        if (!ok && lane == 0) report_failure(a.err, kDevTimeoutEpilogue);
      }
      const int32_t base = (ub + k) * kUnit + wq * 32;
      if (ok && base < w.t1 && base + 32 > w.t0) {
        if (base >= full_lo && base + 32 <= full_hi) {
          process(k, std::false_type{});
        } else {
          const int32_t first = (ub + k) * kUnit, from = base > w.t0 ? base : w.t0, to = base + 32 < w.t1 ? base + 32 : w.t1;
          // (where a window leaves tokens on both sides, all of the warp's are looked at)
          const bool low = w.t0 < full_lo && from < full_lo;
          if (low || (full_hi < w.t1 && to > full_hi))
            take_out(slot, first, low || from > full_hi ? from : full_hi, to);
          process(k, std::true_type{});
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty(slot));
    }

    Cursor nx = c;
    more = next(nx);
    if (more) fetch(nx);

    // ---- the warps' parts of the item, added in warp order, four rows at a time
    const bool whole = c.k0 == 0 && c.k1 == w.units;
    const int slot_id = 2 * blockIdx.x + (c.item0 + c.k0 == u0 ? 0 : 1);
    float* part_o = p.partials + static_cast<int64_t>(slot_id) * kRows * (D + 1);
    const int vchunk = D == 128 ? 16 * pg : 8 * g;         // first output element of this lane
#pragma unroll
    for (int part4 = 0; part4 < 2 * NG; ++part4) {
      const int grp = part4 >> 1, hf = part4 & 1;          // rows 8 grp + 4 hf ..: those of lanes t = 2 hf, 2 hf + 1
      if (part4 * C::kJoin >= rows) break;
      named_bar_sync(1, C::kWarps * 32);
      if (part4 == 0 && tid == 0) s_spoilt[(item + 1) & 1] = 0;      // the item before is read, the next not begun
      const float l0 = sum_over_g(l[grp][0]), l1 = sum_over_g(l[grp][1]);
      if ((t >> 1) == hf) {
        const int at = warp * C::kJoin + 2 * (t & 1);
        if (g == 0) {
          red_m[at] = m[grp][0];
          red_m[at + 1] = m[grp][1];
          red_l[at] = l0;
          red_l[at + 1] = l1;
          red_v[at] = mv[grp][0];
          red_v[at + 1] = mv[grp][1];
        }
        float* r0 = red + at * C::kPitch + vchunk;
        float* r1 = r0 + C::kPitch;
#pragma unroll
        for (int j = 0; j < DT; j += 2) {
          *reinterpret_cast<float4*>(r0 + 2 * j) =
              make_float4(acc[grp][j][0], acc[grp][j][2], acc[grp][j + 1][0], acc[grp][j + 1][2]);
          *reinterpret_cast<float4*>(r1 + 2 * j) =
              make_float4(acc[grp][j][1], acc[grp][j][3], acc[grp][j + 1][1], acc[grp][j + 1][3]);
        }
      }
      named_bar_sync(1, C::kWarps * 32);
      // warp w (of a team with its own rows: of its own) finishes row w of the four
      const int w4 = RT == 1 ? warp : wq, w0 = RT == 1 ? 0 : team * 4;
      const int r = row0 + part4 * C::kJoin + w4;
      if (w4 < C::kJoin && r < rows) {
        float top = kNoMax, sum = 0.f;
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) top = fmaxf(top, red_m[(w0 + i) * C::kJoin + w4]);
        float f[C::kParts];
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
          f[i] = ex2(red_m[(w0 + i) * C::kJoin + w4] - top);
          sum += red_l[(w0 + i) * C::kJoin + w4] * f[i];
        }
        // zero only where nothing is seen; a NaN stays one
        float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (s_spoilt[item & 1] >> r & 1u) inv = __uint_as_float(0x7FFFFFFFu);
        const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
        float o[D / 32];
#pragma unroll
        for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll
        for (int i = 0; i < C::kParts; ++i) {
          const float ci = ex2(red_v[(w0 + i) * C::kJoin + w4] - kLift - top) * inv;
          const float* src = red + ((w0 + i) * C::kJoin + w4) * C::kPitch + lane * (D / 32);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) o[e] = fmaf(src[e], ci, o[e]);
        }
        if (whole) {
          const int i = r / a.group, head = c.h * a.group + r - i * a.group;
          __nv_bfloat16* dst = a.out + (w.row0 + i) * a.o_st + head * a.o_sh + lane * (D / 32);
          if (ok) {
            if constexpr (D == 128) st_global_v2(dst, pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0], o[1]);
            if (a.lse != nullptr && lane == 0)
              a.lse[(w.row0 + i) * a.heads + head] = lse2 * 0.6931471805599453f;
          }
        } else {
          if constexpr (D == 128)
            *reinterpret_cast<float4*>(part_o + r * D + lane * 4) = make_float4(o[0], o[1], o[2], o[3]);
          else *reinterpret_cast<float2*>(part_o + r * D + lane * 2) = make_float2(o[0], o[1]);
          if (lane == 0) part_o[kRows * D + r] = lse2;
        }
      }
    }
    if (!whole) {
      // ---- the last CTA of the item to arrive adds the parts in CTA order
      const int64_t i0 = c.item0, i1 = c.item0 + w.units;
      const int c_first = share_of(i0, total, ctas);
      const int c_last = share_of(i1 - 1, total, ctas);
      __threadfence();
      named_bar_sync(1, C::kWarps * 32);
      if (tid == 0) {
        const int n = atomicAdd(p.counters + c_first, 1);
        s_last = n == c_last - c_first;
        if (s_last) p.counters[c_first] = 0;
      }
      named_bar_sync(1, C::kWarps * 32);
      if (s_last) {
        __threadfence();
        // the first CTA's part is its last segment, unless the item begins with its share
        const int first_slot = 2 * c_first + (share_begin(c_first, total, ctas) < i0 ? 1 : 0);
        auto slot_of = [&](int cc) -> const float* {
          return p.partials + static_cast<int64_t>(cc == c_first ? first_slot : 2 * cc) * kRows * (D + 1);
        };
        for (int r = warp; r < rows; r += C::kWarps) {
          // log2 sums and weights a lane each; the parts' loads sixteen at a time
          float top = -INFINITY;
          for (int cc = c_first + lane; cc <= c_last; cc += 32) top = fmaxf(top, __ldcg(slot_of(cc) + kRows * D + r));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float ref = top == -INFINITY ? 0.f : top;
          float sum = 0.f, o[D / 32];
#pragma unroll
          for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
          for (int c0 = c_first; c0 <= c_last; c0 += 32) {
            const float wl = c0 + lane <= c_last ? ex2(__ldcg(slot_of(c0 + lane) + kRows * D + r) - ref) : 0.f;
            const int n = c_last - c0 + 1 < 32 ? c_last - c0 + 1 : 32;
            for (int j0 = 0; j0 < n; j0 += 16) {
              using Vec = typename std::conditional<D == 128, float4, float2>::type;
              Vec v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                v[j] = __ldcg(reinterpret_cast<const Vec*>(slot_of(c0 + (j0 + j < n ? j0 + j : n - 1)) + r * D) + lane);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float wgt = __shfl_sync(0xffffffffu, wl, (j0 + j) & 31);
                if (j0 + j >= n) wgt = 0.f;
                sum += wgt;
                const float* x = reinterpret_cast<const float*>(&v[j]);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) o[e] = fmaf(x[e], wgt, o[e]);
              }
            }
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          const int i = r / a.group, head = c.h * a.group + r - i * a.group;
          __nv_bfloat16* dst = a.out + (w.row0 + i) * a.o_st + head * a.o_sh + lane * (D / 32);
          if (ok) {
            if constexpr (D == 128)
              st_global_v2(dst, pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
            else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
            if (a.lse != nullptr && lane == 0)
              a.lse[(w.row0 + i) * a.heads + head] =
                  sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
    }
    c = nx;
    ++item;
  }
  if (p.behind) griddep_wait();
}

template <int D, int NG, int RT>
cudaError_t launch_decode_ng(const CUtensorMap& k, const CUtensorMap& v, const DecodeArgs& p, int ctas,
                             cudaStream_t stream) {
  using C = DecCfg<D, NG, RT>;
  cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, NG, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_kernel<D, NG, RT>, k, v, p);
}

}  // namespace

int attn_decode_groups(int64_t rows) { return rows <= 32 ? static_cast<int>((rows + 7) / 8) : 4; }

size_t attn_decode_partial_bytes(int groups, int dim, int ctas) {
  return static_cast<size_t>(2) * ctas * groups * 8 * (dim + 1) * sizeof(float);
}

cudaError_t launch_attn_decode(const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int groups, int ctas,
                               int32_t* counters, float* partials, bool behind, cudaStream_t stream) {
  DecodeArgs p;
  p.a = a;
  p.counters = counters;
  p.partials = partials;
  p.wait_limit = 1ull << 31;
  p.behind = behind;
  if (a.c.dim == 128) {
    switch (groups) {
      case 1: return launch_decode_ng<128, 1, 1>(k, v, p, ctas, stream);
      case 2: return launch_decode_ng<128, 2, 1>(k, v, p, ctas, stream);
      case 3: return launch_decode_ng<128, 1, 3>(k, v, p, ctas, stream);
      default: return launch_decode_ng<128, 2, 2>(k, v, p, ctas, stream);
    }
  }
  switch (groups) {
    case 1: return launch_decode_ng<64, 1, 1>(k, v, p, ctas, stream);
    case 2: return launch_decode_ng<64, 2, 1>(k, v, p, ctas, stream);
    case 3: return launch_decode_ng<64, 1, 3>(k, v, p, ctas, stream);
    default: return launch_decode_ng<64, 2, 2>(k, v, p, ctas, stream);
  }
}

}  // namespace bfp8
