// bfp8_kvweigh_tile.cu -- the attention weight that cached tokens receive from
// many new tokens, on the 5th-generation tensor cores.
//
// A tile of 256 tokens of a sequence and kv head, in two halves, stays while the query rows
// that see it (new tokens x the group's heads, heads innermost) pass by, up to 128 at a time:
//   S^T = K Q^T    tcgen05.mma kind::f16 on bf16: K's codes converted once a tile (exact), Q as it is, by TMA
//   a += exp2(S^T ks scale log2 e - lse log2 e)
// so that a thread holds a token, its sum stays in a register, and the rows' log
// sums are the same for all threads (read from shared memory, four at a time).
// (Tiles of 128 tokens and units of 256 rows asked the L2 cache for twice the
// queries: a chunk of 4096 tokens at a context of 16384, 64 / 8 heads of 128, took 893 us.)
// Roles: a warpgroup of exponentials for each half, four warps that
// convert keys (the next tile's beside this one's rows), one for the MMAs,
// one for the queries' TMA and one for the rows' log sums.
//
// The row tiles of all token tiles form one line that the persistent CTAs
// share equally; a token tile cut by a border leaves 256 partial sums in the
// workspace and the last CTA to arrive adds them in CTA order.
#include <cuda.h>
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

constexpr int kHalf = 128, kTile = 2 * kHalf;  // tokens of a half, and of a tile
constexpr int kRowsMax = 128;              // query rows of a unit
constexpr int kWarpMma = 8, kWarpQuery = 9, kWarpBias = 10, kWarpConv = 12, kConvWarps = 4;
constexpr int kThreads = (kWarpConv + kConvWarps) * 32;
constexpr int kItemCost = 1;               // places of a token tile in the line besides its units
constexpr int kSeqChunk = 1024;            // sequences whose places are held at once
constexpr int kBiasSlots = 4;

template <int D>
struct Cfg {
  static constexpr int kParts = D / 64;                   // of a row, 128 bytes each
  static constexpr int kA = kHalf * D * 2;                // keys of a half, bf16
  static constexpr int kQ = kRowsMax * D * 2;             // queries of a unit
  static constexpr int kASlots = D == 128 ? 3 : 4, kQStages = D == 128 ? 3 : 4;
  static constexpr int kOffA = 0;
  static constexpr int kOffQ = kASlots * kA;
  static constexpr int kOffBias = kOffQ + kQStages * kQ;
  static constexpr int kOffKs = kOffBias + kBiasSlots * kRowsMax * 4;   // key scale, as the exponent takes it
  static constexpr int kOffAt = kOffKs + kASlots * kHalf * 4;           // where the token's sum is; -1: nowhere
  static constexpr int kOffBar = kOffAt + kASlots * kHalf * 8;
  static constexpr int kBars = 2 * kQStages + 2 * kBiasSlots + 2 * kASlots + 8;
  static constexpr int kSmem = kOffBar + kBars * 8 + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kSeqChunk * 8 <= kOffBias, "sequences' places fit the operands' space");
};

struct TileArgs {
  WeighArgs w;
  int32_t* counters;          // two a CTA, zero between calls
  float* partials;            // two slots a CTA of 256 sums
  unsigned long long wait_limit;
  int32_t step;               // new tokens of a unit
};

// A sequence's tokens and new tokens.
struct Seq {
  int64_t row0;
  int32_t q_len, kv_len, pos0;
  int32_t tiles;              // 0: not this kernel's
};
__device__ __forceinline__ Seq seq_of(const TileArgs& p, int b) {
  const SeqLens s = seq_lens(p.w.a, b);
  Seq w;
  w.row0 = s.row0;
  w.q_len = s.q_len;
  w.kv_len = s.kv_len;
  w.pos0 = s.kv_len - s.q_len;
  w.tiles = static_cast<int64_t>(s.q_len) * p.w.a.group > p.w.a.few_rows ? (s.kv_len + kTile - 1) / kTile : 0;
  return w;
}
// New tokens [lo, hi) that see token j.
__device__ __forceinline__ void seen_from(const AttnArgs& a, const Seq& w, int32_t j, int32_t& lo, int32_t& hi) {
  lo = a.causal && j > w.pos0 ? j - w.pos0 : 0;
  hi = w.q_len;
  if (a.window > 0) {
    const int64_t end = static_cast<int64_t>(j) + a.window - w.pos0;
    if (end < hi) hi = end > 0 ? static_cast<int32_t>(end) : 0;
  }
}
// Units of token tile kt, the first of them at new token r0 * step.
__device__ __forceinline__ int32_t tile_units(const TileArgs& p, const Seq& w, int32_t kt, int32_t& r0) {
  int32_t lo, hi, x;
  seen_from(p.w.a, w, kt * kTile, lo, x);
  const int32_t last = kt * kTile + kTile < w.kv_len ? kt * kTile + kTile - 1 : w.kv_len - 1;
  seen_from(p.w.a, w, last, x, hi);
  r0 = lo / p.step;
  if (hi <= lo) {                                         // no row sees any: their sums may yet begin here
    r0 = 0;
    return p.w.add ? 0 : 1;
  }
  return (hi + p.step - 1) / p.step - r0;
}
__device__ __forceinline__ int32_t cost_of(int32_t units) { return units > 0 ? units + kItemCost : 0; }

struct Cursor {
  int64_t item0;              // line position of the item's first unit
  Seq w;
  int32_t b, h, kt;
  int32_t n, r0;              // units of the item
  int32_t k0, k1;             // ... in this share
};

// kind::f16, A = B = bf16, D = f32, both K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One lane of the warp, the same every time, known to the compiler as one thread.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i])::"memory");
}
// bf16 pairs of an e4m3 word (exact).
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  float f[4];
  e4m3x4_to_f32(w, f);
  lo = pack_bf16x2(f[0], f[1]);
  hi = pack_bf16x2(f[2], f[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TileArgs p) {
  using C = Cfg<D>;
  const AttnArgs& a = p.w.a;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset: the compiler has to see that this is shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.c.heads;
  auto bar = [&](int i) { return sbase + static_cast<uint32_t>(C::kOffBar + 8 * i); };
  // full and empty: queries, log sums, keys of a half, scores of a half (buffer * 2 + half)
  constexpr int bQf = 0, bQe = bQf + C::kQStages, bBf = bQe + C::kQStages, bBe = bBf + kBiasSlots, bAf = bBe + kBiasSlots,
                bAe = bAf + C::kASlots, bTf = bAe + C::kASlots, bTe = bTf + 4;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_total;
  __shared__ Cursor s_first;
  __shared__ int s_last[2];

  if (tid == 0) {
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(bar(bQf + i), 1);
      mbar_init(bar(bQe + i), 1);
    }
    for (int i = 0; i < kBiasSlots; ++i) {
      mbar_init(bar(bBf + i), 1);
      mbar_init(bar(bBe + i), 8);
    }
    for (int i = 0; i < C::kASlots; ++i) {
      mbar_init(bar(bAf + i), kConvWarps);
      mbar_init(bar(bAe + i), 1 + 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(bTf + i), 1);
      mbar_init(bar(bTe + i), 4);
    }
    fence_barrier_init();
  }
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's share [u0, u1) of the line: the places of each sequence and kv head, a warp a sequence, in the
  // operands' space; then one warp adds up
  int64_t* cnt = reinterpret_cast<int64_t*>(smem);
  auto count_chunk = [&](int b0) {
    const int n = a.batch - b0 < kSeqChunk ? a.batch - b0 : kSeqChunk;
    for (int i = warp; i < n; i += kThreads / 32) {
      const Seq w = seq_of(p, b0 + i);
      int64_t v = 0;
      int32_t r0;
      for (int32_t kt = lane; kt < w.tiles; kt += 32) v += cost_of(tile_units(p, w, kt, r0));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) cnt[i] = v;
    }
    __syncthreads();
    return n;
  };
  int64_t run = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kSeqChunk) {
    const int n = count_chunk(b0);
    if (warp == 0) {
      int64_t v = 0;
      for (int i = lane; i < n; i += 32) v += cnt[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) s_total = v;
    }
    __syncthreads();
    run += s_total;
    __syncthreads();
  }
  const int64_t total = run * H;
  const int64_t ctas = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= ctas) return;                       // whole CTA: nothing allocated or in flight yet
  const int64_t u0 = share_begin(blockIdx.x, total, ctas), u1 = share_begin(blockIdx.x + 1, total, ctas);
  run = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kSeqChunk) {
    const int n = a.batch <= kSeqChunk ? a.batch : count_chunk(b0);
    if (warp == 0) {
      for (int i0 = 0; i0 < n; i0 += 32) {
        const int64_t own = i0 + lane < n ? cnt[i0 + lane] : 0;
        int64_t v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        const int64_t before = (run + v - own) * H;
        const uint32_t here = __ballot_sync(0xffffffffu, own > 0 && before <= u0 && u0 < before + own * H);
        if (here != 0u) {
          // the head by a division, its token tile by adding up those before it, 32 at a time
          const int at = __ffs(here) - 1, b = b0 + i0 + at;
          const int64_t mine = __shfl_sync(0xffffffffu, own, at), first = __shfl_sync(0xffffffffu, before, at);
          const Seq w = seq_of(p, b);
          const int h = static_cast<int>((u0 - first) / mine);
          int64_t place = first + h * mine;
          for (int32_t kt0 = 0; kt0 < w.tiles; kt0 += 32) {
            int32_t r0 = 0;
            const int32_t units = kt0 + lane < w.tiles ? tile_units(p, w, kt0 + lane, r0) : 0;
            int64_t x = cost_of(units);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int64_t t = __shfl_up_sync(0xffffffffu, x, o);
              if (lane >= o) x += t;
            }
            const int64_t start = place + x - cost_of(units);
            if (units > 0 && start <= u0 && u0 < start + cost_of(units)) {
              s_first.item0 = start;
              s_first.w = w;
              s_first.b = b;
              s_first.h = h;
              s_first.kt = kt0 + lane;
              s_first.n = units;
              s_first.r0 = r0;
            }
            place += __shfl_sync(0xffffffffu, x, 31);
          }
        }
        run += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  fence_proxy_async_smem();                             // the counts' space is handed to the TMA
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // ---- every warp walks the share by itself
  Cursor c = s_first;
  auto clip = [&]() {                                   // false: only the item's end lies in the share
    c.k0 = static_cast<int32_t>(u0 > c.item0 ? u0 - c.item0 : 0);
    c.k1 = static_cast<int32_t>(c.item0 + c.n < u1 ? c.n : u1 - c.item0);
    return c.k0 < c.k1;
  };
  auto next = [&]() -> bool {                           // false: the share is done
    do {
      c.item0 += cost_of(c.n);
      if (c.item0 >= u1) return false;
      do {
        if (++c.kt == c.w.tiles) {
          c.kt = 0;
          if (++c.h == H) {
            c.h = 0;
            do {
              c.w = seq_of(p, ++c.b);
            } while (c.w.tiles == 0);
          }
        }
        c.n = tile_units(p, c.w, c.kt, c.r0);
      } while (c.n == 0);
    } while (!clip());
    return true;
  };
  bool more = clip() || next();
  bool ok = true;
  // one lane waits for its warp
  auto wait_warp = [&](int i, uint32_t parity, int code) {
    if (!ok) return;
    int r = 1;
    if (lane == 0) r = mbar_wait_bounded(bar(i), parity, p.wait_limit);
    ok = __shfl_sync(0xffffffffu, r, 0) != 0;
    if (!ok && lane == 0) report_failure(a.err, code);
  };
  // every lane waits (it reads what the barrier guards)
  auto wait_all = [&](int i, uint32_t parity, int code) {
    if (!ok) return;
    const bool r = mbar_wait_bounded(bar(i), parity, p.wait_limit);
    ok = __all_sync(0xffffffffu, r);
    if (!ok && lane == 0) report_failure(a.err, code);
  };
  auto ph = [](uint32_t q, int stages) { return (q / static_cast<uint32_t>(stages)) & 1u; };
  uint32_t q = 0, item = 0;                             // units and items begun

  if (warp < 8) {
    // ------------------------------------------------------------ exponentials
    const int half = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float* s_ks = reinterpret_cast<const float*>(smem + C::kOffKs);
    const int64_t* s_at = reinterpret_cast<const int64_t*>(smem + C::kOffAt);
    for (; more; more = next(), ++item) {
      const uint32_t hq = 2 * item + half;
      const int slot = static_cast<int>(hq % C::kASlots);
      wait_all(bAf + slot, ph(hq, C::kASlots), kDevTimeoutEpilogue);
      const float ks = s_ks[slot * kHalf + r];
      const int64_t at = s_at[slot * kHalf + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bAe + slot));
      const int32_t j = c.kt * kTile + half * kHalf + r;
      const bool whole = c.k0 == 0 && c.k1 == c.n;
      const bool writes = at >= 0 && ok;
      float old = 0.f;
      if (writes && whole && !begins_here(p.w, j, c.w.pos0)) old = p.w.w[at];
      int32_t lo, hi;
      seen_from(a, c.w, j, lo, hi);
      const uint64_t ks2 = pack_u32x2(__float_as_uint(ks), __float_as_uint(ks));
      uint64_t sum2[2] = {0, 0};
      for (int32_t k = c.k0; k < c.k1; ++k, ++q) {
        const int bs = static_cast<int>(q % kBiasSlots), ts = static_cast<int>(q & 1);
        const int64_t first = static_cast<int64_t>(c.r0 + k) * p.step;         // new token of the unit's first row
        // this thread's rows among the unit's columns
        auto column = [&](int32_t i) {
          const int64_t n = i - first;
          return static_cast<int32_t>(n < 0 ? 0 : n > p.step ? p.step : n) * a.group;
        };
        const int32_t from = column(lo), to = column(hi);
        wait_all(bBf + bs, ph(q, kBiasSlots), kDevTimeoutEpilogue);
        wait_all(bTf + 2 * ts + half, ph(q, 2), kDevTimeoutEpilogue);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tS = tmem + lanes + ts * 2 * kRowsMax + half * kRowsMax;
        const float* bias = reinterpret_cast<const float*>(smem + C::kOffBias) + bs * kRowsMax;
        // (full units of groups that divide 128; chunks of 4096 at 16384: 64 / 8 heads 1160 TFLOP/s, 40 / 8 and 24 / 8, whose units
        // have 125 and 126 rows, 660 by the loop below)
        if (__all_sync(0xffffffffu, from == 0 && to == kRowsMax)) {
          // 32 columns at a time, the next ones on their way from tensor memory meanwhile
          uint32_t o[2][32];
          tmem_ld32(tS, o[0]);
#pragma unroll
          for (int x = 0; x < kRowsMax / 32; ++x) {
            uint32_t(&now)[32] = o[x & 1];
            tmem_wait_ld();
            reg_fence32(now);
            if (x + 1 < kRowsMax / 32) tmem_ld32(tS + 32 * (x + 1), o[(x + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(bias + 32 * x + e);
              float y[4];
              unpack_f32x2(fma_f32x2(pack_u32x2(now[e], now[e + 1]), ks2, b2.x), y[0], y[1]);
              unpack_f32x2(fma_f32x2(pack_u32x2(now[e + 2], now[e + 3]), ks2, b2.y), y[2], y[3]);
              sum2[0] = add_f32x2(sum2[0], pack_u32x2(__float_as_uint(ex2(y[0])), __float_as_uint(ex2(y[1]))));
              sum2[1] = add_f32x2(sum2[1], pack_u32x2(__float_as_uint(ex2(y[2])), __float_as_uint(ex2(y[3]))));
            }
          }
        } else {
#pragma unroll 1
          for (int c0 = 0; c0 < kRowsMax; c0 += 32) {
            if (!__any_sync(0xffffffffu, from < c0 + 32 && to > c0 && from < to)) continue;
            uint32_t o[32];
            tmem_ld32(tS + c0, o);
            tmem_wait_ld();
            reg_fence32(o);
            const int32_t f = from - c0, t = to - c0;
            float part[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = ex2(fmaf(__uint_as_float(o[e]), ks, bias[c0 + e]));
              if (e >= f && e < t) part[e & 1] += x;
            }
            sum2[0] = add_f32x2(sum2[0], pack_u32x2(__float_as_uint(part[0]), __float_as_uint(part[1])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bTe + 2 * ts + half));
          mbar_arrive(bar(bBe + bs));
        }
      }
      float s0, s1;
      unpack_f32x2(add_f32x2(sum2[0], sum2[1]), s0, s1);
      const float sum = s0 + s1;
      if (whole) {
        if (writes && ok) p.w.w[at] = old + sum;
      } else {
        // ---- the last CTA of the item to arrive adds the parts in CTA order
        const int c_first = share_of(c.item0, total, ctas), c_last = share_of(c.item0 + c.n - 1, total, ctas);
        const int slot_id = 2 * blockIdx.x + (c.item0 + c.k0 == u0 ? 0 : 1);
        p.partials[static_cast<int64_t>(slot_id) * kTile + half * kHalf + r] = sum;
        __threadfence();
        named_bar_sync(1 + half, kHalf);
        if (r == 0) {
          const int n = atomicAdd(p.counters + 2 * c_first + half, 1);
          s_last[half] = n == c_last - c_first;
          if (s_last[half]) p.counters[2 * c_first + half] = 0;
        }
        named_bar_sync(1 + half, kHalf);
        if (s_last[half] && writes && ok) {
          __threadfence();
          // the first CTA's part is its last segment, unless the item begins with its share
          const int first_slot = 2 * c_first + (share_begin(c_first, total, ctas) < c.item0 ? 1 : 0);
          float v = 0.f;
          for (int cc = c_first; cc <= c_last; ++cc)
            v += __ldcg(p.partials + static_cast<int64_t>(cc == c_first ? first_slot : 2 * cc) * kTile + half * kHalf + r);
          p.w.w[at] = begins_here(p.w, j, c.w.pos0) ? v : p.w.w[at] + v;
        }
      }
    }
  } else if (warp == kWarpMma) {
    // -------------------------------------------------------------------- MMA
    const uint64_t desc = sdesc_k_sw128(sbase);
    const uint32_t lo = static_cast<uint32_t>(desc), hi = static_cast<uint32_t>(desc >> 32);
    uint32_t done = 0, items_done = 0;
    auto wait1 = [&](int i, uint32_t parity) {
      if (ok && !mbar_wait_bounded(bar(i), parity, p.wait_limit)) {
        report_failure(a.err, kDevTimeoutMma);
        ok = false;
      }
    };
    for (; more; more = next(), ++item) {
      const uint32_t hq = 2 * item;
      const int slot[2] = {static_cast<int>(hq % C::kASlots), static_cast<int>((hq + 1) % C::kASlots)};
      if (elect_one()) {
        wait1(bAf + slot[0], ph(hq, C::kASlots));
        wait1(bAf + slot[1], ph(hq + 1, C::kASlots));
        for (int32_t k = c.k0; k < c.k1; ++k, ++q) {
          const int qs = static_cast<int>(q % C::kQStages), ts = static_cast<int>(q & 1);
          wait1(bQf + qs, ph(q, C::kQStages));
          const int64_t left = c.w.q_len - static_cast<int64_t>(c.r0 + k) * p.step;
          const int rows = static_cast<int>(left < p.step ? left : p.step) * a.group;
          const uint32_t id = idesc_bf16(kHalf, (rows + 15) / 16 * 16);
          const uint32_t qd = lo + ((C::kOffQ + qs * C::kQ) >> 4);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait1(bTe + 2 * ts + half, ph(q, 2) ^ 1u);
            if (!ok) break;
            tc_fence_after();
            const uint32_t ad = lo + ((C::kOffA + slot[half] * C::kA) >> 4);
#pragma unroll
            for (int h = 0; h < C::kParts; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_bf16_ss(tmem + ts * 2 * kRowsMax + half * kRowsMax, ad + h * (kHalf * 128 >> 4) + 2 * i,
                            qd + h * (kRowsMax * 128 >> 4) + 2 * i, hi, id, (h | i) != 0);
            mma_commit(bar(bTf + 2 * ts + half));
          }
          if (!ok) break;
          mma_commit(bar(bQe + qs));
          done = q + 1;
        }
        if (ok) {
          mma_commit(bar(bAe + slot[0]));
          mma_commit(bar(bAe + slot[1]));
          items_done = item + 1;
        }
      }
      __syncwarp();
    }
    // every commit has arrived before the CTA exits (the last one comes after all others)
    if (elect_one()) {
      for (uint32_t i = done > C::kQStages ? done - C::kQStages : 0; i < done; ++i)
        mbar_wait_bounded(bar(bQe + static_cast<int>(i % C::kQStages)), ph(i, C::kQStages), p.wait_limit);
      if (ok)
        for (uint32_t i = items_done > 0 ? 2 * items_done - 2 : 0; i < 2 * items_done; ++i)
          mbar_wait_bounded(bar(bAe + static_cast<int>(i % C::kASlots)), ph(i, C::kASlots), p.wait_limit);
    }
    __syncwarp();
  } else if (warp == kWarpQuery) {
    // ---------------------------------------------------------------- queries
    const uint32_t bytes = static_cast<uint32_t>(C::kParts * 128 * p.step * a.group);
    for (; more && ok; more = next()) {
      for (int32_t k = c.k0; k < c.k1; ++k) {
        const int qs = static_cast<int>(q % C::kQStages);
        wait_warp(bQe + qs, ph(q, C::kQStages) ^ 1u, kDevTimeoutProducer);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(bQf + qs), bytes);
          const uint32_t dst = sbase + static_cast<uint32_t>(C::kOffQ + qs * C::kQ);
          const int32_t row = static_cast<int32_t>(c.w.row0 + static_cast<int64_t>(c.r0 + k) * p.step);
#pragma unroll
          for (int h = 0; h < C::kParts; ++h)
            tma_load_3d(dst + h * kRowsMax * 128, &tmQ, bar(bQf + qs), 128 * h, c.h * a.group, row);
        }
        __syncwarp();
        ++q;
      }
    }
    // no copy may still be landing when the CTA exits
    for (uint32_t i = q > C::kQStages ? q - C::kQStages : 0; i < q; ++i)
      if (lane == 0 && !mbar_wait_bounded(bar(bQf + static_cast<int>(i % C::kQStages)), ph(i, C::kQStages), p.wait_limit)) {
        report_failure(a.err, kDevTimeoutTail);
        break;
      }
    __syncwarp();
  } else if (warp == kWarpBias) {
    // --------------------------------------------------------------- log sums
    // rows lane, lane + 32 .. of a unit: their new token (of the unit) and head stay the same
    int32_t tok[kRowsMax / 32], head[kRowsMax / 32];
#pragma unroll
    for (int e = 0; e < kRowsMax / 32; ++e) {
      tok[e] = (lane + 32 * e) / a.group;
      head[e] = lane + 32 * e - tok[e] * a.group;
    }
    for (; more && ok; more = next()) {
      for (int32_t k = c.k0; k < c.k1; ++k) {
        const int bs = static_cast<int>(q % kBiasSlots);
        const int64_t first = static_cast<int64_t>(c.r0 + k) * p.step;
        float v[kRowsMax / 32];
#pragma unroll
        for (int e = 0; e < kRowsMax / 32; ++e) {
          const int64_t i = first + tok[e];
          v[e] = tok[e] < p.step && i < c.w.q_len ? __ldg(a.lse + (c.w.row0 + i) * a.heads + c.h * a.group + head[e]) : INFINITY;
        }
        wait_warp(bBe + bs, ph(q, kBiasSlots) ^ 1u, kDevTimeoutProducer);
        if (!ok) break;
        float* dst = reinterpret_cast<float*>(smem + C::kOffBias) + bs * kRowsMax + lane;
#pragma unroll
        for (int e = 0; e < kRowsMax / 32; ++e) dst[32 * e] = v[e] * -1.4426950408889634f;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bBf + bs));
        ++q;
      }
    }
  } else if (warp >= kWarpConv) {
    // ------------------------------------------------------------------- keys
    constexpr int CH = D / 16, RPI = 32 / CH, IT = 32 / RPI;       // chunks of a token, tokens at once, steps
    const int cw = warp - kWarpConv, ch = lane % CH, sub = lane / CH;
    float* s_ks = reinterpret_cast<float*>(smem + C::kOffKs);
    int64_t* s_at = reinterpret_cast<int64_t*>(smem + C::kOffAt);
    // this warp's 32 tokens of a half: a lane looks up its token's page, then eight (or four) lanes read a token
    struct Data {
      uint4 k[IT];
      float ks;
      int64_t at;
    };
    auto fetch = [&](Data& d, int half) {
      const int32_t j = c.kt * kTile + half * kHalf + cw * 32 + lane;
      int64_t code = -1;
      d.at = -1;
      d.ks = 0.f;
      if (j < c.w.kv_len) {
        const int32_t page = __ldg(a.table + c.b * a.ld_table + (j >> a.c.page_shift));
        const int off = j & (a.c.page_size - 1);
        if (page < 0 || page >= a.c.num_pages) {
          report_failure(a.err, kDevBadCacheIndex);
        } else {
          code = page * a.c.st_page + c.h * a.c.st_head + off * a.c.st_tok;
          d.at = page * p.w.ws_page + c.h * p.w.ws_head + off;
          d.ks = __ldg(a.c.ks + page * a.c.ss_page + c.h * a.c.ss_head + off) * a.scale * 1.4426950408889634f;
        }
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, code, i * RPI + sub);
        d.k[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.c.k + at + 16 * ch)) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    Data cur, nxt;
    uint32_t hq = 0;                                              // halves begun
    if (more) fetch(cur, 0);
    while (more && ok) {
      const int slot = static_cast<int>(hq % C::kASlots);
      if (hq & 1) more = next();
      if (more) fetch(nxt, (hq & 1) ^ 1);
      wait_warp(bAe + slot, ph(hq, C::kASlots) ^ 1u, kDevTimeoutProducer);
      if (!ok) break;
      uint8_t* dst = smem + C::kOffA + slot * C::kA + (ch / 4) * (kHalf * 128);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int row = cw * 32 + i * RPI + sub;
        uint32_t o[8];
        const uint32_t w[4] = {cur.k[i].x, cur.k[i].y, cur.k[i].z, cur.k[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(w[e], o[2 * e], o[2 * e + 1]);
        const int c0 = 2 * (ch & 3);
        *reinterpret_cast<uint4*>(dst + row * 128 + ((c0 ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(dst + row * 128 + (((c0 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      s_ks[slot * kHalf + cw * 32 + lane] = cur.ks;
      s_at[slot * kHalf + cw * 32 + lane] = cur.at;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bAf + slot));
      cur = nxt;
      ++hq;
    }
  }
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_tile(const CUtensorMap& q, const TileArgs& p, int ctas, cudaStream_t stream) {
  using C = Cfg<D>;
  cudaError_t e = cudaFuncSetAttribute(weigh_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weigh_tile_kernel<D>, q, p);
}

}  // namespace

int weigh_tile_tokens(int group, int max_q) {
  const int most = kRowsMax / group;
  return max_q < most ? max_q : most;
}

size_t weigh_tile_partial_bytes(int ctas) { return static_cast<size_t>(2) * ctas * kTile * sizeof(float); }

cudaError_t launch_weigh_tile(const CUtensorMap& q, const WeighArgs& w, int ctas, int32_t* counters, float* partials,
                              cudaStream_t stream) {
  TileArgs p;
  p.w = w;
  p.counters = counters;
  p.partials = partials;
  p.wait_limit = 1ull << 31;
  p.step = weigh_tile_tokens(w.a.group, w.a.max_q);
  return w.a.c.dim == 128 ? launch_tile<128>(q, p, ctas, stream) : launch_tile<64>(q, p, ctas, stream);
}

}  // namespace bfp8
