// bfp8_attn_tile.cu -- attention of many new tokens a sequence over the paged
// e4m3 cache, on the 5th-generation tensor cores: bound by the two products.
//
// The query rows of a kv head (new tokens x the group's heads, heads innermost)
// are cut into blocks of 256: two 128-row tiles a CTA, which take turns on the
// tensor core and the softmax.  A block's context comes in 128-token tiles.
//   S = Q K^T   tcgen05.mma kind::f8f6f4 straight from the cache's codes.  A bf16
//               query element (8 significant bits) is the sum of two e4m3 numbers
//               (4 bits each) after scaling its row by a power of two, so Q is kept
//               as two e4m3 operands and S takes two passes: exact products of what the
//               operands hold (elements to 2^-17 of their row's largest) at the
//               time of one 16-bit pass, and no conversion of K.
//   O += P V    kind::f16: P from tensor memory, over the columns of S; V converted
//               from e4m3 by two warps, scaled by its token's scale relative
//               to the tile's largest (one f16 rounding).
// Roles: two softmax warpgroups (a thread a row: scores from tensor memory, key
// scales, mask, running maximum and sum, P, and the rare rescaling of O), two warps
// converting V, one for the MMAs, and one for TMA and the tiles' scales.
//
// Scores x are in powers of two.  A tile's values share the scale 2^lv, which
// joins the exponent: P = 2^(x + lv - mv + 7) with mv a running maximum of x + lv,
// and the sum of the weights collects P 2^-lv, 64 columns' sum at a time.  mv may
// lag for as long as 64 weights sum to 2^15 at most, which every f16 holds; only
// where they pass that is the chunk's maximum looked for, O and the sum
// rescaled and the chunk done again.  So a tile takes no pass for its maximum:
// of the softmax's time a row (800 cycles beside another warp) that was 140.  Where a tile's value scales
// differ by more than 2^11 its tokens' own log2 scales join the exponents instead.
//
// A pair of 128 x 128 tiles (two query tiles over 128 tokens) takes 3400 cycles
// against 2090 of the MMAs alone: a query tile's scores wait for its weights, which
// stand in their place, so that its softmax (1630 cycles, and 480 until the last
// of its four warps has finished) and its MMAs (1050) take turns, and the other
// tile's turns fill what gaps they can.  4096 tokens of 64 / 8 heads of 128 at a
// context of 16384: 1.42 to 1.48 ms, 1300 to 1350 TFLOP/s (4 D flop a score; the queries'
// second part not counted), 0.68 to 0.71 of the measured bf16 rate.  A block costs 15000 cycles
// besides (queries, first scores, output).
//
// As in the kernel for few rows, the tiles of all blocks form one line (with
// kBlockCost places behind each block's for the time that a block costs besides)
// that the persistent CTAs share equally; a block cut by a border leaves fp32 partial
// rows in the workspace and the last CTA to arrive adds them in CTA order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_attn.cuh"
#include "bfp8_attn_math.cuh"
#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"

namespace bfp8 {

namespace {

constexpr int kTile = 128;                 // tokens of a tile, rows of a query tile
constexpr int kBlockRows = 2 * kTile;
// 8 softmax warps, one for the MMAs, one for TMA and the tiles' scales, two that
// convert V.  Three warpgroups and no more: the compiler plans for the registers
// that a thread has at launch (168); with 128, and four warps converting, a chunk
// took 11% longer.
// 208 and 88 a thread after they are handed around.
constexpr int kTileThreads = 384;
constexpr int kWarpMma = 8, kWarpLoad = 9, kWarpConv = 10, kConvWarps = 2;
constexpr int kBlockCost = 8;              // (places of a block besides its tiles' pairs (3400 cycles): 15000 cycles, more where parts are joined;
                                           // 5 to 10 time alike, 12 is 3% slower on a mixed batch)
constexpr int kSeqChunk = 2048;            // sequences whose tile counts are held at once
constexpr int kKStages = 3, kVStages = 2, kFStages = 2, kScSlots = 4;
constexpr int kBadSlots = 8;               // > blocks in flight: the loader is at most kScSlots tiles ahead
constexpr float kNoMax = -3.0e38f;
constexpr float kLift = 7.f;               // a weight at the running maximum is 2^7
constexpr float kMost = 32768.f;           // sum of 64 weights up to which the maximum may lag: each fits f16
constexpr int kVUp = 6;                    // values are scaled up by 2^6 in f16: 448 * 2^6 < 65504
constexpr float kWide = 0x1p-11f;          // below this ratio of value scales a tile takes the other path

template <int D>
struct TileCfg {
  static constexpr int kQ = kTile * D;                    // one e4m3 part of a query tile
  static constexpr int kK = kTile * D;
  static constexpr int kV16 = kTile * D * 2;
  static constexpr int kHalf = kTile * 128;               // 64 columns of V in f16
  static constexpr int kOffQ = 0;                         // [tile][hi, lo]
  static constexpr int kOffK = kOffQ + 4 * kQ;
  static constexpr int kOffV = kOffK + kKStages * kK;
  static constexpr int kOffF = kOffV + kVStages * kK;
  static constexpr int kOffRaw = kOffF + kFStages * kV16;     // scales as in the cache: K then V
  static constexpr int kOffKs = kOffRaw + kScSlots * 2 * kTile * 4;
  static constexpr int kOffRv = kOffKs + kScSlots * kTile * 4;
  static constexpr int kOffDl = kOffRv + kScSlots * kTile * 8;   // wide tiles: log2 vs - lv
  static constexpr int kOffIv = kOffDl + kScSlots * kTile * 4;   // wide tiles: 1 / vs
  static constexpr int kOffInfo = kOffIv + kScSlots * kTile * 4; // lv, 2^-lv, wide
  static constexpr int kOffBad = kOffInfo + kScSlots * 16;       // a flag a block
  static constexpr int kOffCur = kOffBad + kBadSlots * 4;        // a cursor a warp
  static constexpr int kOffBar = kOffCur + (kTileThreads / 32) * 80;
  static constexpr int kBars = 2 * kKStages + 2 * kVStages + 2 * kFStages + 3 * kScSlots + 8;
  static constexpr int kSmem = kOffBar + kBars * 8 + 64 + 1024;
  static constexpr uint32_t kColO = 256;                  // S (and P) of the tiles at 0 and 128
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kSeqChunk * 8 <= kOffRaw, "tile counts fit the operands' space");
};

struct TileArgs {
  AttnArgs a;
  int32_t* counters;          // two a CTA, zero between calls
  float* partials;            // two slots a CTA
  unsigned long long wait_limit;
  int32_t min_tiles;          // least tiles of a share
};

// Floats of a slot: [2 tiles][D / 4][128 rows][4], then the rows' log2 sums.
template <int D>
__host__ __device__ constexpr int64_t slot_floats() { return kBlockRows * D + kBlockRows; }

// Row blocks and context of a sequence.
struct SeqBlocks {
  int64_t row0;
  int32_t q_len, kv_len, pos0;
  int32_t blocks;             // 0: not this kernel's
};
__device__ __forceinline__ SeqBlocks seq_blocks(const AttnArgs& a, int b) {
  const SeqLens s = seq_lens(a, b);
  SeqBlocks w;
  w.row0 = s.row0;
  w.q_len = s.q_len;
  w.kv_len = s.kv_len;
  w.pos0 = s.kv_len - s.q_len;
  const int64_t rows = static_cast<int64_t>(s.q_len) * a.group;
  w.blocks = rows > a.few_rows ? static_cast<int32_t>((rows + kBlockRows - 1) / kBlockRows) : 0;
  return w;
}
// Tokens [t0, t1) that some row of block rb sees, [f0, f1) that every row sees, and its tiles.
__device__ __forceinline__ int32_t block_tiles(const AttnArgs& a, const SeqBlocks& w, int rb, int32_t& t0,
                                               int32_t& t1, int32_t& f0, int32_t& f1) {
  const uint32_t r0 = static_cast<uint32_t>(rb) * kBlockRows, group = static_cast<uint32_t>(a.group);   // < 2^32: 2^24 tokens, 128 heads
  const int32_t i0 = static_cast<int32_t>(r0 / group);
  int32_t i1 = static_cast<int32_t>((r0 + kBlockRows - 1) / group);
  if (i1 > w.q_len - 1) i1 = w.q_len - 1;
  int32_t lo, hi;
  seen_range(a, w.kv_len, w.pos0 + i0, lo, f1);
  seen_range(a, w.kv_len, w.pos0 + i1, f0, hi);
  t0 = lo;
  t1 = hi;
  return hi > lo ? (hi + kTile - 1) / kTile - lo / kTile : 1;
}

// Query tiles of row block rb that hold rows: a sequence's last block may need only the first (16 sequences of 5
// tokens at 8192, 40 rows each: 132 us against 152 with the empty tile computed beside it, by events around single
// calls; 118 now, back to back).
__device__ __forceinline__ int block_query_tiles(const AttnArgs& a, const SeqBlocks& w, int rb) {
  return static_cast<int64_t>(w.q_len) * a.group - static_cast<int64_t>(rb) * kBlockRows > kTile ? 2 : 1;
}

struct Cursor {
  int64_t item0;
  SeqBlocks w;
  int32_t b, h, rb;
  int32_t n, k0, k1;
  int32_t t0, t1;             // tokens that some row sees
  int32_t f0, f1;             // ... that every row sees
  uint32_t blk;               // blocks of the share before it
};
static_assert(sizeof(Cursor) <= 80, "space of a warp's cursor");

// What is not finite among a block's scales and values must not reach rows that do not see its token, not even as
// 0 x NaN.  It is taken out where the tiles are made ready; a flag says so, and only then the block's rows look, at their
// end, at the tokens that they see.  (Looked for tile by tile in the softmax it cost 8% of a chunk, and any more
// instructions in the converters' or the loader's loops much the same.)
// What spoils the row that sees tokens [lo, hi) of the block's sequence among those of this CTA's tiles: 1 a key scale,
// 2 a value.
template <int D>
__device__ __noinline__ uint32_t bad_of_row(const AttnArgs& a, const Cursor& c, int32_t lo, int32_t hi) {
  uint32_t kinds = 0;
  const int32_t base = c.t0 / kTile * kTile;
  lo = max(lo, base + c.k0 * kTile);
  hi = min(hi, base + c.k1 * kTile);
  for (int32_t j = lo; j < hi; ++j) {
    const int32_t page = a.table[c.b * a.ld_table + (j >> a.c.page_shift)];
    if (page < 0 || page >= a.c.num_pages) continue;
    const int off = j & (a.c.page_size - 1);
    const int64_t so = page * a.c.ss_page + c.h * a.c.ss_head + off;
    const float ks = a.c.ks[so];
    if (ks != ks) kinds |= 1u;
    if (!(a.c.vs[so] < INFINITY)) kinds |= 2u;
    if (j >= c.f0 && j < c.f1) continue;                       // a NaN code there is in the product
    const uint4* v = reinterpret_cast<const uint4*>(a.c.v + page * a.c.st_page + c.h * a.c.st_head + off * a.c.st_tok);
    for (int e = 0; e < D / 16; ++e)
      if ((nan_codes(v[e].x) | nan_codes(v[e].y) | nan_codes(v[e].z) | nan_codes(v[e].w)) != 0u) kinds |= 2u;
  }
  return kinds;
}

// Readies converter cw's rows of a tile of values (a warp): rows outside [z0, z1) hold no token and become zero (they
// may hold anything); rows outside [p0, p1) are not seen by every query row and lose their NaN codes.  Were there any?
template <int D>
__device__ __forceinline__ bool prepare_rows_here(uint8_t* tile, int cw, const Cursor& c, int32_t k) {
  const int32_t tok0 = (c.t0 / kTile + k) * kTile, z0 = c.t0 - tok0, z1 = c.t1 - tok0, p0 = min(c.f0 - tok0, kTile), p1 = c.f1 - tok0;
  constexpr int kLanes = D / 16, kRows = 32 / kLanes, kGroup = kRows * kConvWarps;
  const int lane = threadIdx.x & 31, ch = lane % kLanes, r0 = cw * kRows + lane / kLanes;
  // (rows kGroup apart have the same swizzle)
  uint8_t* at = tile + (D == 128 ? (ch ^ (r0 & 7)) << 4 : (ch ^ ((r0 >> 1) & 3)) << 4);
  uint32_t any = 0;
  auto row = [&](int r) {
    uint4* x = reinterpret_cast<uint4*>(at + r * D);
    if (r < z0 || r >= z1) {
      *x = make_uint4(0u, 0u, 0u, 0u);
    } else {
      const uint4 w = *x;
      const uint32_t f = nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w);
      if (f != 0u)
        *x = make_uint4(without_nan_codes(w.x), without_nan_codes(w.y), without_nan_codes(w.z), without_nan_codes(w.w));
      any |= f;
    }
  };
#pragma unroll 1
  for (int r = r0; r < p0; r += kGroup) row(r);
#pragma unroll 1
  for (int r = r0 + (p1 > r0 ? (p1 - r0 + kGroup - 1) / kGroup * kGroup : 0); r < kTile; r += kGroup) row(r);
  __syncwarp();
  return any != 0u;
}

// Out of the way of the loop's instructions with heads of 128 (a chunk of 4096 at 16384 1438 us, 1466 inlined), inlined with
// heads of 64 (8 chunks of 512: 100 us, 103 called).
template <int D>
__device__ __noinline__ bool prepare_rows_called(uint8_t* tile, int cw, const Cursor& c, int32_t k) {
  return prepare_rows_here<D>(tile, cw, c, k);
}
template <int D>
__device__ __forceinline__ bool prepare_rows(uint8_t* tile, int cw, const Cursor& c, int32_t k) {
  if constexpr (D == 128) return prepare_rows_called<D>(tile, cw, c, k);
  else return prepare_rows_here<D>(tile, cw, c, k);
}

// MMAs whose descriptors come as low words (start address >> 4 and leading
// offset) and a constant high word: the issuing thread keeps few registers.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16, A = B = f16, D = f32, A K-major, B MN-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_f16_bmn(int m, int n) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// K-major rows of 64 bytes with the 64-byte swizzle: 8-row groups 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_k_sw64(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(16u >> 4) << 16;
  d |= static_cast<uint64_t>(512u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(4u) << 61;
  return d;
}
// MN-major f16 with the 128-byte swizzle: rows (contraction index) of 64
// elements, 8-row groups 1024 bytes apart (stride offset), the next 64
// elements `next` bytes on (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t next) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(next >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
// One lane of the warp, the same every time.  Where a branch hangs on it the compiler knows that one thread runs
// and keeps an MMA's operands in uniform registers; on lane == 0 it cannot, and an MMA took so many instructions
// that the softmax warps' held it up: 16 MMAs beside warps that never stop issuing 4177 cycles, with this 1246.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Orders later uses of the registers after the preceding wait.
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ TileArgs p) {
  using C = TileCfg<D>;
  const AttnArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset: the compiler has to see that this is shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.c.heads;
  // barriers
  auto bar = [&](int i) { return sbase + static_cast<uint32_t>(C::kOffBar + 8 * i); };
  const int bKf = 0, bKe = bKf + kKStages, bVf = bKe + kKStages, bVe = bVf + kVStages, bFf = bVe + kVStages,
            bFe = bFf + kFStages, bRf = bFe + kFStages, bSf = bRf + kScSlots, bSe = bSf + kScSlots,
            bQ = bSe + kScSlots, bS = bQ + 2, bP = bS + 2, bO = bP + 2;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_total;
  __shared__ int64_t s_u0, s_u1;                 // this CTA's share of the line of s_total tiles
  __shared__ int s_ctas;
  __shared__ Cursor s_first;                     // the block in which the share begins
  __shared__ int s_last[2];

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(bar(bKf + i), 1);
      mbar_init(bar(bKe + i), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(bar(bVf + i), 1);
      mbar_init(bar(bVe + i), kConvWarps);
    }
    for (int i = 0; i < kFStages; ++i) {
      mbar_init(bar(bFf + i), kConvWarps);
      mbar_init(bar(bFe + i), 1);
    }
    for (int i = 0; i < kScSlots; ++i) {
      mbar_init(bar(bRf + i), 1);
      mbar_init(bar(bSf + i), 1);
      mbar_init(bar(bSe + i), 8 + kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bQ + i), 4);
      mbar_init(bar(bS + i), 1);
      mbar_init(bar(bP + i), 4);
      mbar_init(bar(bO + i), 1);
    }
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();                  // after the wait: what starts behind this needs no wait of its own

  // the page table is looked at once the share is known: into the cache with it (no more than a line a thread)
  {
    const int64_t at = static_cast<int64_t>(tid) * 32;
    if (at < static_cast<int64_t>(a.batch - 1) * a.ld_table + 1)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + at));
  }
  // ---- this CTA's share of the line of tiles: the tiles of each sequence and
  // kv head, a warp a sequence, in the operands' space; then one warp adds up
  int64_t* cnt = reinterpret_cast<int64_t*>(smem);
  auto count_chunk = [&](int b0) {
    const int n = a.batch - b0 < kSeqChunk ? a.batch - b0 : kSeqChunk;
    for (int i = warp; i < n; i += kTileThreads / 32) {
      const SeqBlocks w = seq_blocks(a, b0 + i);
      int64_t v = 0;
      int32_t t0, t1, f0, f1;
      for (int rb = lane; rb < w.blocks; rb += 32) v += block_tiles(a, w, rb, t0, t1, f0, f1) + kBlockCost;
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
  {
    const int64_t total = run * H;
    int64_t ctas = total / p.min_tiles;
    if (ctas < 1) ctas = 1;
    if (ctas > gridDim.x) ctas = gridDim.x;
    if (total == 0 || blockIdx.x >= ctas) return;       // whole CTA: nothing allocated or in flight yet
    if (tid == 0) {
      s_total = total;
      s_ctas = static_cast<int>(ctas);
      s_u0 = share_begin(blockIdx.x, total, ctas);
      s_u1 = share_begin(blockIdx.x + 1, total, ctas);
    }
    __syncthreads();
  }
  run = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kSeqChunk) {
    const int n = a.batch <= kSeqChunk ? a.batch : count_chunk(b0);
    if (warp == 0) {
      const int64_t u0 = s_u0;
      int64_t mine = 0, first = 0;               // the sequence with u0: a head's places, its first place
      int hit = -1;
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
          const int at = __ffs(here) - 1;
          hit = b0 + i0 + at;
          mine = __shfl_sync(0xffffffffu, own, at);
          first = __shfl_sync(0xffffffffu, before, at);
        }
        run += __shfl_sync(0xffffffffu, v, 31);
      }
      if (hit >= 0) {
        // its head by a division, the head's block by adding up the blocks before it, 32 at a time (walking
        // there block by block cost a chunk of 4096 tokens 160 us)
        const SeqBlocks w = seq_blocks(a, hit);
        const int h = static_cast<int>((u0 - first) / mine);
        int64_t place = first + h * mine;
        for (int rb0 = 0; rb0 < w.blocks; rb0 += 32) {
          int32_t t0 = 0, t1 = 0, f0 = 0, f1 = 0;
          const int64_t own = rb0 + lane < w.blocks ? block_tiles(a, w, rb0 + lane, t0, t1, f0, f1) + kBlockCost : 0;
          int64_t v = own;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
          }
          if (own > 0 && place + v - own <= u0 && u0 < place + v) {
            s_first.item0 = place + v - own;
            s_first.w = w;
            s_first.b = hit;
            s_first.h = h;
            s_first.rb = rb0 + lane;
            s_first.n = static_cast<int32_t>(own) - kBlockCost;
            s_first.t0 = t0;
            s_first.t1 = t1;
            s_first.f0 = f0;
            s_first.f1 = f1;
            s_first.blk = 0;
          }
          place += __shfl_sync(0xffffffffu, v, 31);
        }
      }
    }
    __syncthreads();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  fence_proxy_async_smem();                     // the counts' space is handed to the TMA
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Cursor over the share: block (b, h, rb), its tiles [k0, k1) here, its place
  // in the line.  Each warp has one in shared memory, kept by its first lane:
  // the loops over tiles need their registers for other things.
  auto step_block = [&](Cursor& c) {            // the block after (b, h, rb)
    ++c.blk;
    if (++c.rb == c.w.blocks) {
      c.rb = 0;
      if (++c.h == H) {
        c.h = 0;
        do {
          c.w = seq_blocks(a, ++c.b);
        } while (c.w.blocks == 0);
      }
    }
    c.n = block_tiles(a, c.w, c.rb, c.t0, c.t1, c.f0, c.f1);
  };
  auto clip = [&](Cursor& c) {                  // false: only the block's end lies in the share
    c.k0 = static_cast<int32_t>(s_u0 > c.item0 ? s_u0 - c.item0 : 0);
    c.k1 = static_cast<int32_t>(c.item0 + c.n < s_u1 ? c.n : s_u1 - c.item0);
    return c.k0 < c.k1;
  };
  Cursor& c = reinterpret_cast<Cursor*>(smem + C::kOffCur)[warp];
  uint32_t* const bad_blocks = reinterpret_cast<uint32_t*>(smem + C::kOffBad);
  auto advance = [&](Cursor& c) {               // false: the share is done
    do {
      c.item0 += c.n + kBlockCost;
      if (c.item0 >= s_u1) return false;
      step_block(c);
    } while (!clip(c));
    return true;
  };
  auto start = [&]() -> bool {
    int more = 0;
    if (lane == 0) {
      c = s_first;
      more = clip(c) || advance(c);
    }
    more = __shfl_sync(0xffffffffu, more, 0);
    __syncwarp();
    return more != 0;
  };
  auto next = [&]() -> bool {
    __syncwarp();
    int more = 0;
    if (lane == 0) more = advance(c);
    more = __shfl_sync(0xffffffffu, more, 0);
    __syncwarp();
    return more != 0;
  };

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

  if (warp >= kWarpMma) {
    setmaxnreg_dec<88>();
    if (warp == kWarpLoad) {
      // --------------------------------------------- TMA and the tiles' scales
      // scales of tile q as the softmax and the converters take them, from the raw ones; run one
      // tile after their load, before anything that waits for the tile's consumers
      auto scales = [&](uint32_t q, int32_t tok0, int32_t t0, int32_t t1, uint32_t blk) {
        const int sl = static_cast<int>(q % kScSlots);
        wait_all(bRf + sl, ph(q, kScSlots), kDevTimeoutEpilogue);
        const int32_t tok = tok0 + lane * 4;
        const float4 kr = *reinterpret_cast<const float4*>(smem + C::kOffRaw + (sl * 2 * kTile + lane * 4) * 4);
        const float4 vr = *reinterpret_cast<const float4*>(smem + C::kOffRaw + ((sl * 2 + 1) * kTile + lane * 4) * 4);
        float ks[4] = {kr.x, kr.y, kr.z, kr.w}, vs[4] = {vr.x, vr.y, vr.z, vr.w};
        bool bad = false;
        float top = 0.f, low = 3.0e38f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool live = tok + e >= t0 && tok + e < t1, finite = vs[e] < INFINITY;
          bad |= live && (ks[e] != ks[e] || !finite);
          // masked scores are -inf before the key scale: it must not be zero or NaN
          ks[e] = live ? fmaxf(ks[e], 1.2e-38f) : 1.f;
          if (!live || !finite) vs[e] = 0.f;
          top = fmaxf(top, vs[e]);
          if (live) low = fminf(low, vs[e]);
        }
        if (bad) bad_blocks[blk % kBadSlots] = 1u;
        // (not negative: ordered as their bits are; with shuffles a mixed batch took 3% longer)
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        low = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(low)));
        // vref = 2^E >= top; values are held as code * (vs / vref) * 2^kVUp, so 2^lv = vref 2^-kVUp
        uint32_t bits = (__float_as_uint(top) + 0x7FFFFFu) & 0xFF800000u;
        if (bits < 0x10000000u) bits = 0x10000000u;                    // 2^-95: an all-zero tile
        const float vinv = __uint_as_float(0x7F000000u - bits);
        const bool wide = low < top * kWide;
        const float lv = static_cast<float>(static_cast<int>(bits >> 23) - 127 - kVUp);
        float4 dl, iv;
        float rr[4], dd[4], ii[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rr[e] = !(vs[e] > 0.f) ? 0.f : wide ? static_cast<float>(1 << kVUp) : vs[e] * vinv * static_cast<float>(1 << kVUp);
          // a scale of zero is a value of zero: its weight counts all the same
          dd[e] = vs[e] > 0.f ? lg2(vs[e] * vinv) : 0.f;
          ii[e] = (vs[e] > 0.f ? 1.f / vs[e] : vinv) * static_cast<float>(1 << kVUp);
        }
        dl = make_float4(dd[0], dd[1], dd[2], dd[3]);
        iv = make_float4(ii[0], ii[1], ii[2], ii[3]);
        *reinterpret_cast<float4*>(smem + C::kOffKs + (sl * kTile + lane * 4) * 4) =
            wide ? make_float4(1.f, 1.f, 1.f, 1.f) : make_float4(ks[0], ks[1], ks[2], ks[3]);
        // the value factor as two f16 numbers, each twice: rh + rl holds 22 bits of it
        uint32_t rh[4], rl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half h = __float2half_rn(rr[e]);
          const __half d = __float2half_rn(rr[e] - __half2float(h));
          rh[e] = __half_as_ushort(h) * 0x10001u;
          rl[e] = __half_as_ushort(d) * 0x10001u;
        }
        uint4* rv = reinterpret_cast<uint4*>(smem + C::kOffRv + (sl * kTile + lane * 4) * 8);
        rv[0] = make_uint4(rh[0], rl[0], rh[1], rl[1]);
        rv[1] = make_uint4(rh[2], rl[2], rh[3], rl[3]);
        if (wide) {
          *reinterpret_cast<float4*>(smem + C::kOffDl + (sl * kTile + lane * 4) * 4) = dl;
          *reinterpret_cast<float4*>(smem + C::kOffIv + (sl * kTile + lane * 4) * 4) = iv;
        }
        if (lane == 0)
          *reinterpret_cast<float4*>(smem + C::kOffInfo + sl * 16) =
              make_float4(lv, vinv * static_cast<float>(1 << kVUp), wide ? 1.f : 0.f, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bSf + sl));
      };
      const int page = a.c.page_size, shift = a.c.page_shift;
      const int ppu = page >= kTile ? 1 : kTile / page;
      const int box = page >= kTile ? kTile : page;
      uint32_t q = 0, pending = 0;                      // loads begun; a tile whose scales wait
      int32_t p_tok = 0, p_t0 = 0, p_t1 = 0;
      uint32_t p_blk = 0;
      for (bool more = start(); more; more = next() && ok) {
        const int32_t ub = c.t0 / kTile, t0 = c.t0, t1 = c.t1, h = c.h, k1 = c.k1;
        const int32_t* row = a.table + c.b * a.ld_table;
        int32_t cached = -1, entry = 0;
        const uint32_t blk = c.blk;
        if (lane == 0) bad_blocks[blk % kBadSlots] = 0u;        // (its last user is kBadSlots blocks back)
        for (int32_t k = c.k0; k < k1 && ok; ++k) {
          const int32_t tok = (ub + k) * kTile;
          const int32_t first = tok / box;
          if (first / 32 != cached) {
            cached = first / 32;
            const int64_t t = (static_cast<int64_t>(cached) * 32 + lane) * box;
            entry = 0;
            if (t < t1 && t + box > t0) {
              entry = __ldg(row + (t >> shift));
              if (entry < 0 || entry >= a.c.num_pages) {
                report_failure(a.err, kDevBadCacheIndex);
                entry = 0;
              }
            }
          }
          const int32_t t = tok + lane * box;
          const bool live = lane < ppu && t < t1 && t + box > t0;
          const int n = __popc(__ballot_sync(0xffffffffu, live));
          const int32_t pg = __shfl_sync(0xffffffffu, entry, (first + lane) & 31);
          const int off = t & (page - 1);
          const int sc = static_cast<int>(q % kScSlots), ks = static_cast<int>(q % kKStages),
                    vs = static_cast<int>(q % kVStages);
          wait_warp(bSe + sc, ph(q, kScSlots) ^ 1u, kDevTimeoutProducer);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(bRf + sc), static_cast<uint32_t>(n * 2 * box * 4));
          }
          __syncwarp();
          if (live) {
            const int64_t so = pg * a.c.ss_page + h * a.c.ss_head + off;
            const uint32_t sd = sbase + static_cast<uint32_t>(C::kOffRaw + (sc * 2 * kTile + lane * box) * 4);
            bulk_load(sd, a.c.ks + so, box * 4, bar(bRf + sc));
            bulk_load(sd + kTile * 4, a.c.vs + so, box * 4, bar(bRf + sc));
          }
          ++q;                                          // its copies are in flight
          if (pending) scales(q - 2, p_tok, p_t0, p_t1, p_blk);
          pending = q > 1;
          p_tok = tok;
          p_t0 = t0;
          p_t1 = t1;
          p_blk = blk;
          wait_warp(bKe + ks, ph(q - 1, kKStages) ^ 1u, kDevTimeoutProducer);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(bKf + ks), static_cast<uint32_t>(n * box * D));
          __syncwarp();
          if (live)
            tma_load_4d(sbase + static_cast<uint32_t>(C::kOffK + ks * C::kK + lane * box * D), &tmK, bar(bKf + ks), 0,
                        off, h, pg);
          wait_warp(bVe + vs, ph(q - 1, kVStages) ^ 1u, kDevTimeoutProducer);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(bVf + vs), static_cast<uint32_t>(n * box * D));
          __syncwarp();
          if (live)
            tma_load_4d(sbase + static_cast<uint32_t>(C::kOffV + vs * C::kK + lane * box * D), &tmV, bar(bVf + vs), 0,
                        off, h, pg);
          if (q == 1) scales(0, tok, t0, t1, blk);      // the first tile's are waited for
        }
      }
      if (pending) scales(q - 1, p_tok, p_t0, p_t1, p_blk);
      // no copy may still be landing when the CTA exits (after a failure: bounded waits all the same)
      auto drain = [&](int b0, int stages) {
        for (uint32_t i = q > static_cast<uint32_t>(stages) ? q - stages : 0; i < q; ++i)
          if (lane == 0 && !mbar_wait_bounded(bar(b0 + static_cast<int>(i % stages)), ph(i, stages), p.wait_limit)) {
            report_failure(a.err, kDevTimeoutTail);
            break;
          }
        __syncwarp();
      };
      drain(bRf, kScSlots);
      drain(bKf, kKStages);
      drain(bVf, kVStages);
    } else if (warp == kWarpMma) {
      // ------------------------------------------------------------- MMA
      // the whole warp walks; one lane waits and issues
      const uint32_t idS = idesc_e4m3_f32(128, 128), idO = idesc_f16_bmn(128, D);
      auto wait1 = [&](int i, uint32_t parity) {
        if (ok && !mbar_wait_bounded(bar(i), parity, p.wait_limit)) {
          report_failure(a.err, kDevTimeoutMma);
          ok = false;
        }
        return ok;
      };
      const uint64_t kdesc = D == 128 ? sdesc_k_sw128(sbase) : sdesc_k_sw64(sbase), vdesc = sdesc_mn_sw128(sbase, C::kHalf);
      const uint32_t klo = static_cast<uint32_t>(kdesc), khi = static_cast<uint32_t>(kdesc >> 32),
                     vlo = static_cast<uint32_t>(vdesc), vhi = static_cast<uint32_t>(vdesc >> 32);
      auto qk = [&](int t, int ks) {
        const uint32_t kd = klo + (C::kOffK >> 4) + ks * (C::kK >> 4), qd = klo + (C::kOffQ >> 4) + 2 * t * (C::kQ >> 4);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            mma_f8_ss(tmem + t * 128, qd + part * (C::kQ >> 4) + 2 * i, kd + 2 * i, khi, idS, (part | i) != 0);
      };
      auto pv = [&](int t, int fs, bool first) {
        const uint32_t vd = vlo + (C::kOffF >> 4) + fs * (C::kV16 >> 4);
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          mma_f16_ts(tmem + C::kColO + t * 128, tmem + t * 128 + 8 * i, vd + 128 * i, vhi, idO, !(first && i == 0));
      };
      uint32_t q = 0, done = 0;                  // stages are counted in 32 bits: at most 2^30 tokens an item
      uint32_t item = 0;
      uint32_t q1 = 0, item1 = 0;                // as q and item, of the blocks with two query tiles
      for (bool more_blocks = start(); more_blocks; more_blocks = next()) {
        const int32_t n = c.k1 - c.k0;
        if (elect_one()) {
          wait1(bQ, item & 1);
          const int nt = block_query_tiles(a, c.w, c.rb);
          if (nt == 2) wait1(bQ + 1, item1++ & 1);
          wait1(bKf + static_cast<int>(q % kKStages), ph(q, kKStages));
          if (ok) {
            tc_fence_after();
            qk(0, static_cast<int>(q % kKStages));
            mma_commit(bar(bS));
            if (nt == 2) {
              qk(1, static_cast<int>(q % kKStages));
              mma_commit(bar(bS + 1));
            }
            mma_commit(bar(bKe + static_cast<int>(q % kKStages)));
          }
          for (int32_t k = 0; k < n && ok; ++k, ++q) {
            const bool more = k + 1 < n;
            const int fs = static_cast<int>(q % kFStages), kn = static_cast<int>((q + 1) % kKStages);
            wait1(bFf + fs, ph(q, kFStages));
            if (more) wait1(bKf + kn, ph(q + 1, kKStages));
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
              if (!wait1(bP + t, (t == 0 ? q : q1) & 1)) break;
              tc_fence_after();
              pv(t, fs, k == 0);
              if (t == nt - 1) mma_commit(bar(bFe + fs));
              if (more) {
                qk(t, kn);
                mma_commit(bar(bS + t));
                if (t == nt - 1) mma_commit(bar(bKe + kn));
              } else {
                mma_commit(bar(bO + t));
              }
            }
            if (nt == 2) ++q1;
            if (ok) done = q + 1;
          }
          ++item;
        }
      }
      // every commit has arrived before the CTA exits
      if (elect_one()) {
        for (uint32_t i = done > kFStages ? done - kFStages : 0; i < done; ++i)
          mbar_wait_bounded(bar(bFe + static_cast<int>(i % kFStages)), ph(i, kFStages), p.wait_limit);
        for (uint32_t i = done > kKStages ? done - kKStages : 0; i < done; ++i)
          mbar_wait_bounded(bar(bKe + static_cast<int>(i % kKStages)), ph(i, kKStages), p.wait_limit);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- converters
      const int cw = warp - kWarpConv, c8 = lane & 7, rsub = lane >> 3;
      constexpr int CH = D / 16;                        // 16-code chunks of a row
      uint32_t q = 0;
      for (bool more = start(); more; more = next()) {
        // tiles with places without a token, or tokens that only some rows see: before part0, from part1 on
        const int32_t ub = c.t0 / kTile, part0 = (c.f0 + kTile - 1) / kTile - ub, part1 = c.f1 / kTile - ub;
        for (int32_t k = c.k0; k < c.k1; ++k, ++q) {
          const int sl = static_cast<int>(q % kScSlots), vs = static_cast<int>(q % kVStages),
                    fs = static_cast<int>(q % kFStages);
          wait_all(bSf + sl, ph(q, kScSlots), kDevTimeoutEpilogue);
          wait_all(bVf + vs, ph(q, kVStages), kDevTimeoutEpilogue);
          wait_all(bFe + fs, ph(q, kFStages) ^ 1u, kDevTimeoutEpilogue);
          if (__builtin_expect((k < part0 || k >= part1) && ok, 0) && prepare_rows<D>(smem + C::kOffV + vs * C::kK, cw, c, k))
            bad_blocks[c.blk % kBadSlots] = 1u;
          const uint8_t* src = smem + C::kOffV + vs * C::kK;
          uint8_t* dst = smem + C::kOffF + fs * C::kV16;
          const uint2* rv = reinterpret_cast<const uint2*>(smem + C::kOffRv) + sl * kTile;
          constexpr int RPI = 32 / CH;                  // rows a warp takes at once
          const int ch = D == 128 ? c8 : lane & 3, sub = D == 128 ? rsub : lane >> 2;
#pragma unroll 1
          for (int i0 = 0; i0 < kTile / kConvWarps / RPI; i0 += 4) {
            // four rows' loads, then their arithmetic, then their stores: the compiler cannot tell that
            // the stores leave the loads alone
            uint4 w[4];
            uint2 r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int row = ((i0 + u) * kConvWarps + cw) * RPI + sub;     // the warps' rows in turn: both have some to ready
              w[u] = *reinterpret_cast<const uint4*>(
                  src + (D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4)));
              r[u] = rv[row];
            }
            uint32_t o[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) e4m3x4_to_f16(ww[e], o[u][2 * e], o[u][2 * e + 1]);
            }
            // code * rh + (code * rl): one f16 rounding of the product, and 2^-22 of it
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int e = 0; e < 8; ++e) o[u][e] = hfma2(o[u][e], r[u].x, hmul2(o[u][e], r[u].y));
            // two 16-byte chunks of the row's 64-column half; lanes of the second half store them in
            // the other order, so that a quarter-warp's stores fall on different banks
            const int half = ch >> 2, c0 = 2 * (ch & 3), f0 = half & 1;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int row = ((i0 + u) * kConvWarps + cw) * RPI + sub;
              uint8_t* drow = dst + half * C::kHalf + row * 128;
              const uint4 lo = make_uint4(o[u][0], o[u][1], o[u][2], o[u][3]),
                          hi = make_uint4(o[u][4], o[u][5], o[u][6], o[u][7]);
              *reinterpret_cast<uint4*>(drow + (((c0 + f0) ^ (row & 7)) << 4)) = f0 ? hi : lo;
              *reinterpret_cast<uint4*>(drow + (((c0 + 1 - f0) ^ (row & 7)) << 4)) = f0 ? lo : hi;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(bFf + fs));
            mbar_arrive(bar(bVe + vs));
            mbar_arrive(bar(bSe + sl));
          }
        }
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    setmaxnreg_inc<208>();
    const int t = warp >> 2;                          // query tile of this warpgroup
    const int r = (warp & 3) * 32 + lane;             // row of the tile
    const uint32_t tS = tmem + t * 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tO = tS - t * 128 + C::kColO + t * 128;
    uint32_t q = 0;
    uint32_t qs = 0, item = 0;                        // tiles and blocks of this query tile
    bool more = start();
    while (more) {
      if (t >= block_query_tiles(a, c.w, c.rb)) {
        // no rows here: only the tiles' scales are given back, each once it is there (an earlier arrival could
        // fall into the slot's phase before)
        for (int32_t k = c.k0; k < c.k1; ++k, ++q) {
          const int sl = static_cast<int>(q % kScSlots);
          wait_all(bSf + sl, ph(q, kScSlots), kDevTimeoutEpilogue);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bSe + sl));
        }
        more = next();
        continue;
      }
      // ---- this row's query, as two e4m3 rows
      const int64_t R = static_cast<int64_t>(c.rb) * kBlockRows + t * kTile + r;
      const int32_t i = static_cast<int32_t>(R / a.group);
      const int head = c.h * a.group + static_cast<int>(R - static_cast<int64_t>(i) * a.group);
      const bool live = i < c.w.q_len;
      // (rows past the last token see everything: their scores are computed beside the others' and
      // dropped, and must not make tiles look masked)
      int32_t lo = 0, hi = 0x7FFFFFFF;
      if (live) seen_range(a, c.w.kv_len, c.w.pos0 + i, lo, hi);
      float cq;
      {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (c.w.row0 + (live ? i : 0)) * a.q_st + head * a.q_sh);
        uint4 raw[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          raw[j] = live ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
          // largest magnitude of the bf16 pairs: the halves compare as integers
          const uint32_t ww[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, ww[e] & 0x7FFF7FFFu);
        }
        top = (top >> 16) > (top & 0xFFFFu) ? top >> 16 : top & 0xFFFFu;
        int ex = static_cast<int>(top >> 7) - 127;
        if (ex < -126) ex = -126;
        const int sh = 7 - ex, s1 = sh / 2, s2 = sh - s1;           // |q| 2^sh < 2^8
        float f1 = __uint_as_float(static_cast<uint32_t>(127 + s1) << 23);
        const float f2 = __uint_as_float(static_cast<uint32_t>(127 + s2) << 23);
        const float d1 = __uint_as_float(static_cast<uint32_t>(127 - s1) << 23);
        const float d2 = __uint_as_float(static_cast<uint32_t>(127 - s2) << 23);
        cq = fmaxf(fabsf(a.scale) * 1.4426950408889634f * d1 * d2, 1.2e-38f);
        if (a.scale < 0.f) f1 = -f1;
        if (a.scale == 0.f) f1 = 0.f;
        // e4m3 holds no infinity: the factor carries it, as a NaN, unless the row sees nothing
        if (ex > 127 && lo < hi) cq = __uint_as_float(0x7FFFFFFFu);
        uint8_t* qh = smem + C::kOffQ + 2 * t * C::kQ;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint4& u = raw[2 * j + (e >> 1)];
            const uint32_t w0 = e & 1 ? u.z : u.x, w1 = e & 1 ? u.w : u.y;
            const float f[4] = {__uint_as_float(w0 << 16) * f1 * f2, __uint_as_float(w0 & 0xFFFF0000u) * f1 * f2,
                                __uint_as_float(w1 << 16) * f1 * f2, __uint_as_float(w1 & 0xFFFF0000u) * f1 * f2};
            hi[e] = cvt_e4m3x2(f[0], f[1]) | (static_cast<uint32_t>(cvt_e4m3x2(f[2], f[3])) << 16);
            float back[4];
            e4m3x4_to_f32(hi[e], back);
            lo[e] = cvt_e4m3x2(f[0] - back[0], f[1] - back[1]) |
                    (static_cast<uint32_t>(cvt_e4m3x2(f[2] - back[2], f[3] - back[3])) << 16);
          }
          const uint32_t off = D == 128 ? static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4))
                                        : static_cast<uint32_t>(r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
          *reinterpret_cast<uint4*>(qh + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(qh + C::kQ + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bQ + t));

      float m = kNoMax, l = 0.f;
      const int32_t ub = c.t0 / kTile, k0 = c.k0, k1 = c.k1;
      for (int32_t k = k0; k < k1; ++k, ++q, ++qs) {
        const int sl = static_cast<int>(q % kScSlots);
        wait_all(bSf + sl, ph(q, kScSlots), kDevTimeoutEpilogue);
        const float4 info = *reinterpret_cast<const float4*>(smem + C::kOffInfo + sl * 16);
        const float lv = info.x;
        const bool wide = info.z != 0.f;
        const ulonglong2* ks2 = reinterpret_cast<const ulonglong2*>(smem + C::kOffKs) + sl * (kTile / 4);
        const int32_t from = lo - (ub + k) * kTile, to = hi - (ub + k) * kTile;
        const bool odd = wide || __any_sync(0xffffffffu, from > 0 || to < kTile);
        const float cc = wide ? 1.f : cq;
        // moves the running maximum to `top`, `chunks` of this tile's weights being stored already
        auto move_max = [&](float top, int chunks) {
          const float mn = fmaxf(m, top);
          const float f = ex2(m - mn);
          m = mn;
          l *= f;
          if (chunks > 0) {
            tmem_wait_st();
#pragma unroll 1
            for (int g = 0; g < chunks; ++g) {
              uint32_t o[16];
              tmem_ld16(tS + 16 * g, o);
              tmem_wait_ld();
              reg_fence16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
                o[e] = pack_f16x2(v.x * f, v.y * f);
              }
              tmem_st16(tS + 16 * g, o);
            }
          }
          if (k > k0) {
#pragma unroll 1
            for (int g = 0; g < D / 16; ++g) {
              uint32_t o[16];
              tmem_ld16(tO + 16 * g, o);
              tmem_wait_ld();
              reg_fence16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tO + 16 * g, o);
            }
          }
        };
        wait_all(bS + t, qs & 1, kDevTimeoutEpilogue);
        tc_fence_after();
        if (odd && !wide) {
          // masked scores become -inf, in tensor memory
#pragma unroll 1
          for (int g = 0; g < kTile / 32; ++g) {
            const int32_t f = from - 32 * g, e1 = to - 32 * g;
            if (!__any_sync(0xffffffffu, f > 0 || e1 < 32)) continue;
            uint32_t o[32];
            tmem_ld32(tS + 32 * g, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = e >= f && e < e1 ? o[e] : 0xFF800000u;
            tmem_st32(tS + 32 * g, o);
          }
          tmem_wait_st();
        } else if (odd) {
          // a wide tile: its scores take their tokens' own scales too (its ks are ones)
          const float* kr = reinterpret_cast<const float*>(smem + C::kOffRaw) + sl * 2 * kTile;
          const float* dl = reinterpret_cast<const float*>(smem + C::kOffDl) + sl * kTile;
          float top = -INFINITY;
#pragma unroll 1
          for (int g = 0; g < kTile / 16; ++g) {
            uint32_t o[16];
            tmem_ld16(tS + 16 * g, o);
            tmem_wait_ld();
            reg_fence16(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = 16 * g + e;
              float v = __uint_as_float(o[e]);
              v = fmaf(v * kr[j], cq, dl[j]);
              v = j >= from && j < to ? v : -INFINITY;
              top = fmaxf(top, v);
              o[e] = __float_as_uint(v);
            }
            tmem_st16(tS + 16 * g, o);
          }
          tmem_wait_st();
          {
            // its weights are summed here, by the maximum that the pass below then need not move
            if (__any_sync(0xffffffffu, live && top + lv > m)) move_max(top + lv, 0);
            const float* iv = reinterpret_cast<const float*>(smem + C::kOffIv) + sl * kTile;
            const float off = lv - m + kLift;
            float ws = 0.f;
#pragma unroll 1
            for (int g = 0; g < kTile / 16; ++g) {
              uint32_t o[16];
              tmem_ld16(tS + 16 * g, o);
              tmem_wait_ld();
              reg_fence16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) ws = fmaf(ex2(__uint_as_float(o[e]) + off), iv[16 * g + e], ws);
            }
            l += ws;
          }
        }
        // ---- 64 columns at a time: key scales, weights by the maximum so far, their sum, and once more by the
        // chunk's own maximum if that lagged too far.  A loop, and few live registers: with a whole row in them
        // the compiler had none left to overlap anything, and the two chunks written out took 13% longer, the
        // instruction cache being what four kinds of warps wait for most
        const uint64_t cc2 = pack_u32x2(__float_as_uint(cc), __float_as_uint(cc));
#pragma unroll 1
        for (int g = 0; g < kTile / 64; ++g) {
          bool look = k == k0 && g == 0, sure = false;    // look for the maximum first; the weights fit
          uint32_t nw[32];
          float part;
          while (true) {
            if (__builtin_expect(look, 0)) {
              float top = -INFINITY;
#pragma unroll 1
              for (int g1 = 4 * g; g1 < 4 * g + 4; ++g1) {
                uint32_t o[16];
                tmem_ld16(tS + 16 * g1, o);
                tmem_wait_ld();
                reg_fence16(o);
                const float* kr = reinterpret_cast<const float*>(ks2) + 16 * g1;
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, __uint_as_float(o[e]) * kr[e]);
              }
              move_max(fmaf(top, cc, lv), 2 * g);
              sure = true;
            }
            uint32_t sr[2][32];
            tmem_ld32(tS + 64 * g, sr[0]);
            tmem_ld32(tS + 64 * g + 32, sr[1]);
            tmem_wait_ld();
            reg_fence32(sr[0]);
            reg_fence32(sr[1]);
            const float off = lv - m + kLift;
            const uint64_t off2 = pack_u32x2(__float_as_uint(off), __float_as_uint(off));
            float w[64];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const ulonglong2 kv = ks2[16 * g + e / 2];
              const int c0 = 2 * e % 32;
              const uint64_t y0 = mul_f32x2(pack_u32x2(sr[e / 16][c0], sr[e / 16][c0 + 1]), kv.x),
                             y1 = mul_f32x2(pack_u32x2(sr[e / 16][c0 + 2], sr[e / 16][c0 + 3]), kv.y);
              unpack_f32x2(fma_f32x2(y0, cc2, off2), w[2 * e], w[2 * e + 1]);
              unpack_f32x2(fma_f32x2(y1, cc2, off2), w[2 * e + 2], w[2 * e + 3]);
            }
#pragma unroll
            for (int e = 0; e < 64; ++e) w[e] = ex2(w[e]);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              nw[e] = pack_f16x2(w[2 * e], w[2 * e + 1]);
              sum[e & 1] = add_f32x2(sum[e & 1], pack_u32x2(__float_as_uint(w[2 * e]), __float_as_uint(w[2 * e + 1])));
            }
            float s0, s1;
            unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
            part = s0 + s1;
            // (rows past the last token see whatever unused places hold: they have no say, or that would show in the
            // others' roundings)
            if (__builtin_expect(sure || __all_sync(0xffffffffu, !live || part <= kMost), 1)) break;
            look = true;
          }
          if (!wide) l = fmaf(part, info.y, l);
#pragma unroll
          for (int h = 0; h < 2; ++h) tmem_st16(tS + 32 * g + 16 * h, reinterpret_cast<const uint32_t(&)[16]>(nw[16 * h]));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(bP + t));
          mbar_arrive(bar(bSe + sl));
        }
      }

      // ---- output rows
      wait_all(bO + t, item & 1, kDevTimeoutEpilogue);
      tc_fence_after();
      // zero only where nothing is seen; a NaN stays one
      float inv = l == 0.f ? 0.f : 1.f / l;
      if (__builtin_expect(bad_blocks[c.blk % kBadSlots] != 0u, 0) && live) {
        const uint32_t kinds = bad_of_row<D>(a, c, lo, hi);
        if (kinds != 0u) inv = __uint_as_float(0x7FFFFFFFu);
        if (kinds & 1u) l = inv;
      }
      const float lse2 = l == 0.f ? -INFINITY : m - kLift + log2f(l);
      const bool whole = c.k0 == 0 && c.k1 == c.n;
      const int slot_id = 2 * blockIdx.x + (c.item0 + c.k0 == s_u0 ? 0 : 1);
      float* part = p.partials + slot_id * slot_floats<D>();
      float* part_lse = part + kBlockRows * D;
      __nv_bfloat16* dst = a.out + (c.w.row0 + (live ? i : 0)) * a.o_st + head * a.o_sh;
#pragma unroll 1
      for (int g = 0; g < D / 32; ++g) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * g, o);
        tmem_wait_ld();
        reg_fence32(o);
        if (whole) {
          if (live && ok) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              st_global_v4(dst + 32 * g + e,
                           pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                           pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                           pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                           pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + ((t * (D / 4) + 8 * g + e / 4) * kTile + r) * 4) =
                make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                            __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
        }
      }
      if (whole) {
        if (live && ok && a.lse != nullptr) a.lse[(c.w.row0 + i) * a.heads + head] = lse2 * 0.6931471805599453f;
      } else {
        part_lse[t * kTile + r] = lse2;
        const int64_t i0 = c.item0, i1 = c.item0 + c.n, total = s_total, ctas = s_ctas;
        const int c_first = share_of(i0, total, ctas);
        const int c_last = share_of(i1 - 1, total, ctas);
        __threadfence();
        named_bar_sync(1 + t, kTile);
        if (r == 0) {
          const int n = atomicAdd(p.counters + 2 * c_first + t, 1);
          s_last[t] = n == c_last - c_first;
          if (s_last[t]) p.counters[2 * c_first + t] = 0;
        }
        named_bar_sync(1 + t, kTile);
        if (s_last[t]) {
          __threadfence();
          // the first CTA's part is its last segment, unless the block begins with its share
          const int first_slot = 2 * c_first + (share_begin(c_first, total, ctas) < i0 ? 1 : 0);
          auto slot_of = [&](int cta) -> const float* {
            return p.partials + (cta == c_first ? first_slot : 2 * cta) * slot_floats<D>();
          };
          float best = -INFINITY;
          for (int cta = c_first; cta <= c_last; ++cta)
            best = fmaxf(best, __ldcg(slot_of(cta) + kBlockRows * D + t * kTile + r));
          const float ref = best == -INFINITY ? 0.f : best;
          float sum = 0.f;
#pragma unroll 1
          for (int g = 0; g < D / 64; ++g) {         // 64 columns' loads in flight
            float o[64];
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] = 0.f;
            sum = 0.f;
#pragma unroll 1
            for (int cta = c_first; cta <= c_last; ++cta) {
              const float* src = slot_of(cta);
              const float w = ex2(__ldcg(src + kBlockRows * D + t * kTile + r) - ref);
              sum += w;
              float4 v[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[e] = __ldcg(reinterpret_cast<const float4*>(src + ((t * (D / 4) + 16 * g + e) * kTile + r) * 4));
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                o[4 * e] = fmaf(v[e].x, w, o[4 * e]);
                o[4 * e + 1] = fmaf(v[e].y, w, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(v[e].z, w, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(v[e].w, w, o[4 * e + 3]);
              }
            }
            const float is = sum == 0.f ? 0.f : 1.f / sum;
            if (live && ok) {
#pragma unroll
              for (int e = 0; e < 64; e += 8)
                st_global_v4(dst + 64 * g + e, pack_bf16x2(o[e] * is, o[e + 1] * is),
                             pack_bf16x2(o[e + 2] * is, o[e + 3] * is), pack_bf16x2(o[e + 4] * is, o[e + 5] * is),
                             pack_bf16x2(o[e + 6] * is, o[e + 7] * is));
            }
          }
          if (live && ok && a.lse != nullptr)
            a.lse[(c.w.row0 + i) * a.heads + head] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
        }
      }
      tc_fence_before();                       // O and S are read: the next block may overwrite them
      ++item;
      more = next();
    }
  }
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_tile(const CUtensorMap& k, const CUtensorMap& v, const TileArgs& p, int ctas, cudaStream_t stream) {
  using C = TileCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(attn_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_tile_kernel<D>, k, v, p);
}

}  // namespace

size_t attn_tile_partial_bytes(int dim, int ctas) {
  return static_cast<size_t>(2) * ctas * (dim == 128 ? slot_floats<128>() : slot_floats<64>()) * sizeof(float);
}

cudaError_t launch_attn_tile(const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int ctas, int32_t* counters,
                             float* partials, cudaStream_t stream) {
  TileArgs p;
  p.a = a;
  p.counters = counters;
  p.partials = partials;
  p.wait_limit = 1ull << 31;
  p.min_tiles = 4;
  return a.c.dim == 128 ? launch_tile<128>(k, v, p, ctas, stream) : launch_tile<64>(k, v, p, ctas, stream);
}

}  // namespace bfp8
