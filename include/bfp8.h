/*
 * bfp8.h -- libbfp8: DeepSeek-style blocked W8A8 FP8 linear layer on GB300
 * (sm_103a).  Plain C ABI: raw pointers, sizes and an opaque stream handle.
 *
 * The layer has two steps (vLLM PR 49932 digest, "implementation breakdown"
 * and "key source snippet"; lmdeploy PR 4830, "Kernel design"):
 *   1. per-token group quantisation of the activations to float8_e4m3fn in
 *      1 x 128 groups, with one fp32 scale per group (amax / 448);
 *   2. the block-scaled GEMM
 *        out[m, n] = sum over 128-wide K blocks kb of
 *                    (A[m, kb] . B[n, kb]) * As[m, kb] * Bs[n / 128, kb]
 *      with 128 x 128 weight-scale tiles and a bf16 output.
 *
 * Conventions for every entry point:
 *   - Device pointers are CUDA device (or managed) addresses on the current
 *     device; the caller owns every buffer, including the GEMM workspace.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Calls only enqueue work: they neither allocate device memory
 *     nor synchronise.
 *   - Every argument is validated on the host before anything is launched; a
 *     rejected call returns a status other than BFP8_OK, launches nothing and
 *     leaves a reason in bfp8_last_error().  Nothing is thrown across the ABI.
 *   - Inputs must be finite.  NaN or infinite inputs give unspecified outputs
 *     (never a fault).
 *   - Only GB300-class devices (compute capability 10.3) are supported.
 */
#ifndef BFP8_H_
#define BFP8_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BFP8_VERSION 1

typedef enum {
  BFP8_OK = 0,
  BFP8_ERR_INVALID_ARG = 1,     /* null pointer, bad size, bad leading dimension */
  BFP8_ERR_ALIGNMENT = 2,       /* a pointer or stride breaks a stated alignment rule */
  BFP8_ERR_UNSUPPORTED = 3,     /* no device, or a device that is not sm_103 */
  BFP8_ERR_CUDA = 4,            /* a CUDA runtime / driver call failed */
  BFP8_ERR_WORKSPACE = 5,       /* workspace missing, too small or misaligned */
  BFP8_ERR_DEVICE_TIMEOUT = 6   /* a kernel-side wait gave up (see bfp8_device_status) */
} bfp8_status;

typedef enum { BFP8_IN_BF16 = 0, BFP8_IN_F32 = 1 } bfp8_in_dtype;

/* ------------------------------------------------------------------------ */
/* Step 1: per-token group quantisation                                      */
/* ------------------------------------------------------------------------ */

/*
 * bfp8_group_quant -- per_token_group_quant_fp8(x, group_size=128,
 * column_major_scales) as called in the vLLM PR 49932 digest's test.
 *
 *   x      [M, K] row-major activations, bf16 or fp32 (in_dtype), leading
 *          dimension ld_x elements (ld_x >= K).
 *   group  must be 128 (the only activation block shape the pages use).
 *   q      [M, K] float8_e4m3fn codes, leading dimension ld_q bytes (>= K).
 *   s      G = ceil(K / 128) fp32 scales per row:
 *            col_major = 0: s[m * ld_s + g], ld_s >= G
 *            col_major = 1: s[g * ld_s + m], ld_s >= M
 *          (bfp8_scale_ld(M) gives the 16-byte-aligned column-major stride the
 *          GEMM prefers).  Entries of a padded layout that hold no scale are
 *          not written.
 * For each group: amax = max |x| over the group's real elements (the last
 * group of a row has K - 128 * (G - 1) elements), scale = max(amax, 1e-10)
 * / 448 (IEEE fp32 division), q = round-to-nearest-even, saturating
 * e4m3(x / scale) with an IEEE fp32 division per element; a zero or an
 * underflow to zero keeps its sign.
 * Any M >= 0 and K >= 0 (empty inputs launch nothing).  No alignment is
 * required; 16-byte aligned rows take the vectorised path.
 */
bfp8_status bfp8_group_quant(const void* x, int in_dtype, int64_t M, int64_t K, int64_t ld_x,
                             int group, int col_major, void* q, int64_t ld_q, float* s,
                             int64_t ld_s, void* stream);

/* ------------------------------------------------------------------------ */
/* UE8M0 scale variant                                                       */
/* ------------------------------------------------------------------------ */

/*
 * The transformers DeepGEMM integration (`_ceil_to_ue8m0`, and
 * `_select_fp8_cast_kwargs` with use_ue8m0) rounds every fp32 scale UP to the
 * nearest power of two -- the UE8M0 format keeps only the biased exponent --
 * for the SM100 kernels.  That is a different function from the fp32-scale
 * layer above: activations are quantised with the rounded scale, and weight
 * scales are rounded the same way.  The blocked GEMM below computes it as it
 * stands (bfp8_gemm with such As and Bs); the scales stay fp32 values.
 */
typedef enum { BFP8_SCALE_FP32 = 0, BFP8_SCALE_UE8M0 = 1 } bfp8_scale_fmt;

/* bfp8_group_quant with a choice of scale format.  BFP8_SCALE_FP32: as
 * bfp8_group_quant.  BFP8_SCALE_UE8M0: each group's scale max(amax, 1e-10) /
 * 448 (IEEE fp32 division) is rounded up to a power of two (2^-42 for an
 * all-zero group), and q = e4m3(x / scale) with the quotient exact; |x / scale|
 * <= 448, so no code saturates.  Other arguments, layouts and errors as for
 * bfp8_group_quant; BFP8_ERR_INVALID_ARG for another scale_fmt. */
bfp8_status bfp8_group_quant_ex(const void* x, int in_dtype, int64_t M, int64_t K, int64_t ld_x,
                                int group, int col_major, int scale_fmt, void* q, int64_t ld_q,
                                float* s, int64_t ld_s, void* stream);

/* out[i] = in[i] rounded up to the nearest power of two, for n >= 0 positive
 * finite fp32 scales (e.g. a weight-scale tensor Bs for the UE8M0 variant);
 * other inputs give unspecified values.  in == out is allowed.  Device
 * pointers, 4-byte aligned; asynchronous on `stream`. */
bfp8_status bfp8_scale_ceil_ue8m0(const float* in, float* out, int64_t n, void* stream);

/* Column-major scale stride the GEMM prefers: M rounded up to a multiple of 4
 * (16 bytes of fp32, the TMA stride rule lmdeploy PR 4830 pads for). */
int64_t bfp8_scale_ld(int64_t M);

/* ------------------------------------------------------------------------ */
/* Step 2: block-scaled GEMM                                                 */
/* ------------------------------------------------------------------------ */

typedef enum {
  BFP8_SCHEDULE_AUTO = 0,
  BFP8_SCHEDULE_SWAP_AB = 1,  /* weights fill the 128-row MMA slot (small M) */
  BFP8_SCHEDULE_WIDE = 2,     /* activations fill it; 128 x 256 output tiles */
  BFP8_SCHEDULE_GEMV = 3      /* M <= 32 only: the decode kernel on warp-level
                                 MMAs (16-row weight tiles streamed by TMA, one
                                 k-block per MMA warp, no workspace use); needs
                                 K % 128 == 0 and 16-byte aligned A and B.  AUTO
                                 takes it for M <= 24 when its 16-row tiles fit
                                 one wave of 2 x SMs, and for M <= 16 when they
                                 spread evenly enough over the SMs or the
                                 weights take up to 64 MB */
} bfp8_schedule;

/* How the output tiles and their K dimension are shared out among CTAs when
 * the tiles do not fill whole waves of SMs (decode-sized M, few weight rows,
 * or a partly filled last wave). */
typedef enum {
  BFP8_KSPLIT_AUTO = 0,      /* the cheapest of the three below by a cost model
                                of this GPU */
  BFP8_KSPLIT_STREAM_K = 1,  /* persistent CTAs; tiles left after whole waves are
                                split into (tile, k-block) units, partial sums
                                meet in the workspace */
  BFP8_KSPLIT_CLUSTER = 2,   /* thread-block clusters of 2..8 CTAs share a tile,
                                each takes a slice of its k-blocks, and the
                                partial tiles are added in distributed shared
                                memory (no workspace traffic) */
  BFP8_KSPLIT_NONE = 3       /* whole tiles only, balanced over ceil(tiles /
                                waves) CTAs: nothing is split, some SMs may idle */
} bfp8_ksplit;

/* Wide tiles on CTA pairs: a 1-D cluster of two CTAs computes 256 x 256
 * output tiles with 2-SM MMAs (tcgen05.mma.cta_group::2), each CTA loading its
 * 128 activation rows and half of the 256 weight rows of every unit, so each
 * SM takes in a third less operand data per FLOP than with 128 x 256 tiles.
 * Whole tiles only (no k split), plain GEMM calls only (not grouped, not
 * fused), tiles of 256 weight rows. */
typedef enum {
  BFP8_PAIRS_AUTO = 0,    /* when the planner prefers them: never in this
                             version (they measured slower than 128 x 256
                             tiles on every shape tried) */
  BFP8_PAIRS_NEVER = 1,
  BFP8_PAIRS_ALWAYS = 2   /* whenever the call allows them; BFP8_ERR_UNSUPPORTED
                             when it does not (swap-AB or 128-wide tiles, at
                             most 64 rows, an explicit stream-K or cluster
                             split, grouped or fused calls) */
} bfp8_pairs;

/* Optional tuning / test controls; a NULL options pointer means all zero. */
typedef struct {
  int schedule;        /* bfp8_schedule */
  int max_ctas;        /* cap on CTAs; 0 = one per SM */
  int tile_n;          /* width of the second MMA operand's tile: wide 128 or
                          256 (0 = 256); swap-AB 16, 32, 64, 128 or 256 (0 =
                          the planner's choice for M) */
  int prefetch_weights;/* 1: the GEMM may start streaming B and Bs before the
                          kernel launched just before it on the stream has
                          finished (programmatic dependent launch).  Only valid
                          when that kernel does not write B or Bs, e.g. when it
                          is the bfp8_group_quant of this layer's activations. */
  int k_split;         /* bfp8_ksplit.  CLUSTER applies only when the output
                          has fewer tiles than max_ctas and K > 128; otherwise
                          stream-K runs. */
  int cluster_size;    /* CLUSTER: CTAs per tile, 2..8, clamped to ceil(K/128);
                          0 = the size the cost model prefers among those with
                          tiles * size <= max_ctas */
  int pairs;           /* bfp8_pairs: 256 x 256 tiles on CTA pairs (2-SM MMAs) */
  int reserved[1];
} bfp8_gemm_options;

/*
 * bfp8_gemm -- out = blocked_fp8_gemm(A, B, As, Bs), the computation of
 * native_w8a8_block_matmul / apply_block_scaled_mm in the vLLM PR 49932
 * digest, without its padding of M to a multiple of 4: ragged M, N and K
 * (including a partial last K block) are handled by the library.
 *
 *   A    [M, K] float8_e4m3fn, row-major, row stride K bytes.
 *   B    [N, K] float8_e4m3fn, row-major, row stride K bytes (the "NT" form:
 *        out = A @ B^T).
 *   As   activation scales, G = ceil(K / 128) per row:
 *          as_col_major = 1: As[kb * ld_as + m], ld_as >= M; the buffer holds
 *                            G * ld_as floats (rows are copied whole, as the
 *                            [G, bfp8_scale_ld(M)] buffers of bfp8_group_quant).
 *                            With ld_as - M < 4 and rows that begin on 16 bytes
 *                            it may end with the last scale: what is copied past
 *                            that lies in the same 16-byte line, is not used, and
 *                            is there in any CUDA allocation
 *          as_col_major = 0: As[m * ld_as + kb], ld_as >= G
 *   Bs   [ceil(N / 128), G] fp32, row-major, one scale per 128 x 128 weight tile.
 *   out  [M, N] bfloat16, row-major; each element is the fp32 accumulation of
 *        the scaled block partial sums, rounded to nearest even.
 *   workspace / workspace_bytes
 *        caller-owned device scratch of at least the size bfp8_gemm_workspace_size
 *        reports for the same (M, N, K, options), 256-byte aligned.  It must be
 *        zero-filled once after allocation; every call that completes leaves it
 *        ready for the next (its counters return to zero), whatever the shapes
 *        of later calls.  Concurrent calls must not share a workspace.  After
 *        BFP8_ERR_DEVICE_TIMEOUT, zero it again.
 * Results are deterministic: the same inputs give bitwise the same output on
 * every call, whichever SM finishes first.
 * Requirements: M, N, K >= 1; As, Bs 4-byte aligned.  Fast path: A and B
 * 16-byte aligned with K % 16 == 0, As column-major with ld_as % 4 == 0 and
 * 16-byte aligned, Bs 16-byte aligned with ceil(N/128) * G % 4 == 0 (what
 * bfp8_group_quant and bfp8_scale_ld produce for column-major scales).  Other
 * inputs are first re-laid out into the workspace by the library, in the
 * same call, at the cost of one or two small extra kernels.
 */
bfp8_status bfp8_gemm(const void* A, const void* B, const float* As, int as_col_major,
                      int64_t ld_as, const float* Bs, void* out, int64_t M, int64_t N, int64_t K,
                      void* workspace, size_t workspace_bytes, void* stream);

/* bfp8_gemm with explicit schedule controls (opt may be NULL).  Every
 * schedule computes the same function; they differ only in speed. */
bfp8_status bfp8_gemm_ex(const void* A, const void* B, const float* As, int as_col_major,
                         int64_t ld_as, const float* Bs, void* out, int64_t M, int64_t N,
                         int64_t K, void* workspace, size_t workspace_bytes,
                         const bfp8_gemm_options* opt, void* stream);

/* Workspace bytes bfp8_gemm / bfp8_gemm_ex need for this problem on the
 * current device: a 16 KB counter header, the stream-K partial sums, room for
 * re-laid-out scales and, when K % 16 != 0 or `operands_unaligned` is nonzero
 * (A or B not 16-byte aligned), room for re-laid-out operands.  Writes
 * *bytes; returns BFP8_ERR_UNSUPPORTED without a suitable device. */
bfp8_status bfp8_gemm_workspace_size(int64_t M, int64_t N, int64_t K,
                                     const bfp8_gemm_options* opt, int operands_unaligned,
                                     size_t* bytes);

/* Description of the schedule bfp8_gemm_ex runs.  num_sms = 0: for the
 * current device (its SM count and how many GEMM clusters of each size it
 * runs at once; needs the device).  num_sms > 0: host-only, for a device with
 * that many SMs whose cluster capacity is estimated (a little below
 * num_sms / size, since GPCs differ in size), so the cluster size may differ
 * from the one the current device would get. */
typedef struct {
  int swap_ab;          /* 1: weights in the MMA M slot */
  int tile_n;           /* MMA N (rows of the second operand per tile) */
  int stages;           /* shared-memory pipeline depth */
  int grid;             /* persistent CTAs */
  int64_t tiles;        /* output tiles */
  int64_t k_blocks;     /* G = ceil(K / 128) */
  int64_t dp_tiles;     /* tiles computed whole, round-robin */
  int64_t sk_units;     /* (tile, k-block) units split across CTAs */
  int relayout;         /* operands re-laid out into the workspace first */
  size_t workspace_bytes;
  int cluster;          /* CTAs per tile: > 1 for cluster split-K (grid =
                           tiles * cluster, dp_tiles = sk_units = 0), else 1.
                           Whole tiles only: dp_tiles = tiles, sk_units = 0,
                           grid possibly below the SM count. */
  int gemv;             /* 1: the warp-MMA decode kernel runs (BFP8_SCHEDULE_GEMV);
                           the tile fields above then describe the tensor-core
                           plan it replaces */
  int pair;             /* 1: 256 x 256 tiles on CTA pairs (grid counts CTAs,
                           tiles the 256 x 256 tiles) */
} bfp8_plan_info;

bfp8_status bfp8_gemm_plan(int64_t M, int64_t N, int64_t K, int num_sms,
                           const bfp8_gemm_options* opt, int operands_unaligned,
                           bfp8_plan_info* info);

/* The work split of a plan (num_sms as for bfp8_gemm_plan): for CTA `cta`,
 * the number of (tile, k-block) units it processes and, for unit j, its tile
 * and k-block.  Returns BFP8_ERR_INVALID_ARG for indices out of range. */
bfp8_status bfp8_plan_unit(int64_t M, int64_t N, int64_t K, int num_sms,
                           const bfp8_gemm_options* opt, int cta, int64_t j,
                           int64_t* num_units, int64_t* tile, int64_t* k_block);

/*
 * bfp8_gemm_grouped -- the same blocked FP8 GEMM for a mixture-of-experts
 * layer whose token rows are grouped by expert ("M-grouped contiguous"
 * layout: the transformers DeepGEMM integration, `_build_deepgemm_contiguous_
 * layout` and `deepgemm_fp8_fp4_experts_forward`, in its SM100 "psum" form).
 *
 *   A    [M, K] e4m3, row-major: rows sorted by expert, each expert's block
 *        padded to a multiple of 128 rows (padding rows hold anything; their
 *        outputs are computed and may be ignored).
 *   As   activation scales as for bfp8_gemm.
 *   B    [num_experts, N, K] e4m3, row-major (expert e's weights are rows
 *        e*N .. e*N+N-1 of a [num_experts*N, K] matrix).
 *   Bs   [num_experts, ceil(N/128), G] fp32, row-major.
 *   grouped_layout  device int32 [num_experts]: cumulative sums of the
 *        aligned per-expert row counts (grouped_layout[e] = end of expert e's
 *        block); non-decreasing multiples of 128.  Device memory, read by the
 *        kernel after the preceding kernel in the stream completes, so it may
 *        be produced on the device just before the call.
 *   out  [M, N] bf16: row m of expert e gets
 *          out[m, n] = sum_kb (A[m,kb] . B[e,n,kb]) * As[m,kb] * Bs[e, n/128, kb];
 *        rows m >= grouped_layout[num_experts-1] are not written (rows the
 *        caller's upper bound on M reserved but no expert uses).
 * Runs the wide schedule (128-row tiles, each inside one expert); options as
 * for bfp8_gemm_ex except `schedule` (ignored) and `prefetch_weights`
 * (ignored: the expert of a tile is known only after the wait).  Workspace
 * from bfp8_gemm_grouped_workspace_size.  Requirements as for bfp8_gemm plus
 * 1 <= num_experts <= 1024 and grouped_layout 4-byte aligned.  Its contents
 * live on the device and are checked there: when they are not non-decreasing
 * multiples of 128, the kernel writes nothing and records
 * BFP8_DEV_BAD_GROUPED_LAYOUT in the failure word (bfp8_device_status).
 */
bfp8_status bfp8_gemm_grouped(const void* A, const void* B, const float* As, int as_col_major,
                              int64_t ld_as, const float* Bs, const int32_t* grouped_layout,
                              int num_experts, void* out, int64_t M, int64_t N, int64_t K,
                              void* workspace, size_t workspace_bytes,
                              const bfp8_gemm_options* opt, void* stream);

/* Workspace bytes bfp8_gemm_grouped needs (current device). */
bfp8_status bfp8_gemm_grouped_workspace_size(int64_t M, int64_t N, int64_t K, int num_experts,
                                             const bfp8_gemm_options* opt,
                                             int operands_unaligned, size_t* bytes);

/*
 * bfp8_gemm_fused -- bfp8_gemm with the next steps of a linear layer folded
 * into the GEMM's epilogue (the transformers DeepGEMM integration's
 * `deepgemm_fp8_fp4_linear`: bias added to the bf16 product; and the next
 * layer's per_token_group_quant_fp8 of that bf16 result, vLLM PR 49932
 * digest, "key source snippet").  For every row m and column n:
 *   y[m, n] = bf16(bf16(sum_kb ...) + bias[n])     (bias == NULL: bf16(sum ...))
 * i.e. the bf16 GEMM result plus the bias as a bf16 tensor addition (one fp32
 * addition, rounded to bf16), then, when q != NULL, the 1 x 128 group
 * quantisation of y along n exactly as bfp8_group_quant computes it:
 *   s[m, g] = fl32(max(amax_g |y|, 1e-10) / 448),  q[m, n] = e4m3(fl32(y / s)).
 *   bias  bf16 [N] or NULL.
 *   out   bf16 [M, N] row-major, or NULL to skip the bf16 output.
 *   q     e4m3 [M, N] row-major (row stride N bytes), or NULL.
 *   s     fp32 scales of q: s_col_major = 1: s[g * ld_s + m], ld_s >= M;
 *         s_col_major = 0: s[m * ld_s + g], ld_s >= ceil(N / 128).  NULL iff q is.
 * Other arguments as for bfp8_gemm_ex; the fused epilogue runs on the wide
 * schedule with the stream-K split (options.schedule and options.k_split are
 * ignored when bias or q is given); workspace from
 * bfp8_gemm_fused_workspace_size.  Errors: BFP8_ERR_INVALID_ARG when out and
 * q are both NULL, q and s are not both given, or ld_s is too small;
 * BFP8_ERR_ALIGNMENT for s not 4-byte or bias not 2-byte aligned.
 */
bfp8_status bfp8_gemm_fused(const void* A, const void* B, const float* As, int as_col_major,
                            int64_t ld_as, const float* Bs, const void* bias, void* out, void* q,
                            float* s, int s_col_major, int64_t ld_s, int64_t M, int64_t N,
                            int64_t K, void* workspace, size_t workspace_bytes,
                            const bfp8_gemm_options* opt, void* stream);

/* Workspace bytes bfp8_gemm_fused needs (current device). */
bfp8_status bfp8_gemm_fused_workspace_size(int64_t M, int64_t N, int64_t K,
                                           const bfp8_gemm_options* opt, int operands_unaligned,
                                           size_t* bytes);

/*
 * bfp8_linear -- the whole W8A8 blocked linear layer from bf16 activations in
 * one call:
 *   out = bfp8_gemm(q, B, s, Bs)  with  (q, s) = bfp8_group_quant(x, group 128,
 *   column-major scales)
 * (per_token_group_quant_fp8 followed by w8a8_block_fp8_matmul, the two steps
 * of the vLLM PR 49932 digest's blocked FP8 linear), bitwise what those two
 * calls give with the same options.  Two kernels: the quantisation writes q
 * and s into the workspace, and the GEMM, launched behind it with
 * programmatic dependent launch, streams the weights while it runs.
 *   x    bf16 [M, K], row stride ld_x elements (ld_x >= K), 2-byte aligned.
 *   B, Bs, out, M, N, K, opt, stream as for bfp8_gemm_ex (opt.prefetch_weights
 *        is always on).
 *   workspace / workspace_bytes
 *        at least bfp8_linear_workspace_size bytes, 256-byte aligned, zero-filled
 *        once after allocation: its first part serves the GEMM as for
 *        bfp8_gemm (left ready for the next call), the rest holds q and s.
 * Errors: BFP8_ERR_INVALID_ARG / ALIGNMENT / WORKSPACE as for bfp8_gemm_ex.
 */
bfp8_status bfp8_linear(const void* x, int64_t ld_x, const void* B, const float* Bs, void* out,
                        int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                        const bfp8_gemm_options* opt, void* stream);

/* Workspace bytes bfp8_linear needs (current device); weights_unaligned: B
 * not 16-byte aligned. */
bfp8_status bfp8_linear_workspace_size(int64_t M, int64_t N, int64_t K, const bfp8_gemm_options* opt,
                                       int weights_unaligned, size_t* bytes);

/*
 * bfp8_gemm_noalloc -- bfp8_gemm for callers that cannot allocate device
 * memory.  (Not from the pages: they have no counterpart; this is a
 * convenience of this library.)
 *
 * Some callers have no way to provide the GEMM workspace: code running while a
 * stream is being captured into a CUDA graph in a mode that forbids
 * cudaMalloc, plug-ins living inside a host framework that owns every device
 * allocation through its own pool and exposes no hook to them, and
 * latency-critical loops that must not pay for an allocation or risk one
 * failing.  This entry point computes exactly what bfp8_gemm computes (same
 * arguments minus the workspace, same kernels, same results) but takes its
 * scratch from a fixed array built into the library: BFP8_NOALLOC_SCRATCH_BYTES
 * (16 MiB) of device memory that every GPU which loads the library holds until
 * the process exits.  It never calls cudaMalloc, cudaFree or any allocating
 * routine.
 *
 * Limits and rules:
 *   - Problems whose workspace (bfp8_gemm_workspace_size with default
 *     options) exceeds BFP8_NOALLOC_SCRATCH_BYTES are rejected with
 *     BFP8_ERR_WORKSPACE and a reason in bfp8_last_error(); nothing is
 *     launched.  Decode-sized problems fit (e.g. M <= 64 at N = K = 4096);
 *     large-M problems generally do not.
 *   - The first call on each device looks up the scratch's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture begins.  The address is kept for the life of
 *     the process: after cudaDeviceReset() on a device, do not call this
 *     entry point on that device again.
 *   - Every call on a device shares the one scratch array, and it keeps the
 *     previous call's contents: each call first clears (cudaMemsetAsync on
 *     `stream`) the part that must start at zero.  Calls whose kernels can
 *     overlap on the GPU (different streams without ordering between them)
 *     race on the scratch and give wrong results; serialise them.
 */
#define BFP8_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
bfp8_status bfp8_gemm_noalloc(const void* A, const void* B, const float* As, int as_col_major,
                              int64_t ld_as, const float* Bs, void* out, int64_t M, int64_t N,
                              int64_t K, void* stream);

/* ------------------------------------------------------------------------ */
/* Around the linear layers: norm, paged 8-bit cache, attention              */
/* ------------------------------------------------------------------------ */

/*
 * bfp8_rmsnorm_quant -- the root-mean-square norm before a linear layer, with
 * the residual's addition before it and the layer's input quantisation after
 * it, in one pass.  For every row m:
 *   h[k]  = x[m, k] + residual[m, k]                 (residual NULL: h = x)
 *   residual_out[m, k] = h[k] in x's type            (residual_out NULL: not written)
 *   y[k]  = h[k] * rsqrt(sum_k h[k]^2 / K + eps) * weight[k]
 *   y_out[m, k] = bf16(y[k])                         (y_out NULL: not written)
 *   q[m, k], s[m, g]: the 1 x 128 group quantisation of the unrounded y
 *                     (as bfp8_group_quant_ex)       (q and s NULL: not written)
 * All of it in fp32; each output is rounded once (h is not rounded to x's type
 * before the norm, nor y to bf16 before the quantisation).
 *   x             [M, K] bf16 or fp32 (in_dtype), row stride ld_x elements.
 *   residual      [M, K] of x's type, row stride ld_r, or NULL.
 *   residual_out  [M, K] of x's type, row stride ld_ro, or NULL; may be
 *                 `residual` or `x` itself (same stride), else no overlap.
 *   weight        [K] bf16 or fp32 (weight_dtype), or NULL (ones).
 *   y_out         bf16 [M, K], row stride ld_y, or NULL.
 *   q, ld_q, s, ld_s, col_major, scale_fmt   as for bfp8_group_quant_ex.
 * Any M >= 0 and 1 <= K <= 2^20 (M == 0 launches nothing).  No alignment
 * beyond the element size is required; K % 8 == 0 with 16-byte aligned rows
 * takes the vectorised path.  Errors: BFP8_ERR_INVALID_ARG when there is
 * nothing to write (residual_out, y_out and q all NULL), q and s are not both
 * given, eps is negative or not finite, or a stride is too small.
 */
bfp8_status bfp8_rmsnorm_quant(const void* x, int in_dtype, int64_t ld_x, const void* residual,
                               int64_t ld_r, void* residual_out, int64_t ld_ro,
                               const void* weight, int weight_dtype, float eps, int64_t M,
                               int64_t K, void* y_out, int64_t ld_y, int col_major, int scale_fmt,
                               void* q, int64_t ld_q, float* s, int64_t ld_s, void* stream);

/*
 * A paged cache of keys and values in e4m3, one fp32 scale per (token, kv
 * head): value = code * scale, scales not negative (the attention takes scales
 * of values from 2^-95 to 2^126, and 0; those that bfp8_kv_cache_write makes
 * of finite rows lie between 2^-43 and 2^120).  Token `o` of page `p`, kv head `h`:
 *   codes  k + p * stride_page + h * stride_head + o * stride_token, head_dim bytes
 *   scale  k_scale[p * scale_stride_page + h * scale_stride_head + o]
 * and the same offsets in v and v_scale.  A slot is p * page_size + o.
 * page_size 16, 32, 64, 128 or 256; head_dim 64 or 128; code strides in bytes
 * and multiples of 16 (stride_token >= head_dim); scale strides in floats and
 * multiples of 4; all four pointers 16-byte aligned.  Both [page, head, token,
 * dim] and [page, token, head, dim] orders of the codes, and keys and values
 * interleaved by page, are strides of this form.
 */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int64_t num_pages;
  int page_size;
  int num_kv_heads;
  int head_dim;
  int reserved;
  int64_t stride_page, stride_head, stride_token;
  int64_t scale_stride_page, scale_stride_head;
} bfp8_kv_cache;

/*
 * bfp8_kv_cache_write -- quantises T new tokens' keys and values into the
 * cache: for every token t and kv head h, scale = max(amax, 1e-10) / 448 over
 * the head's elements (rounded up to a power of two for BFP8_SCALE_UE8M0) and
 * codes = e4m3(x / scale), the arithmetic of bfp8_group_quant_ex with the head
 * as the group.
 *   k, v   [T, num_kv_heads, head_dim] bf16 or fp32 (in_dtype) with token and
 *          head strides >= 0 in elements (e.g. columns of a fused projection's
 *          output); element strides 1.
 *   slots  device int64 [T]: where token t goes; a negative slot skips the
 *          token.  Slots of one call are distinct.  A slot past the last page
 *          writes nothing and records BFP8_DEV_BAD_CACHE_INDEX.
 * T == 0 launches nothing.
 */
bfp8_status bfp8_kv_cache_write(const void* k, const void* v, int in_dtype, int64_t k_stride_token,
                                int64_t k_stride_head, int64_t v_stride_token,
                                int64_t v_stride_head, const int64_t* slots, int64_t T,
                                int scale_fmt, const bfp8_kv_cache* cache, void* stream);

/*
 * bfp8_kv_cache_read -- k_out[t, h, :] = code * scale of slot slots[t], rounded
 * once to out_dtype (bf16 or fp32), and v_out likewise; [T, num_kv_heads,
 * head_dim] with token strides in elements and heads contiguous.  k_out or
 * v_out may be NULL (not both).  A negative slot gives zeros; a slot past the
 * last page gives zeros and records BFP8_DEV_BAD_CACHE_INDEX.
 */
bfp8_status bfp8_kv_cache_read(const bfp8_kv_cache* cache, const int64_t* slots, int64_t T,
                               int out_dtype, void* k_out, int64_t k_stride_token, void* v_out,
                               int64_t v_stride_token, void* stream);

/*
 * bfp8_paged_attention -- attention of each sequence's newest tokens over its
 * whole context in the paged cache (which already holds the new tokens).
 * Sequence b has q_len = cu_q[b+1] - cu_q[b] new tokens, rows cu_q[b] .. of q,
 * and a context of kv_lens[b] tokens; token j of it is at page
 * block_table[b * ld_table + j / page_size], offset j % page_size.  New token
 * i stands at position p = kv_lens[b] - q_len + i and sees the tokens
 *   0 <= j <= p                     (causal = 1; causal = 0: 0 <= j < kv_lens[b])
 *   j > p - window                  (window > 0; 0: no window)
 * Query head h reads kv head h / (num_heads / num_kv_heads).
 *   S_j   = softmax_scale * q . k_j,   w = softmax(S over the tokens seen)
 *   out   = sum_j w_j v_j,   lse = log sum_j exp(S_j)   (natural logarithm)
 * A row that sees no token (q_len > kv_lens[b], an empty context) gets out = 0
 * and lse = -infinity.  Queries, keys and values that are not finite reach only
 * the rows that see them.  Softmax and sums are fp32; the products run on the
 * tensor cores from the e4m3 codes and the bf16 queries (elements smaller than
 * 2^-17 of their row's largest may be lost), with the weights
 * rounded to fp16 (11 bits) for the second product.
 *   q, out   bf16 [total_q, num_heads, head_dim] with token and head strides
 *            in elements (element stride 1; 16-byte aligned pointers and
 *            strides that are multiples of 8).
 *   lse      fp32 [total_q, num_heads] contiguous, or NULL.
 *   block_table  device int32 [batch, max_pages], row stride ld_table.
 *   cu_q     device int32 [batch + 1], non-decreasing, cu_q[0] >= 0,
 *            cu_q[batch] <= total_q.  Rows outside every sequence are not written.
 *   kv_lens  device int32 [batch].
 *   max_q_len, max_kv_len   host upper bounds of the lengths (they size the
 *            launch; the lengths themselves stay on the device, so that a
 *            captured graph serves other lengths within the bounds).
 *   workspace  as for bfp8_gemm (zero-filled once, left ready by every call;
 *            one buffer may serve both), at least
 *            bfp8_paged_attention_workspace_size bytes, 256-byte aligned.
 * Page numbers outside the cache, and lengths outside the bounds, give
 * unspecified outputs for their sequence, never a fault; page numbers are also
 * recorded as BFP8_DEV_BAD_CACHE_INDEX.  Results are deterministic.
 * batch == 0 or total_q == 0 launches nothing; max_q_len and max_pages may then
 * be 0 too.
 */
typedef struct {
  const void* q;
  void* out;
  float* lse;
  int64_t total_q;
  int num_heads;
  int batch;
  int64_t q_stride_token, q_stride_head, out_stride_token, out_stride_head;
  const int32_t* block_table;
  int64_t ld_table;
  int max_pages;
  int max_q_len;
  int64_t max_kv_len;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  float softmax_scale;
  int causal;
  int window;
  int reserved;
} bfp8_attention_args;

bfp8_status bfp8_paged_attention(const bfp8_attention_args* args, const bfp8_kv_cache* cache,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes bfp8_paged_attention needs on the current device for up to
 * max_q_len new tokens a sequence. */
bfp8_status bfp8_paged_attention_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                                int max_q_len, size_t* bytes);

/*
 * bfp8_shared_prefix_attention -- bfp8_paged_attention for a batch whose
 * sequences begin with the same text: the tokens of a shared prefix are read
 * once for all rows that see them, where a block table with the same pages in
 * many rows would have them read once a sequence.  Prefix f has lens[f] tokens
 * on the pages block_table[f * ld_table ..] and is seen whole by the rows
 * cu_q[f] .. cu_q[f+1] of q (usually those of neighbouring sequences); a row
 * outside cu_q[0] .. cu_q[prefixes] sees no prefix.  The sequences' own tokens (args) are
 * what comes behind the prefix: kv_lens and block_table count and hold them alone,
 * and a row sees them as in bfp8_paged_attention, so that it stands at
 * position lens[f] + kv_lens[b] - q_len + i of the whole.  Out and lse are those of
 * one softmax over all tokens that a row sees; a row that sees none of
 * either part gets 0 and -infinity.
 *   args     as for bfp8_paged_attention, with window = 0 (BFP8_ERR_INVALID_ARG else).
 *   prefix   block_table, cu_q [prefixes + 1] (non-decreasing, from 0 to total_q at most) and
 *            lens [prefixes] are device int32; max_q_len bounds the rows of one
 *            prefix (cu_q[f+1] - cu_q[f]), max_len the lens.  prefixes == 0: bfp8_paged_attention.
 *   workspace  as for bfp8_paged_attention, bfp8_shared_prefix_attention_workspace_size
 *            bytes: the part over the prefix (and in some calls that over the own tokens) is held
 *            there in fp32 for every row.
 * The output is rounded once.  Page numbers and lengths as for bfp8_paged_attention; rows of
 * a prefix past its bound max_q_len have unspecified outputs.  Results are deterministic.
 */
typedef struct {
  const int32_t* block_table;
  int64_t ld_table;
  int max_pages;
  int prefixes;
  const int32_t* cu_q;
  const int32_t* lens;
  int max_q_len;
  int reserved;
  int64_t max_len;
} bfp8_prefix_args;

bfp8_status bfp8_shared_prefix_attention(const bfp8_attention_args* args, const bfp8_prefix_args* prefix,
                                         const bfp8_kv_cache* cache, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* Workspace bytes bfp8_shared_prefix_attention needs on the current device for up
 * to max_prefix_q_len rows a prefix, max_q_len new tokens a sequence and total_q rows.  (A
 * call with fewer new tokens than the bound may compute its parts one after the other where the
 * bytes of its own bounds would have let them run beside each other.) */
bfp8_status bfp8_shared_prefix_attention_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                                        int max_prefix_q_len, int max_q_len,
                                                        int64_t total_q, size_t* bytes);

/*
 * bfp8_kv_cache_weigh -- how much attention every cached token received: to the
 * sum of token j and kv head h is added
 *   sum over the query heads of h, over the new tokens i that see j, of exp(softmax_scale * q_i . k_j - lse_i)
 * where lse is what an attention call returned for these rows (of
 * bfp8_shared_prefix_attention too, whose softmax runs over the prefix as well: then the
 * sequences' own tokens are weighed with the arguments of that call, the prefix's with
 * its table, its cu_q and lens, and causal = 0).  All in fp32, from
 * the bf16 queries and the codes.
 *   args     as for bfp8_paged_attention; out and its strides are not used,
 *            lse [total_q, num_heads] is an input, q strides are at least head_dim.
 *   weights  fp32 sums, one for every token of the cache's pages and kv head: token o of
 *            page p at weights[p * weights_stride_page + h * weights_stride_head + o];
 *            strides in floats, at least page_size.  4-byte aligned.
 *   accumulate  1: the sums of the tokens that were cached before are added to, those of
 *            the new tokens (causal = 1: the last q_len of the context) begin here,
 *            whatever their places held; 0: the sums of the whole context begin here
 *            (0 where no row sees a token).
 * A sequence without new tokens keeps its sums.  Rows with a query, a key or an lse that is not a
 * number make the sums of the tokens that they see NaN, and of no others.
 *   workspace  as for bfp8_paged_attention, bfp8_kv_cache_weigh_workspace_size bytes.
 * Sequences of one call have no page in common (the sums of a page in two tables would be those of
 * either).  Page numbers and lengths as for bfp8_paged_attention; the sums of a token on a
 * page outside the cache go nowhere.  Results are deterministic.
 */
bfp8_status bfp8_kv_cache_weigh(const bfp8_attention_args* args, const bfp8_kv_cache* cache,
                                float* weights, int64_t weights_stride_page,
                                int64_t weights_stride_head, int accumulate, void* workspace,
                                size_t workspace_bytes, void* stream);

bfp8_status bfp8_kv_cache_weigh_workspace_size(int num_heads, int num_kv_heads, int head_dim,
                                               int max_q_len, size_t* bytes);

/*
 * bfp8_kv_cache_evict -- shortens sequences to `budget` tokens.  A sequence of
 * n = kv_lens[b] > budget tokens keeps, for each kv head by itself, its first
 * `first` and its last `recent` tokens and of the others the budget - first -
 * recent with the largest weights (as bfp8_kv_cache_weigh sums them; of equal
 * ones, those of lower position; a NaN counts as larger than any number).  They
 * keep their order: the i-th of them becomes token i of the shortened sequence,
 * with its codes, scales and weight.  What it saw of positions (a rotary
 * encoding) was applied before it was cached and stays as it was.
 * new_lens[b] = min(n, budget).
 *   block_table  device int32 [batch, max_pages], row stride ld_table.
 *   out_table    device int32 [batch, max_out_pages], row stride ld_out: the pages that the
 *            tokens move to, max_out_pages * page_size >= min(budget, max_kv_len).  None of them is among the
 *            pages that block_table holds for the call's sequences.  A sequence of at
 *            most budget tokens is copied whole.  The pages that it came from are left as they were.
 *            NULL, or block_table itself (the same address, and the same stride unless batch == 1): in place,
 *            to the first pages of block_table (a sequence of at most budget tokens stays as it is);
 *            places behind the budget are left as they were.
 *   weights  as for bfp8_kv_cache_weigh.
 *   kv_lens, new_lens   device int32 [batch], not overlapping.
 *   max_kv_len   host upper bound of the lengths.
 *   budget >= 1, first >= 0, recent >= 0, first + recent <= budget.
 *   workspace  as for bfp8_paged_attention, bfp8_kv_cache_evict_workspace_size bytes.
 * batch * num_kv_heads is at most 65535.  Sequences of one call have no page in common.
 * A page number outside the cache is recorded as BFP8_DEV_BAD_CACHE_INDEX and its tokens
 * are not moved; lengths outside the bounds are taken at the bounds.
 * batch == 0 launches nothing.
 */
typedef struct {
  float* weights;
  int64_t weights_stride_page, weights_stride_head;
  const int32_t* block_table;
  int64_t ld_table;
  const int32_t* out_table;
  int64_t ld_out;
  int max_pages, max_out_pages;
  const int32_t* kv_lens;
  int32_t* new_lens;
  int64_t max_kv_len;
  int64_t budget, recent, first;
  int batch;
  int reserved;
} bfp8_evict_args;

bfp8_status bfp8_kv_cache_evict(const bfp8_evict_args* args, const bfp8_kv_cache* cache, void* workspace,
                                size_t workspace_bytes, void* stream);

bfp8_status bfp8_kv_cache_evict_workspace_size(int batch, int num_kv_heads, int64_t max_kv_len,
                                               int64_t budget, size_t* bytes);

/* ------------------------------------------------------------------------ */
/* Status and diagnostics                                                    */
/* ------------------------------------------------------------------------ */

/* Reason for the last failure on the calling thread ("" if none). */
const char* bfp8_last_error(void);

/* Static name of a status code. */
const char* bfp8_status_string(int status);

/* Synchronises the current device and reads the library's device-side failure
 * word for it; clears it when `clear` is nonzero.  The word holds the first
 * failure a kernel reported since the last clear: */
#define BFP8_DEV_OK 0                       /* none */
#define BFP8_DEV_TIMEOUT_PRODUCER 1         /* a bounded wait gave up: operand loader */
#define BFP8_DEV_TIMEOUT_MMA 2              /*   MMA issuer */
#define BFP8_DEV_TIMEOUT_EPILOGUE 3         /*   promotion / epilogue warps */
#define BFP8_DEV_TIMEOUT_TAIL 4             /*   draining copies before exit */
#define BFP8_DEV_BAD_GROUPED_LAYOUT 5       /* bfp8_gemm_grouped: invalid grouped_layout */
#define BFP8_DEV_BAD_CACHE_INDEX 6          /* a slot or page number outside the cache */
/* After a timeout code, a workspace the call used may hold non-zero counters:
 * zero it before reusing it. */
bfp8_status bfp8_device_status(int* code, int clear);

/* The number of the graph capture that `stream` is part of, 0 when it is not
 * capturing.  For callers that keep workspaces: a buffer that a captured call
 * was given has to outlive the graph, and one that was allocated and zeroed
 * within a capture is zero only when that graph runs. */
bfp8_status bfp8_stream_capture_id(void* stream, unsigned long long* id);

/* Self-test of the bounded wait every kernel uses: launches one warp that
 * waits on a shared-memory barrier nothing ever arrives on, giving up after
 * `limit_cycles` SM cycles.  Synchronises the stream and returns
 * BFP8_ERR_DEVICE_TIMEOUT when the wait gave up as designed (and *elapsed
 * holds the cycles it waited), BFP8_OK if the barrier completed. */
bfp8_status bfp8_selftest_bounded_wait(uint64_t limit_cycles, uint64_t* elapsed, void* stream);

int bfp8_version(void);

#ifdef __cplusplus
}
#endif
#endif /* BFP8_H_ */
