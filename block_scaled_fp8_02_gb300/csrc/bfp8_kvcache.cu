// bfp8_kvcache.cu -- the paged e4m3 key/value cache: quantising new tokens into
// it and reading tokens back (sm_103a).
//
//   write: s = max(amax_d |x|, 1e-10) / 448, code = e4m3(x / s) per (token, head)
//   read:  x' = code * s, one rounding
//
// A thread holds 16 elements of one (key or value, head) place and keeps that
// place from token to token, so that a token costs it a slot and two address
// sums; places that do not fill a block of 256 threads share it with the next
// tokens, those beyond it are the grid's second dimension.  Bound by memory:
// write 2 bytes in and 1 + 4 / head_dim out an element (bf16), read the other
// way round; reading 65536 tokens of 8 heads of 128 takes 65 us, 0.92 of the
// measured copy rate, writing 8192 of them 15.4 us, 0.49 of it, held up by the
// latency of the loads of one token a thread and, beside it, by the arithmetic that
// makes every code the correctly rounded quotient's (10 million warp instructions,
// issue slots 47 % full).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bfp8_devstatus.cuh"
#include "bfp8_internal.h"
#include "bfp8_kvcache.cuh"
#include "bfp8_ptx.cuh"
#include "bfp8_vec8.cuh"

namespace bfp8 {

namespace {

constexpr int kThreads = 256;
// Tokens that a reading thread's loads are issued for together, with four blocks a SM
// resident: 65536 tokens of 8 heads of 128, 65.1 us with four against 78.1 with
// two.  Writing takes one at a time: 8192 tokens 15.6 us against 16.6 with two (and 18.9
// with four), 16.5 with five blocks; there the arithmetic is what counts.
constexpr int kReadTokens = 4, kBlocksPerSm = 4;

// The places of a token: nkv x heads x (dim / 16), shared out as above.
struct Places {
  int32_t count;                      // of a token
  int32_t tokens;                     // that a block holds at once
};

struct WriteArgs {
  const void* k;
  const void* v;
  int64_t k_st, k_sh, v_st, v_sh;     // element strides
  const int64_t* slots;
  int64_t T;
  int32_t vec;
  Places pl;
  CacheView c;
  int* err;
};

template <bool kF32, bool kUe8m0, int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) kv_write_kernel(const __grid_constant__ WriteArgs a) {
  using T = typename std::conditional<kF32, float, uint16_t>::type;
  constexpr int LPR = D / 16;                         // threads of a row
  const int ti = static_cast<int>(threadIdx.x) / a.pl.count;                   // token of the block
  const int place = static_cast<int>(blockIdx.y) * kThreads + static_cast<int>(threadIdx.x) - ti * a.pl.count;
  const bool mine = ti < a.pl.tokens && place < a.pl.count;
  const int li = place % LPR, row = mine ? place / LPR : 0;
  const bool is_v = row >= a.c.heads;
  const int head = is_v ? row - a.c.heads : row;
  const T* src = (is_v ? static_cast<const T*>(a.v) + head * a.v_sh : static_cast<const T*>(a.k) + head * a.k_sh) + li * 16;
  const int64_t st = is_v ? a.v_st : a.k_st;
  uint8_t* q = (is_v ? a.c.v : a.c.k) + head * a.c.st_head + li * 16;
  float* s = (is_v ? a.c.vs : a.c.ks) + head * a.c.ss_head;
  const int64_t nslots = a.c.num_pages * a.c.page_size;
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.pl.tokens;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.pl.tokens; t0 < a.T; t0 += step) {
    const int64_t t = t0 + ti;
    const bool ok = mine && t < a.T;
    const int64_t slot = ok ? __ldg(a.slots + t) : -1;
    Raw8<kF32> x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i].load(src + (ok ? t : 0) * st + 8 * i, a.vec, ok ? 8 : 0);
    float v[16];
    x[0].get(reinterpret_cast<float(&)[8]>(v[0]));
    x[1].get(reinterpret_cast<float(&)[8]>(v[8]));
    float scale;
    uint32_t w[4];
    quant16<LPR, kUe8m0>(v, scale, w);
    if (slot < 0) continue;
    if (slot >= nslots) {
      report_failure(a.err, kDevBadCacheIndex);
      continue;
    }
    const int64_t page = slot >> a.c.page_shift, o = slot & (a.c.page_size - 1);
    *reinterpret_cast<uint4*>(q + page * a.c.st_page + o * a.c.st_tok) = make_uint4(w[0], w[1], w[2], w[3]);
    if (li == 0) s[page * a.c.ss_page + o] = scale;
  }
}

struct ReadArgs {
  void* k;                            // or nullptr
  void* v;                            // or nullptr
  int64_t k_st, v_st;                 // element strides of tokens
  const int64_t* slots;
  int64_t T;
  int32_t vec;
  Places pl;
  CacheView c;
  int* err;
};

template <bool kF32, int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  using T = typename std::conditional<kF32, float, __nv_bfloat16>::type;
  constexpr int LPR = D / 16;
  const int ti = static_cast<int>(threadIdx.x) / a.pl.count;
  const int place = static_cast<int>(blockIdx.y) * kThreads + static_cast<int>(threadIdx.x) - ti * a.pl.count;
  griddep_launch_dependents();
  griddep_wait();
  if (ti >= a.pl.tokens || place >= a.pl.count) return;
  const int li = place % LPR, row = place / LPR;
  const bool is_v = row >= a.c.heads || a.k == nullptr;
  const int head = row >= a.c.heads ? row - a.c.heads : row;
  const uint8_t* q = (is_v ? a.c.v : a.c.k) + head * a.c.st_head + li * 16;
  const float* s = (is_v ? a.c.vs : a.c.ks) + head * a.c.ss_head;
  T* dst = static_cast<T*>(is_v ? a.v : a.k) + head * D + li * 16;
  const int64_t st = is_v ? a.v_st : a.k_st;
  const int64_t nslots = a.c.num_pages * a.c.page_size;
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.pl.tokens;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.pl.tokens + ti; t0 < a.T; t0 += step * kReadTokens) {
    uint4 w[kReadTokens];
    float sc[kReadTokens];
    int64_t slot[kReadTokens];
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) slot[u] = t0 + u * step < a.T ? __ldg(a.slots + t0 + u * step) : -1;
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) {
      w[u] = make_uint4(0u, 0u, 0u, 0u);
      sc[u] = 0.f;
      if (slot[u] >= nslots) {
        report_failure(a.err, kDevBadCacheIndex);
      } else if (slot[u] >= 0) {
        const int64_t page = slot[u] >> a.c.page_shift, o = slot[u] & (a.c.page_size - 1);
        w[u] = __ldg(reinterpret_cast<const uint4*>(q + page * a.c.st_page + o * a.c.st_tok));
        sc[u] = __ldg(s + page * a.c.ss_page + o);
      }
    }
#pragma unroll
    for (int u = 0; u < kReadTokens; ++u) {
      if (t0 + u * step >= a.T) break;
      const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      T* d = dst + (t0 + u * step) * st;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8], lo[4], hi[4];
        e4m3x4_to_f32(ww[2 * h], lo);
        e4m3x4_to_f32(ww[2 * h + 1], hi);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = __fmul_rn(lo[e], sc[u]);
          v[4 + e] = __fmul_rn(hi[e], sc[u]);
        }
        store8<kF32>(d + 8 * h, a.vec, 8, v);
      }
    }
  }
}

Places places_of(int nkv, const CacheView& c) {
  Places p;
  p.count = nkv * c.heads * (c.dim / 16);
  p.tokens = p.count < kThreads ? kThreads / p.count : 1;
  return p;
}

template <typename F, typename A>
cudaError_t launch_places(F* f, const A& a, int num_sms, cudaStream_t stream) {
  const int64_t gy = (a.pl.count + kThreads - 1) / kThreads;
  int64_t gx = (a.T + a.pl.tokens - 1) / a.pl.tokens;
  const int64_t cap = (static_cast<int64_t>(num_sms) * kBlocksPerSm + gy - 1) / gy;
  if (gx > cap) gx = cap;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, a);
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

template <typename... V>
bfp8_status bad(const char* fmt, V... v) {
  return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...);
}

// Tokens x heads of one launch.
constexpr int64_t kMaxRows = int64_t{1} << 31;

}  // namespace

bfp8_status check_cache(const bfp8_kv_cache* c, CacheView* view) {
  if (!c) return bad("cache is null");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale)
    return bad("cache: null pointer (k=%p v=%p k_scale=%p v_scale=%p)", c->k, c->v, (void*)c->k_scale,
               (void*)c->v_scale);
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size)
    return bad("cache: page_size = %d (expected 16, 32, 64, 128 or 256)", c->page_size);
  if (c->head_dim != 64 && c->head_dim != 128) return bad("cache: head_dim = %d (expected 64 or 128)", c->head_dim);
  if (c->num_kv_heads < 1 || c->num_kv_heads > 65535)
    return bad("cache: num_kv_heads = %d (expected 1 .. 65535)", c->num_kv_heads);
  if (c->num_pages < 1 || c->num_pages >= (int64_t{1} << 31))
    return bad("cache: num_pages = %lld", (long long)c->num_pages);
  constexpr int64_t kMaxStride = int64_t{1} << 39;      // what a tensor map can hold
  for (int64_t s : {c->stride_page, c->stride_head, c->stride_token})
    if (s < c->head_dim || s >= kMaxStride) return bad("cache: code stride %lld (expected >= head_dim)", (long long)s);
  for (int64_t s : {c->scale_stride_page, c->scale_stride_head})
    if (s < c->page_size || s >= kMaxStride)
      return bad("cache: scale stride %lld (expected >= page_size)", (long long)s);
  if (c->stride_page % 16 || c->stride_head % 16 || c->stride_token % 16 || c->scale_stride_page % 4 ||
      c->scale_stride_head % 4)
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "cache: strides must be multiples of 16 bytes");
  if (off_align(c->k, 16) || off_align(c->v, 16) || off_align(c->k_scale, 16) || off_align(c->v_scale, 16))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "cache: pointers must be 16-byte aligned");
  view->k = static_cast<uint8_t*>(c->k);
  view->v = static_cast<uint8_t*>(c->v);
  view->ks = c->k_scale;
  view->vs = c->v_scale;
  view->num_pages = c->num_pages;
  view->st_page = c->stride_page;
  view->st_head = c->stride_head;
  view->st_tok = c->stride_token;
  view->ss_page = c->scale_stride_page;
  view->ss_head = c->scale_stride_head;
  view->page_size = c->page_size;
  view->page_shift = shift;
  view->heads = c->num_kv_heads;
  view->dim = c->head_dim;
  return BFP8_OK;
}

}  // namespace bfp8

using namespace bfp8;

extern "C" bfp8_status bfp8_kv_cache_write(const void* k, const void* v, int in_dtype,
                                           int64_t k_stride_token, int64_t k_stride_head,
                                           int64_t v_stride_token, int64_t v_stride_head,
                                           const int64_t* slots, int64_t T, int scale_fmt,
                                           const bfp8_kv_cache* cache, void* stream) {
  WriteArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  if (in_dtype != BFP8_IN_BF16 && in_dtype != BFP8_IN_F32)
    return bad("in_dtype = %d (expected BFP8_IN_BF16 or BFP8_IN_F32)", in_dtype);
  if (scale_fmt != BFP8_SCALE_FP32 && scale_fmt != BFP8_SCALE_UE8M0)
    return bad("scale_fmt = %d (expected BFP8_SCALE_FP32 or BFP8_SCALE_UE8M0)", scale_fmt);
  if (T < 0) return bad("T = %lld", (long long)T);
  if (T == 0) return set_last_error(BFP8_OK, "");
  if (!k || !v || !slots) return bad("null pointer (k=%p v=%p slots=%p)", k, v, (const void*)slots);
  for (int64_t s : {k_stride_token, k_stride_head, v_stride_token, v_stride_head})
    if (s < 0) return bad("k and v strides must not be negative (got %lld)", (long long)s);
  const int es = in_dtype == BFP8_IN_F32 ? 4 : 2;
  if (off_align(k, es) || off_align(v, es) || off_align(slots, 8))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "k, v or slots is not aligned to its element size");
  if (T >= kMaxRows / (2 * a.c.heads))
    return set_last_errorf(BFP8_ERR_UNSUPPORTED, "T x heads too large for one launch");
  int sms = 0;
  if ((st = device_for_call(&sms, &a.err)) != BFP8_OK) return st;
  a.k = k;
  a.v = v;
  a.k_st = k_stride_token;
  a.k_sh = k_stride_head;
  a.v_st = v_stride_token;
  a.v_sh = v_stride_head;
  a.slots = slots;
  a.T = T;
  a.pl = places_of(2, a.c);
  a.vec = !off_align(k, 16) && !off_align(v, 16) && k_stride_token * es % 16 == 0 &&
          k_stride_head * es % 16 == 0 && v_stride_token * es % 16 == 0 && v_stride_head * es % 16 == 0;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool f32 = in_dtype == BFP8_IN_F32, ue = scale_fmt == BFP8_SCALE_UE8M0;
  auto go = [&](auto f128, auto f64) {
    return a.c.dim == 128 ? launch_places(f128, a, sms, cs) : launch_places(f64, a, sms, cs);
  };
  const cudaError_t e =
      f32 ? (ue ? go(kv_write_kernel<true, true, 128>, kv_write_kernel<true, true, 64>)
                : go(kv_write_kernel<true, false, 128>, kv_write_kernel<true, false, 64>))
          : (ue ? go(kv_write_kernel<false, true, 128>, kv_write_kernel<false, true, 64>)
                : go(kv_write_kernel<false, false, 128>, kv_write_kernel<false, false, 64>));
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache write launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}

extern "C" bfp8_status bfp8_kv_cache_read(const bfp8_kv_cache* cache, const int64_t* slots, int64_t T,
                                          int out_dtype, void* k_out, int64_t k_stride_token,
                                          void* v_out, int64_t v_stride_token, void* stream) {
  ReadArgs a{};
  bfp8_status st = check_cache(cache, &a.c);
  if (st != BFP8_OK) return st;
  if (out_dtype != BFP8_IN_BF16 && out_dtype != BFP8_IN_F32)
    return bad("out_dtype = %d (expected BFP8_IN_BF16 or BFP8_IN_F32)", out_dtype);
  if (T < 0) return bad("T = %lld", (long long)T);
  if (T == 0) return set_last_error(BFP8_OK, "");
  if (!slots) return bad("slots is null");
  if (!k_out && !v_out) return bad("k_out and v_out are null");
  const int64_t width = static_cast<int64_t>(a.c.heads) * a.c.dim;
  if ((k_out && k_stride_token < width) || (v_out && v_stride_token < width))
    return bad("token strides must be >= num_kv_heads * head_dim");
  const int es = out_dtype == BFP8_IN_F32 ? 4 : 2;
  if (off_align(k_out, es) || off_align(v_out, es) || off_align(slots, 8))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "k_out, v_out or slots is not aligned to its element size");
  if (T >= kMaxRows / (2 * a.c.heads))
    return set_last_errorf(BFP8_ERR_UNSUPPORTED, "T x heads too large for one launch");
  int sms = 0;
  if ((st = device_for_call(&sms, &a.err)) != BFP8_OK) return st;
  a.k = k_out;
  a.v = v_out;
  a.k_st = k_stride_token;
  a.v_st = v_stride_token;
  a.slots = slots;
  a.T = T;
  a.pl = places_of(k_out && v_out ? 2 : 1, a.c);
  a.vec = !off_align(k_out, 16) && !off_align(v_out, 16) && (!k_out || k_stride_token * es % 16 == 0) &&
          (!v_out || v_stride_token * es % 16 == 0);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  auto go = [&](auto f128, auto f64) {
    return a.c.dim == 128 ? launch_places(f128, a, sms, cs) : launch_places(f64, a, sms, cs);
  };
  const cudaError_t e = out_dtype == BFP8_IN_F32 ? go(kv_read_kernel<true, 128>, kv_read_kernel<true, 64>)
                                                 : go(kv_read_kernel<false, 128>, kv_read_kernel<false, 64>);
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "cache read launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
