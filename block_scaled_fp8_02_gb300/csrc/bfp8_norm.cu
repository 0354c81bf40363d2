// bfp8_norm.cu -- residual addition, root-mean-square norm and the next linear
// layer's 1 x 128 group quantisation in one pass (sm_103a).
//
//   h = x + r,  y = h * rsqrt(mean(h^2) + eps) * w,
//   s_g = max(amax_g |y|, 1e-10) / 448,  q = e4m3(y / s_g)
//
// One CTA takes a row at a time and keeps its h in registers between the sum
// of squares and the quantisation, so x and r are read once; a thread holds
// chunks of 8 elements, sixteen neighbouring lanes a 128-element group, whose
// amax is four shuffles.  Bound by memory: 7.03 bytes an element for bf16 with
// a residual (x, r in, r out, codes and scales out).  8192 rows of 5120 take
// 58.6 us, 5.0 TB/s or 0.74 of the measured copy rate, with the schedulers busy
// 67% of the cycles: the arithmetic that makes every code the correctly rounded
// quotient's stands beside the loads.  One row takes 3.0 us, a launch's chain.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "bfp8_e4m3.cuh"
#include "bfp8_internal.h"
#include "bfp8_ptx.cuh"
#include "bfp8_vec8.cuh"

namespace bfp8 {

namespace {

struct NormArgs {
  const void* x;
  const void* r;            // or nullptr
  void* ro;                 // or nullptr; may alias x or r
  const void* w;            // or nullptr
  __nv_bfloat16* y;         // or nullptr
  uint8_t* q;               // or nullptr
  float* s;
  int64_t ld_x, ld_r, ld_ro, ld_y, ld_q, ld_s;
  int64_t M;
  int32_t K;
  int32_t w_f32, col_major;
  int32_t vec;              // x, r, ro, y rows and w are 16-byte aligned, q rows 8-byte
  float eps;
};

// The output half of a chunk: y (optional), codes and scale of 8 elements at
// column k; every lane of the warp calls it (lanes past K with n <= 0).
template <bool kUe8m0>
__device__ __forceinline__ void emit(const NormArgs& a, int64_t row, int k, int n, float (&h)[8],
                                     float inv) {
  if (a.w != nullptr) {
    float w[8];
    if (a.w_f32) load8<true>(static_cast<const float*>(a.w) + k, a.vec, n, w);
    else load8<false>(static_cast<const uint16_t*>(a.w) + k, a.vec, n, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __fmul_rn(__fmul_rn(h[e], inv), w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __fmul_rn(h[e], inv);
  }
  if (a.y != nullptr) store8<false>(a.y + row * a.ld_y + k, a.vec, n, h);
  if (a.q == nullptr) return;
  float scale;
  uint32_t lo, hi;
  quant8<16, kUe8m0>(h, scale, lo, hi);
  if (n <= 0) return;
  uint8_t* q = a.q + row * a.ld_q + k;
  if (a.vec && n >= 8) {
    *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) q[e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
  }
  if ((k & 127) == 0) {
    const int64_t g = k >> 7;
    a.s[a.col_major ? g * a.ld_s + row : row * a.ld_s + g] = scale;
  }
}

// The row's sum of squares from every thread's part, added in the same order by
// all; `part` alternates between rows, so one barrier a row is enough.
__device__ __forceinline__ float row_inv(float ss, float* part, const NormArgs& a) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  if (lane == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = part[0];
  for (int i = 1; i < nw; ++i) ss += part[i];
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(a.K)), a.eps));
}

// NC: chunks of 8 elements a thread holds.  The next row's loads are under way
// while this one waits for its sum and is quantised (8192 x 5120 bf16: 85.5 us
// without).  72 registers let two blocks of fp32 rows of up to 7280 share an SM (1000
// x 7168: 19.3 us against 20.6 with 76); 48 for bf16 spill and cost 8%.
template <bool kF32, bool kUe8m0, int NC>
__global__ void __maxnreg__(NC == 1 ? 64 : NC == 2 ? (kF32 ? 72 : 64) : 128) rmsnorm_quant_kernel(const __grid_constant__ NormArgs a) {
  using T = typename std::conditional<kF32, float, uint16_t>::type;
  __shared__ float part[2][32];
  const int tid = threadIdx.x, nt = blockDim.x;
  griddep_launch_dependents();
  griddep_wait();
  Raw8<kF32> rx[NC], rr[NC];
  auto fetch = [&](int64_t row) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (tid + c * nt) * 8, n = row < a.M ? a.K - k : 0;
      rx[c].load(x + k, a.vec, n);
      if (r != nullptr) rr[c].load(r + k, a.vec, n);
    }
  };
  constexpr bool kAhead = !(kF32 && NC == 4);          // (no registers left for it there)
  fetch(blockIdx.x);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, buf ^= 1) {
    T* ro = a.ro != nullptr ? static_cast<T*>(a.ro) + row * a.ld_ro : nullptr;
    float h[NC][8];
    float ss = 0.f;
    if (!kAhead && row != blockIdx.x) fetch(row);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      rx[c].get(h[c]);
      if (a.r != nullptr) {
        float t[8];
        rr[c].get(t);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = __fadd_rn(h[c][e], t[e]);
      }
    }
    if (kAhead) fetch(row + gridDim.x);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
      const int k = (tid + c * nt) * 8;
      if (ro != nullptr) store8<kF32>(ro + k, a.vec, a.K - k, h[c]);
    }
    const float inv = row_inv(ss, part[buf], a);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = (tid + c * nt) * 8;
      emit<kUe8m0>(a, row, k, a.K - k, h[c], inv);
    }
  }
}

// Rows that do not fit the registers of a CTA, read twice (the second time from L2).
template <bool kF32, bool kUe8m0>
__global__ void __launch_bounds__(1024) rmsnorm_quant_long_kernel(const __grid_constant__ NormArgs a) {
  using T = typename std::conditional<kF32, float, uint16_t>::type;
  __shared__ float part[2][32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch_dependents();
  griddep_wait();
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, buf ^= 1) {
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* r = a.r != nullptr ? static_cast<const T*>(a.r) + row * a.ld_r : nullptr;
    T* ro = a.ro != nullptr ? static_cast<T*>(a.ro) + row * a.ld_ro : nullptr;
    auto load_h = [&](int k, float (&h)[8]) {
      load8<kF32>(x + k, a.vec, a.K - k, h);
      if (r != nullptr) {
        float t[8];
        load8<kF32>(r + k, a.vec, a.K - k, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(h[e], t[e]);
      }
    };
    float h[8], ss = 0.f;
    for (int k = tid * 8; k < a.K; k += nt * 8) {
      load_h(k, h);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[e], h[e], ss);
    }
    const float inv = row_inv(ss, part[buf], a);
    for (int k0 = warp * 256; k0 < a.K; k0 += nt * 8) {       // whole warps: emit shuffles
      const int k = k0 + lane * 8;
      load_h(k, h);
      if (ro != nullptr) store8<kF32>(ro + k, a.vec, a.K - k, h);
      emit<kUe8m0>(a, row, k, a.K - k, h, inv);
    }
  }
}

template <bool kF32, bool kUe8m0>
cudaError_t launch_norm(const NormArgs& a, int num_sms, cudaStream_t stream) {
  // A chunk a thread where rows are few (all the latency there is to save) or short; else two and
  // more, whose loads hide one another's time.
  const int chunks = (a.K + 7) / 8;
  const bool few = a.M <= 2 * static_cast<int64_t>(num_sms);
  const int nc = chunks <= 1024 && (few || chunks <= 64) ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 0;
  const int threads = nc ? ((chunks + nc - 1) / nc + 31) / 32 * 32 : 1024;
  auto kernel = nc == 1   ? rmsnorm_quant_kernel<kF32, kUe8m0, 1>
                : nc == 2 ? rmsnorm_quant_kernel<kF32, kUe8m0, 2>
                : nc == 4 ? rmsnorm_quant_kernel<kF32, kUe8m0, 4>
                          : rmsnorm_quant_long_kernel<kF32, kUe8m0>;
  // as many blocks as are resident, asked for once a kernel and size
  static std::atomic<int> resident[4][33];
  std::atomic<int>& known = resident[nc == 4 ? 3 : nc][threads / 32];
  int per_sm = known.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e != cudaSuccess) return e;
    known.store(per_sm, std::memory_order_relaxed);
  }
  int64_t blocks = static_cast<int64_t>(per_sm) * num_sms;
  if (blocks > a.M) blocks = a.M;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

inline bool off_align(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

}  // namespace

}  // namespace bfp8

extern "C" bfp8_status bfp8_rmsnorm_quant(const void* x, int in_dtype, int64_t ld_x,
                                          const void* residual, int64_t ld_r, void* residual_out,
                                          int64_t ld_ro, const void* weight, int weight_dtype,
                                          float eps, int64_t M, int64_t K, void* y_out,
                                          int64_t ld_y, int col_major, int scale_fmt, void* q,
                                          int64_t ld_q, float* s, int64_t ld_s, void* stream) {
  using namespace bfp8;
  auto bad = [](const char* fmt, auto... v) { return set_last_errorf(BFP8_ERR_INVALID_ARG, fmt, v...); };
  if (in_dtype != BFP8_IN_BF16 && in_dtype != BFP8_IN_F32)
    return bad("in_dtype = %d (expected BFP8_IN_BF16 or BFP8_IN_F32)", in_dtype);
  if (weight_dtype != BFP8_IN_BF16 && weight_dtype != BFP8_IN_F32)
    return bad("weight_dtype = %d (expected BFP8_IN_BF16 or BFP8_IN_F32)", weight_dtype);
  if (scale_fmt != BFP8_SCALE_FP32 && scale_fmt != BFP8_SCALE_UE8M0)
    return bad("scale_fmt = %d (expected BFP8_SCALE_FP32 or BFP8_SCALE_UE8M0)", scale_fmt);
  if (col_major != 0 && col_major != 1) return bad("col_major = %d (expected 0 or 1)", col_major);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return bad("eps = %g (expected finite and >= 0)", (double)eps);
  if (M < 0 || K < 1 || K > (int64_t{1} << 20))
    return bad("M = %lld, K = %lld (expected M >= 0, 1 <= K <= 2^20)", (long long)M, (long long)K);
  if ((q == nullptr) != (s == nullptr) && M > 0) return bad("q and s go together (q=%p s=%p)", q, (void*)s);
  if (M == 0) return set_last_error(BFP8_OK, "");
  if (!x) return bad("x is null");
  if (!residual_out && !y_out && !q) return bad("nothing to write: residual_out, y_out and q are null");
  const int64_t G = (K + 127) / 128;
  if (ld_x < K) return bad("ld_x = %lld < K = %lld", (long long)ld_x, (long long)K);
  if (residual && ld_r < K) return bad("ld_r = %lld < K = %lld", (long long)ld_r, (long long)K);
  if (residual_out && ld_ro < K) return bad("ld_ro = %lld < K = %lld", (long long)ld_ro, (long long)K);
  if (residual_out && ((residual_out == residual && ld_ro != ld_r) || (residual_out == x && ld_ro != ld_x)))
    return bad("residual_out in place needs the stride of what it replaces");
  if (y_out && ld_y < K) return bad("ld_y = %lld < K = %lld", (long long)ld_y, (long long)K);
  if (q && ld_q < K) return bad("ld_q = %lld < K = %lld", (long long)ld_q, (long long)K);
  if (q && (col_major ? ld_s < M : ld_s < G))
    return bad("ld_s = %lld too small for the %s layout", (long long)ld_s, col_major ? "column-major" : "row-major");
  const int es = in_dtype == BFP8_IN_F32 ? 4 : 2, ws = weight_dtype == BFP8_IN_F32 ? 4 : 2;
  if (off_align(x, es) || off_align(residual, es) || off_align(residual_out, es) || off_align(weight, ws) ||
      off_align(y_out, 2) || off_align(s, 4))
    return set_last_errorf(BFP8_ERR_ALIGNMENT, "a pointer is not aligned to its element size");
  int sms = 0;
  int* err = nullptr;
  const bfp8_status st = device_for_call(&sms, &err);
  if (st != BFP8_OK) return st;
  NormArgs a{};
  a.x = x;
  a.r = residual;
  a.ro = residual_out;
  a.w = weight;
  a.y = static_cast<__nv_bfloat16*>(y_out);
  a.q = static_cast<uint8_t*>(q);
  a.s = s;
  a.ld_x = ld_x;
  a.ld_r = ld_r;
  a.ld_ro = ld_ro;
  a.ld_y = ld_y;
  a.ld_q = ld_q;
  a.ld_s = ld_s;
  a.M = M;
  a.K = static_cast<int32_t>(K);
  a.w_f32 = weight_dtype == BFP8_IN_F32;
  a.col_major = col_major;
  a.eps = eps;
  auto rows16 = [&](const void* p, int64_t ld, int e) { return !p || (!off_align(p, 16) && ld * e % 16 == 0); };
  a.vec = K % 8 == 0 && rows16(x, ld_x, es) && rows16(residual, ld_r, es) && rows16(residual_out, ld_ro, es) &&
          rows16(y_out, ld_y, 2) && !off_align(weight, 16) && (!q || (!off_align(q, 8) && ld_q % 8 == 0));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool f32 = in_dtype == BFP8_IN_F32, ue = scale_fmt == BFP8_SCALE_UE8M0;
  const cudaError_t e = f32 ? (ue ? launch_norm<true, true>(a, sms, cs) : launch_norm<true, false>(a, sms, cs))
                            : (ue ? launch_norm<false, true>(a, sms, cs) : launch_norm<false, false>(a, sms, cs));
  if (e != cudaSuccess) return set_last_errorf(BFP8_ERR_CUDA, "norm launch: %s", cudaGetErrorString(e));
  return set_last_error(BFP8_OK, "");
}
