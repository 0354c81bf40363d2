// bfp8_vec8.cuh -- chunks of 8 elements in fp32 registers: guarded loads and
// stores of bf16 / fp32 rows, and the group quantisation of chunks spread over
// neighbouring lanes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "bfp8_e4m3.cuh"
#include "bfp8_ptx.cuh"

namespace bfp8 {

// v = the 8 elements at p as fp32; `n` of them exist (any value; <= 0: none),
// the rest read as zero.  vec: p is 16-byte aligned.
template <bool kF32>
__device__ __forceinline__ void load8(const void* p, int vec, int n, float (&v)[8]) {
  if (vec && n >= 8) {
    const uint4 a = *static_cast<const uint4*>(p);
    if constexpr (kF32) {
      const uint4 b = *(static_cast<const uint4*>(p) + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = 0.f;
    if (e < n) {
      if constexpr (kF32) v[e] = static_cast<const float*>(p)[e];
      else v[e] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e]) << 16);
    }
  }
}

// The same in two steps, so that other work can stand between a load and its use.
template <bool kF32>
struct Raw8 {
  uint4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int vec, int n) {
    if (vec && n >= 8) {
#pragma unroll
      for (int i = 0; i < (kF32 ? 2 : 1); ++i) w[i] = static_cast<const uint4*>(p)[i];
      return;
    }
    uint32_t t[kF32 ? 8 : 4];
#pragma unroll
    for (int i = 0; i < (kF32 ? 8 : 4); ++i) t[i] = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) {
        if constexpr (kF32) t[e] = static_cast<const uint32_t*>(p)[e];
        else t[e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e]) << (16 * (e & 1));
      }
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i) w[i] = make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (kF32) {
      const uint32_t t[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(t[e]);
    } else {
      const uint32_t t[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(t[e] << 16);
        v[2 * e + 1] = __uint_as_float(t[e] & 0xFFFF0000u);
      }
    }
  }
};

// The first n of 8 fp32 values to p, as fp32 or rounded to bf16.
template <bool kF32>
__device__ __forceinline__ void store8(void* p, int vec, int n, const float (&v)[8]) {
  if (vec && n >= 8) {
    if constexpr (kF32) {
      static_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      static_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *static_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) {
      if constexpr (kF32) static_cast<float*>(p)[e] = v[e];
      else static_cast<__nv_bfloat16*>(p)[e] = __float2bfloat16_rn(v[e]);
    }
}

// Codes (8 bytes, lo then hi) and scale of a group held by LPG neighbouring
// lanes (aligned to LPG), 8 elements each; every lane of the warp calls it.
template <int LPG, bool kUe8m0>
__device__ __forceinline__ void quant8(const float (&v)[8], float& scale, uint32_t& lo, uint32_t& hi) {
  float amax = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
  for (int off = LPG / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  uint32_t pk[4];
  if constexpr (kUe8m0) {
    const Ue8m0Scale us(amax);
    scale = us.scale;
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[i] = e4m3_pair_pow2(v[2 * i], v[2 * i + 1], us.inv);
  } else {
    scale = group_scale(amax);
    const E4m3Bracket br(scale);
    uint32_t undecided = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bool u = false;
      pk[i] = e4m3_pair_bracketed(v[2 * i], v[2 * i + 1], br, u);
      undecided |= static_cast<uint32_t>(u) << i;
    }
    if (__any_sync(0xffffffffu, undecided != 0)) {      // warp-uniform branch
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (undecided & (1u << i)) pk[i] = e4m3_pair_divided(v[2 * i], v[2 * i + 1], scale);
    }
  }
  lo = pk[0] | (pk[1] << 16);
  hi = pk[2] | (pk[3] << 16);
}

// The same for 16 elements a lane: codes in four words.
template <int LPG, bool kUe8m0>
__device__ __forceinline__ void quant16(const float (&v)[16], float& scale, uint32_t (&w)[4]) {
  float amax = fabsf(v[0]);
#pragma unroll
  for (int e = 1; e < 16; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
  for (int off = LPG / 2; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  uint32_t pk[8];
  if constexpr (kUe8m0) {
    const Ue8m0Scale us(amax);
    scale = us.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) pk[i] = e4m3_pair_pow2(v[2 * i], v[2 * i + 1], us.inv);
  } else {
    scale = group_scale(amax);
    const E4m3Bracket br(scale);
    uint32_t undecided = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bool u = false;
      pk[i] = e4m3_pair_bracketed(v[2 * i], v[2 * i + 1], br, u);
      undecided |= static_cast<uint32_t>(u) << i;
    }
    if (__any_sync(0xffffffffu, undecided != 0)) {      // warp-uniform branch
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (undecided & (1u << i)) pk[i] = e4m3_pair_divided(v[2 * i], v[2 * i + 1], scale);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pk[2 * i] | (pk[2 * i + 1] << 16);
}

// fp32 values of the four e4m3 codes of a word (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&v)[4]) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b) : "r"(w));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[0]), "=f"(v[1]) : "r"(a));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[2]), "=f"(v[3]) : "r"(b));
}

}  // namespace bfp8
