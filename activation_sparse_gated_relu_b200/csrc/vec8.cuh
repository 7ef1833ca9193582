// Eight consecutive values of a row in registers: loads from bf16 or fp32,
// stores to bf16, fp32 or e4m3, and the 8-bit scale of a 128-column group.
#pragma once

#include <cuda_fp8.h>

#include "ptx_pair.cuh"

namespace sffn {

// Columns that share a scale of an 8-bit row, and the side of a weight block
// that shares one.
constexpr int Q_GROUP = 128;
// Least amax of a group: a group of zeros gets codes 0 and a finite scale.
constexpr float Q_TINY = 1e-30f;
constexpr float Q_MAX = 448.0f;   // the largest e4m3 value

template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, size_t vec) {   // vec: index of the group of eight
    const uint4* p = reinterpret_cast<const uint4*>(base) + vec * (F32 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void pairs(uint64_t (&f)[4]) const {
    if (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = pack2(__uint_as_float(v[F32 ? i : 0].x), __uint_as_float(v[F32 ? i : 0].y));
        f[2 * i + 1] = pack2(__uint_as_float(v[F32 ? i : 0].z), __uint_as_float(v[F32 ? i : 0].w));
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = pack2(bf16lo(w[i]), bf16hi(w[i]));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[F32 ? i : 0].x);
        f[4 * i + 1] = __uint_as_float(v[F32 ? i : 0].y);
        f[4 * i + 2] = __uint_as_float(v[F32 ? i : 0].z);
        f[4 * i + 3] = __uint_as_float(v[F32 ? i : 0].w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16lo(w[i]);
        f[2 * i + 1] = bf16hi(w[i]);
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void store8_bf16(void* base, size_t vec, const float (&f)[8]) {
  reinterpret_cast<uint4*>(base)[vec] =
      make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8_f32(void* base, size_t vec, const float (&f)[8]) {
  float4* p = reinterpret_cast<float4*>(base) + 2 * vec;
  p[0] = make_float4(f[0], f[1], f[2], f[3]);
  p[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// e4m3 codes of f·inv, rounded to nearest and saturated at +-448; NaN stays NaN.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// amax over the 16 lanes whose eight columns each make up a group of 128
// (lanes 0-15 and 16-31 of a warp); every lane of the warp takes part.
__device__ __forceinline__ float group_amax(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return fmaxf(m, Q_TINY);
}

}  // namespace sffn
