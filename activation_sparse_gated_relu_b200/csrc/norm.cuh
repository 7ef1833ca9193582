// Root-mean-square norm with the residual's addition, and its gradient.
//
//   s = residual + x          (stored, rounded to the residual's type)
//   y = s · rstd · w,   rstd = 1 / sqrt(mean(s^2) + eps)
//
// y uses the fp32 sum, not its stored rounding, and is rounded once: to bf16,
// to fp32 (kept), or to e4m3 codes with one fp32 scale = amax / 448 for each
// 128 columns.  The gradient for upstream dy (and ds, the gradient that
// reaches s past the norm), with g = dy·w and a = sum_j g_j s_j:
//
//   dx = rstd·g - s · a·rstd^3/d + ds,     dw = sum over rows of dy·s·rstd.
//
// Both are bound by memory: each value is read once and each result written
// once.  A row is held in the registers of a group of TPR threads (a power of
// two of 32 to 512, eight columns each, NV times), so that neither the second
// use of s nor the 8-bit scale reads anything again; groups of fewer than 256
// threads share a CTA.  Sums are fp32, in a fixed order.
#pragma once

#include "vec8.cuh"

namespace sffn {

constexpr int NORM_MAX_D = 16384;

struct NormArgs {
  const void* x;
  const void* res;     // or null
  const void* w;
  void* s;             // the sum, in the residual's type (null without one)
  void* y;
  float* scale;        // [T][ceil(d/128)] with e4m3 output
  int T, d, tpr, w_f32;
  float eps;
};

__device__ __forceinline__ void load_w8(const void* w, int w_f32, int vec, float (&f)[8]) {
  if (w_f32) {
    Raw8<true> r;
    r.load(w, vec);
    r.get(f);
  } else {
    Raw8<false> r;
    r.load(w, vec);
    r.get(f);
  }
}

// Sums of v[0..N) over the row's threads: warp sums to shared memory, then
// every thread adds its row's warps in order.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[16], int warps_per_row) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (warps_per_row == 1) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][warp] = v[i];
  __syncthreads();
  const int w0 = warp / warps_per_row * warps_per_row;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int k = 0; k < warps_per_row; ++k) t += red[i][w0 + k];
    v[i] = t;
  }
}

// RES: 0 none, 1 bf16, 2 fp32.  OUT: 0 bf16, 1 fp32, 2 e4m3 with scales.
template <bool XF32, int RES, int OUT, int NV>
__global__ void __launch_bounds__(512) k_rmsnorm(const NormArgs a) {
  __shared__ float red[1][16];
  const int tid = threadIdx.x & (a.tpr - 1);
  const long long t = (long long)blockIdx.x * (blockDim.x / a.tpr) + threadIdx.x / a.tpr;
  const int dv = a.d / 8;
  griddep_wait();
  const bool row = t < a.T;
  Raw8<XF32> rx[NV];
  Raw8<RES == 2> rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * a.tpr;
    rx[i].zero();
    rr[i].zero();
    if (row && v < dv) {
      rx[i].load(a.x, (size_t)t * dv + v);
      if (RES) rr[i].load(a.res, (size_t)t * dv + v);
    }
  }
  float s[NV][8], sum[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    rx[i].get(s[i]);
    if (RES) {
      float r[8];
      rr[i].get(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[i][j] += r[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0] += s[i][j] * s[i][j];
  }
  row_sum<1>(sum, red, a.tpr >> 5);
  const float rstd = rsqrtf(sum[0] / (float)a.d + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * a.tpr;
    const bool in = row && v < dv;
    const size_t at = (size_t)t * dv + v;
    float w[8], y[8];
    if (in) load_w8(a.w, a.w_f32, v, w);
    if (in && RES == 1) store8_bf16(a.s, at, s[i]);
    if (in && RES == 2) store8_f32(a.s, at, s[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = in ? s[i][j] * rstd * w[j] : 0.0f;
    if (OUT == 0 && in) store8_bf16(a.y, at, y);
    if (OUT == 1 && in) store8_f32(a.y, at, y);
    if (OUT == 2) {
      const float m = group_amax(amax8(y));
      if (in) {
        reinterpret_cast<uint2*>(a.y)[at] = codes8(y, Q_MAX / m);
        if ((v & 15) == 0) a.scale[(size_t)t * ((a.d + Q_GROUP - 1) / Q_GROUP) + v / 16] = m / Q_MAX;
      }
    }
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* s;
  const void* ds;      // or null
  const void* w;
  void* dx;            // in s's type
  float* part;         // [gridDim.x · groups per CTA][d] partial sums of dw
  int T, d, tpr, w_f32;
  float eps;
};

// One group of threads takes rows g, g + groups, ... and keeps its part of dw
// in registers over them.
template <bool SF32, bool DYF32, bool DS, int NV>
__global__ void __launch_bounds__(512) k_rmsnorm_bwd(const NormBwdArgs a) {
  __shared__ float red[2][2][16];
  const int tid = threadIdx.x & (a.tpr - 1);
  const int dv = a.d / 8;
  const int rpc = blockDim.x / a.tpr;
  const long long g = (long long)blockIdx.x * rpc + threadIdx.x / a.tpr;
  griddep_wait();
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * a.tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = 0.0f;
    if (v < dv) load_w8(a.w, a.w_f32, v, w[i]);
  }
  int par = 0;
  for (long long t0 = (long long)blockIdx.x * rpc; t0 < a.T; t0 += (long long)gridDim.x * rpc, par ^= 1) {
    const long long t = t0 + threadIdx.x / a.tpr;
    const bool row = t < a.T;
    Raw8<SF32> rs[NV], rd[NV];
    Raw8<DYF32> ry[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * a.tpr;
      rs[i].zero();
      ry[i].zero();
      rd[i].zero();
      if (row && v < dv) {
        rs[i].load(a.s, (size_t)t * dv + v);
        ry[i].load(a.dy, (size_t)t * dv + v);
        if (DS) rd[i].load(a.ds, (size_t)t * dv + v);
      }
    }
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s[8], y[8];
      rs[i].get(s);
      ry[i].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum[0] += s[j] * s[j];
        sum[1] += s[j] * (y[j] * w[i][j]);
      }
    }
    row_sum<2>(sum, red[par], a.tpr >> 5);
    const float rstd = rsqrtf(sum[0] / (float)a.d + a.eps);
    const float c = sum[1] * rstd * rstd * rstd / (float)a.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * a.tpr;
      float s[8], y[8], dx[8];
      rs[i].get(s);
      ry[i].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dx[j] = rstd * (y[j] * w[i][j]) - s[j] * c;
        if (row) dw[i][j] += y[j] * (s[j] * rstd);
      }
      if (DS) {
        rd[i].get(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] += s[j];
      }
      if (row && v < dv) {
        if (SF32) store8_f32(a.dx, (size_t)t * dv + v, dx);
        else store8_bf16(a.dx, (size_t)t * dv + v, dx);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * a.tpr;
    if (v < dv) store8_f32(a.part, (size_t)g * dv + v, dw[i]);
  }
}

// dw[c] = sum over the n_part partial rows, eight warps taking every eighth
// row and added in order.  One CTA per 32 columns.
__global__ void __launch_bounds__(256) k_rmsnorm_dw(const float* part, int n_part, int d, float* dw) {
  __shared__ float red[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  griddep_wait();
  float t = 0.0f;
  if (c < d)
    for (int p = k; p < n_part; p += 8) t += part[(size_t)p * d + c];
  red[k][threadIdx.x & 31] = t;
  __syncthreads();
  if (k == 0 && c < d) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) u += red[i][threadIdx.x];
    dw[c] = u;
  }
}

}  // namespace sffn
