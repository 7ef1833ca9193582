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
// The sum of squares is an fp32 sum: |s| has to stay below about 1e19 / sqrt(d).
//
// Both are bound by memory: each value is read once and each result written
// once.  A row is held by a group of threads, eight columns each, once, twice or
// four times: up to 1024 columns 32, 64 or 128 threads, several groups a CTA of
// 256; above that a CTA of as many warps as the row needs, so that neither the
// second use of s nor the 8-bit scale reads global memory again.  Forward, 4096
// rows of 2048, fp32 x, bf16 residual, sum and y (84 MB): 12.7 us, 6.6 TB/s; 6213
// rows of 5400 51 us, 6.5 TB/s (62 with groups of a power of two).  To e4m3, all
// bf16 before, 8192 rows of 4096 (236 MB) 50 us, 4.7 TB/s: a row is one chain of
// load, sum, scale and store, and the codes leave 8 bytes a thread.  Gradient, 8191
// rows of 4096, all bf16 (268 MB): 49.5 us, 5.4 TB/s, and 3.7 for dw's partial
// sums.  Sums are fp32, in a fixed order.
#pragma once

#include <type_traits>

#include "ptx_pair.cuh"
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
  int T, d, w_f32;
  int tpr, shift, rpc; // threads per row; thread index >> shift: row within the CTA; rows per CTA
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

// Sums of v[0..N) over the row's threads (the same in all of them): warp sums to
// shared memory, then every warp adds its row's, from warp `first` on, in pairs.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*red)[16], int first, int warps_per_row) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (warps_per_row == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][warp] = v[i];
  __syncthreads();
  const int n = 1 << (32 - __clz(warps_per_row - 1)), w = lane & (n - 1);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w < warps_per_row ? red[i][first + w] : 0.0f;
  for (int o = n >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

// RES: 0 none, 1 bf16, 2 fp32.  OUT: 0 bf16, 1 fp32, 2 e4m3 with scales.
template <bool XF32, int RES, int OUT, int NV>
__global__ void __launch_bounds__(512) k_rmsnorm(const NormArgs a) {
  __shared__ float red[1][16];
  const int sub = threadIdx.x >> a.shift, tid = threadIdx.x & ((1 << a.shift) - 1);
  const long long t = (long long)blockIdx.x * a.rpc + sub;
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
  row_sum<1>(sum, red, sub * (a.tpr >> 5), a.tpr >> 5);
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
  float* part;         // [gridDim.x][d] partial sums of dw
  int T, d, w_f32;
  int tpr, shift, rpc; // threads per row, as above, rows per CTA
  float eps;
};

// A row is a chain (load, two sums over its threads, gradient), so several
// rows' values are on their way while one is worked on: every thread copies
// its own columns of the rows to come into shared memory, STAGES - 1 rows
// ahead, and reads them back itself, without any barrier, and again for their
// second use.  That leaves 64 registers a thread enough up to 8192 columns, for
// two CTAs of 512 threads an SM (four of 256).  Where the rows are too wide (d >
// 8192 in fp32), STAGES is 0 and they are loaded as they are needed.  With four
// stages, what is left is bound by instruction issue, so the arithmetic runs on
// pairs of columns.  Measured at 8191 x 4096: rows loaded as they are needed, one
// column at a time 70.5 us, so 49.5; at 4382 x 7656 the values in registers, one
// CTA, 82, so 63.  With two stages (fp32 rows, or more than eight columns a thread)
// only one row is on its way, and that bounds it: 8192 x 4096 fp32 110 us, 4.3 TB/s,
// 6213 x 5400 bf16 65 us, 4.1 TB/s.
template <bool SF32, bool DYF32, bool DS, int NV>
struct NormBwdCfg {
  static constexpr int NS = SF32 ? 2 : 1, NY = DYF32 ? 2 : 1, ND = DS ? NS : 0;
  static constexpr int PER = (NS + NY + ND) * NV;              // 16-byte pieces per thread and row
  static constexpr int STAGES = PER <= 3 ? 4 : PER <= 12 ? 2 : 0;
  static constexpr int smem(int threads) { return STAGES * PER * 16 * threads; }
};

// One group of threads takes rows g, g + groups, ... and keeps its part of dw
// in registers over them.
template <bool SF32, bool DYF32, bool DS, int NV>
__global__ void __launch_bounds__(512, NV <= 2 ? 2 : 1) k_rmsnorm_bwd(const NormBwdArgs a) {
  using Cfg = NormBwdCfg<SF32, DYF32, DS, NV>;
  constexpr int STAGES = Cfg::STAGES, NS = Cfg::NS, NY = Cfg::NY, ND = Cfg::ND;
  __shared__ float red[2][2][16];
  extern __shared__ uint4 ring[];      // [STAGES][PER][threads]
  const int sub = threadIdx.x >> a.shift, tid = threadIdx.x & ((1 << a.shift) - 1);
  const int dv = a.d / 8, rpc = a.rpc;
  const long long g = (long long)blockIdx.x * rpc + sub;
  const long long step = (long long)gridDim.x * rpc;
  griddep_wait();
  uint64_t dw[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = 0;
  // with eight columns per thread the weight stays in registers
  uint64_t w1[4];
  auto weight = [&](int i, uint64_t (&f)[4]) {
    const int v = tid + i * a.tpr;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (v < dv) load_w8(a.w, a.w_f32, v, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pack2(x[2 * j], x[2 * j + 1]);
  };
  if (NV == 1) weight(0, w1);
  // this thread's pieces of the next row to ask for, row t, into ring slot
  // `slot` (zeros past the end)
  long long at_ask = g * dv + tid;
  auto ask = [&](long long t, int slot) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = t < a.T && tid + i * a.tpr < dv;
      const long long at = in ? at_ask + i * a.tpr : 0;
      uint4* to = ring + ((size_t)slot * Cfg::PER + i * (NS + NY + ND)) * blockDim.x + threadIdx.x;
#pragma unroll
      for (int k = 0; k < NS; ++k) copy16_async(to + k * blockDim.x, reinterpret_cast<const uint4*>(a.s) + at * NS + k, in);
#pragma unroll
      for (int k = 0; k < NY; ++k)
        copy16_async(to + (NS + k) * blockDim.x, reinterpret_cast<const uint4*>(a.dy) + at * NY + k, in);
#pragma unroll
      for (int k = 0; k < ND; ++k)
        copy16_async(to + (NS + NY + k) * blockDim.x, reinterpret_cast<const uint4*>(a.ds) + at * NS + k, in);
    }
    at_ask += step * dv;
    copies_commit();
  };
#pragma unroll
  for (int q = 0; q < (STAGES > 0 ? STAGES - 1 : 0); ++q) ask(g + q * step, q);
  int par = 0, slot = 0;
  long long at_row = g * dv + tid;
  for (long long t0 = (long long)blockIdx.x * rpc; t0 < a.T; t0 += step, par ^= 1, at_row += step * dv) {
    const long long t = t0 + sub;
    const bool row = t < a.T;
    if (STAGES > 0) {
      ask(t + (STAGES - 1) * step, (slot + STAGES - 1) & (STAGES > 0 ? STAGES - 1 : 0));
      copies_wait<(STAGES > 0 ? STAGES - 1 : 0)>();
    }
    // this thread's i-th eight values of s, dy or ds: read from the ring as often
    // as they are used, which leaves registers to a second CTA
    auto get = [&](const void* base, auto f32, int i, int first, uint64_t (&f)[4]) {
      Raw8<decltype(f32)::value> r;
      r.zero();
      if (STAGES > 0) {
        const uint4* from = ring + ((size_t)slot * Cfg::PER + i * (NS + NY + ND) + first) * blockDim.x + threadIdx.x;
#pragma unroll
        for (int k = 0; k < (decltype(f32)::value ? 2 : 1); ++k) r.v[k] = from[k * blockDim.x];
      } else if (row && tid + i * a.tpr < dv) {
        r.load(base, at_row + i * a.tpr);
      }
      r.pairs(f);
    };
    const std::integral_constant<bool, SF32> sf;
    const std::integral_constant<bool, DYF32> yf;
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t s[4], y[4], w[4];
      get(a.s, sf, i, 0, s);
      get(a.dy, yf, i, NS, y);
      if (NV > 1) weight(i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s0 = fma2(s[j], s[j], s0);
        s1 = fma2(s[j], mul2(y[j], NV == 1 ? w1[j] : w[j]), s1);
      }
    }
    float sum[2], hi;
    unpack2(s0, sum[0], hi);
    sum[0] += hi;
    unpack2(s1, sum[1], hi);
    sum[1] += hi;
    row_sum<2>(sum, red[par], sub * (a.tpr >> 5), a.tpr >> 5);
    // rows past the end (with several rows a CTA) take any eps but 0, with which
    // their zeros would give an infinity, and NaN in dw
    const float rstd = rsqrtf(sum[0] / (float)a.d + (NV > 1 || row ? a.eps : 1.0f));
    const float c = sum[1] * rstd * rstd * rstd / (float)a.d;
    const uint64_t r2 = pack2(rstd, rstd), c2 = pack2(-c, -c);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t s[4], y[4], w[4], dx[4];
      get(a.s, sf, i, 0, s);
      get(a.dy, yf, i, NS, y);
      if (NV > 1) weight(i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dx[j] = fma2(s[j], c2, mul2(mul2(y[j], NV == 1 ? w1[j] : w[j]), r2));
        dw[i][j] = fma2(y[j], mul2(s[j], r2), dw[i][j]);   // rows past the end add zeros
      }
      if (DS) {
        get(a.ds, sf, i, NS + NY, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) dx[j] = add2(dx[j], s[j]);
      }
      if (row && tid + i * a.tpr < dv) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) unpack2(dx[j], f[2 * j], f[2 * j + 1]);
        if (SF32) store8_f32(a.dx, at_row + i * a.tpr, f);
        else store8_bf16(a.dx, at_row + i * a.tpr, f);
      }
    }
    if (STAGES > 0) slot = (slot + 1) & (STAGES - 1);
  }
  if (STAGES > 0) copies_wait<0>();
  if (rpc > 1) {   // the CTA's groups, eight columns a thread, join in the ring's memory
    static_assert(NV > 1 || STAGES * Cfg::PER * 16 >= 32, "a thread's eight sums");
    float f[8], u[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(dw[0][j], f[2 * j], f[2 * j + 1]);
    __syncthreads();
    store8_f32(ring, threadIdx.x, f);
    __syncthreads();
    if (sub > 0 || tid >= dv) return;
    for (int k = 1; k < rpc; ++k) {
      Raw8<true> r;
      r.load(ring, threadIdx.x + k * a.tpr);
      r.get(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += u[j];
    }
    store8_f32(a.part, (size_t)blockIdx.x * dv + tid, f);
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * a.tpr;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(dw[i][j], f[2 * j], f[2 * j + 1]);
    if (v < dv) store8_f32(a.part, (size_t)blockIdx.x * dv + v, f);
  }
}

// dw[c] = sum over the n_part partial rows, sixteen warps taking every
// sixteenth row and added in order.  One CTA per 32 columns.
__global__ void __launch_bounds__(512) k_rmsnorm_dw(const float* part, int n_part, int d, float* dw) {
  __shared__ float red[16][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  griddep_wait();
  float t = 0.0f;
  if (c < d) {
    int p = k;
    for (; p + 112 < n_part; p += 128) {   // eight loads in flight, added in order
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(size_t)(p + 16 * i) * d + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) t += v[i];
    }
    for (; p < n_part; p += 16) t += part[(size_t)p * d + c];
  }
  red[k][threadIdx.x & 31] = t;
  __syncthreads();
  if (k == 0 && c < d) {
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) u += red[i][threadIdx.x];
    dw[c] = u;
  }
}

}  // namespace sffn
