// e4m3 codes with fp32 scales: rows (one scale for each 128 columns of a row)
// and weight blocks (one for each 128 x 128).  scale = amax / 448, code =
// e4m3(v · 448/amax) rounded to nearest, amax at least Q_TINY.  Bound by
// memory; a group's values stay in registers between its amax and its codes.  13
// rows of 14336 take 2.3 us, nearly all of it a launch's latency, beside which the
// linear kernel that follows sets itself up.
#pragma once

#include "vec8.cuh"

namespace sffn {

// 16 threads per group of 128 columns.
template <bool F32>
__global__ void __launch_bounds__(256) k_quant_rows(const void* x, int T, int d, uint8_t* q, float* scale) {
  const int gpr = (d + Q_GROUP - 1) / Q_GROUP, dv = d / 8;
  const long long n = (long long)T * gpr;
  const int l = threadIdx.x & 15;
  griddep_wait();
  griddep_launch();   // the next kernel may set itself up meanwhile
  for (long long g0 = (long long)blockIdx.x * 16; g0 < n; g0 += (long long)gridDim.x * 16) {
    const long long g = g0 + (threadIdx.x >> 4);
    const long long t = g / gpr;
    const int v = (int)(g - t * gpr) * 16 + l;
    const bool in = g < n && v < dv;
    Raw8<F32> r;
    r.zero();
    if (in) r.load(x, (size_t)t * dv + v);
    float f[8];
    r.get(f);
    const float m = group_amax(amax8(f));
    if (in) {
      reinterpret_cast<uint2*>(q)[(size_t)t * dv + v] = codes8(f, Q_MAX / m);
      if (l == 0) scale[g] = m / Q_MAX;
    }
  }
}

// One CTA per 128 x 128 block of W [n][k]: 16 threads per row, 8 rows each.
template <bool F32>
__global__ void __launch_bounds__(256) k_quant_blocks(const void* W, int n, int k, uint8_t* q, float* scale) {
  __shared__ float red[8];
  const int kv = k / 8, v = blockIdx.x * 16 + (threadIdx.x & 15);
  griddep_wait();
  Raw8<F32> r[8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = blockIdx.y * Q_GROUP + i * 16 + (threadIdx.x >> 4);
    r[i].zero();
    if (row < n && v < kv) r[i].load(W, (size_t)row * kv + v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    r[i].get(f);
    m = fmaxf(m, amax8(f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = Q_TINY;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = blockIdx.y * Q_GROUP + i * 16 + (threadIdx.x >> 4);
    if (row < n && v < kv) {
      float f[8];
      r[i].get(f);
      reinterpret_cast<uint2*>(q)[(size_t)row * kv + v] = codes8(f, Q_MAX / m);
    }
  }
  if (threadIdx.x == 0) scale[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = m / Q_MAX;
}

}  // namespace sffn
