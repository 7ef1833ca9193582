// Linear layer with both operands in e4m3: per 128-wide block b of the inner
// dimension,
//
//   y[t][n] = sum_b xs[t][b] · Ws[n/128][b] · sum_{k in b} xq[t][k] · Wq[n][k]
//
// The products inside a block are exact in fp32 terms; blocks are scaled and
// added in fp32.
#pragma once

#include "vec8.cuh"

namespace sffn {

struct QlinArgs {
  const uint8_t* xq;    // [T][k]
  const float* xs;      // [T][kb]
  const uint8_t* Wq;    // [n][k]
  const float* Ws;      // [ceil(n/128)][kb]
  void* y;              // [T][n], bf16 or fp32
  int T, n, k, kb;
  int y_f32;
  uint32_t* status;
};

__global__ void __launch_bounds__(256) k_qlinear(const QlinArgs a) {
  const int n = blockIdx.x * 32 + (threadIdx.x & 31), t = blockIdx.y * 8 + (threadIdx.x >> 5);
  griddep_wait();
  if (n >= a.n || t >= a.T) return;
  float acc = 0.0f;
  for (int b = 0; b < a.kb; ++b) {
    float p = 0.0f;
    for (int k = b * Q_GROUP; k < min(a.k, (b + 1) * Q_GROUP); ++k) {
      __nv_fp8_e4m3 u, v;
      u.__x = a.xq[(size_t)t * a.k + k];
      v.__x = a.Wq[(size_t)n * a.k + k];
      p += (float)u * (float)v;
    }
    acc += p * (a.xs[(size_t)t * a.kb + b] * a.Ws[(size_t)(n / Q_GROUP) * a.kb + b]);
  }
  if (a.y_f32) reinterpret_cast<float*>(a.y)[(size_t)t * a.n + n] = acc;
  else reinterpret_cast<__nv_bfloat16*>(a.y)[(size_t)t * a.n + n] = __float2bfloat16(acc);
}

}  // namespace sffn
