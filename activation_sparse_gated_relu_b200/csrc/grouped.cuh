// Products grouped by expert with ragged groups: expert e owns the rows
// off[e] .. off[e+1] of x.  With W [E][n][k],
//
//   forward   y[r]  = W[e] x[r]
//   input     dx[r] = W[e]^T dy[r]
//   weight    dW[e] = sum_{r in e} dy[r] x[r]^T
//
// bf16 operands, fp32 sums.
#pragma once

#include "vec8.cuh"

namespace sffn {

// Group e's rows [a, b), clamped to [0, R]; false if the offsets are out of
// range or run backwards (the group is then what the clamping leaves).
__device__ __forceinline__ bool group_rows(const int* off, int e, int R, int* a, int* b) {
  const int u = off[e], v = off[e + 1];
  *a = min(max(u, 0), R);
  *b = max(min(max(v, 0), R), *a);
  return u >= 0 && v >= u && v <= R;
}

struct GroupedArgs {
  const __nv_bfloat16* a;   // x or dy
  const __nv_bfloat16* b;   // W, or (weight gradient) x
  const int* off;           // [E + 1]
  void* out;
  int E, R, k, n, out_f32;
  uint32_t* status;
};

__device__ __forceinline__ void put(void* out, int f32, size_t at, float v) {
  if (f32) reinterpret_cast<float*>(out)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16(v);
}

// MODE 0: y; 1: dx.  One CTA row per expert (blockIdx.y), grid-stride over its rows.
template <int MODE>
__global__ void __launch_bounds__(256) k_grouped_rows(const GroupedArgs a) {
  griddep_wait();
  const int e = blockIdx.y;
  int r0, r1;
  if (!group_rows(a.off, e, a.R, &r0, &r1) && threadIdx.x == 0) atomicOr(a.status, DEV_ERR_RANGE);
  const int cols = MODE == 0 ? a.n : a.k, inner = MODE == 0 ? a.k : a.n;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  if (c >= cols) return;
  const __nv_bfloat16* W = a.b + (size_t)e * a.n * a.k;
  for (int r = r0 + (threadIdx.x >> 5); r < r1; r += 8) {
    float acc = 0.0f;
    for (int i = 0; i < inner; ++i)
      acc += __bfloat162float(a.a[(size_t)r * inner + i]) *
             __bfloat162float(MODE == 0 ? W[(size_t)c * a.k + i] : W[(size_t)i * a.k + c]);
    put(a.out, a.out_f32, (size_t)r * cols + c, acc);
  }
}

__global__ void __launch_bounds__(256) k_grouped_weight(const GroupedArgs a) {
  griddep_wait();
  const int e = blockIdx.z;
  int r0, r1;
  if (!group_rows(a.off, e, a.R, &r0, &r1) && threadIdx.x == 0) atomicOr(a.status, DEV_ERR_RANGE);
  const int i = blockIdx.x * 32 + (threadIdx.x & 31), o = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (i >= a.k || o >= a.n) return;
  float acc = 0.0f;
  for (int r = r0; r < r1; ++r)
    acc += __bfloat162float(a.a[(size_t)r * a.n + o]) * __bfloat162float(a.b[(size_t)r * a.k + i]);
  put(a.out, a.out_f32, ((size_t)e * a.n + o) * a.k + i, acc);
}

}  // namespace sffn
