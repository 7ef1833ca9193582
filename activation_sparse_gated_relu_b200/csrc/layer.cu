// C ABI of the operators around the sparse FFN (see include/sffn.h): RMS norm
// with the residual's addition, the 8-bit linear layer with its quantisers,
// and the experts' grouped products.  Argument validation and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/sffn.h"
#include "grouped.cuh"
#include "host_util.cuh"
#include "norm.cuh"
#include "qlinear.cuh"
#include "quant.cuh"

using namespace sffn;

namespace {

constexpr int kMaxRows = 1 << 24;

sffn_status launched(cudaError_t e) { return e == cudaSuccess ? SFFN_OK : SFFN_ERR_CUDA; }

// The device of a new handle: sm_100, and its number of SMs.
sffn_status pick_device(int* dev, int* n_sm) {
  int major = 0;
  if (cudaGetDevice(dev) != cudaSuccess) {
    cudaGetLastError();
    return SFFN_ERR_NO_DEVICE;
  }
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev);
  cudaDeviceGetAttribute(n_sm, cudaDevAttrMultiProcessorCount, *dev);
  if (major != 10 || *n_sm <= 0) return SFFN_ERR_NO_DEVICE;
  return SFFN_OK;
}

// A handle's calls run on the device it was created on.
bool on_device(int dev) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) cudaGetLastError();
  return cur == dev;
}

sffn_status read_status_word(uint32_t* word, cudaStream_t st) {
  uint32_t v = 0;
  if (cudaStreamSynchronize(st) != cudaSuccess || cudaMemcpy(&v, word, 4, cudaMemcpyDeviceToHost) != cudaSuccess ||
      (v && cudaMemset(word, 0, 4) != cudaSuccess)) {
    cudaGetLastError();
    return SFFN_ERR_CUDA;
  }
  return (v & DEV_ERR_TIMEOUT) ? SFFN_ERR_TIMEOUT : (v & DEV_ERR_RANGE) ? SFFN_ERR_DEVICE : SFFN_OK;
}

// Device memory of a handle is freed on its own device, after its last call.
void free_on(int dev, void* p) {
  int cur = -1;
  cudaGetDevice(&cur);
  if (cur != dev) cudaSetDevice(dev);
  cudaDeviceSynchronize();
  if (p) cudaFree(p);
  if (cur >= 0 && cur != dev) cudaSetDevice(cur);
  cudaGetLastError();
}

bool is_value_type(int t) { return t == SFFN_BF16 || t == SFFN_FP32; }

}  // namespace

// ---------------------------------------------------------------------------
// RMS norm
namespace {

struct NormShape {
  int tpr, nv, threads, rpc;   // threads per row, vectors per thread, threads and rows per CTA
};

NormShape norm_shape(int d) {
  NormShape s;
  const int dv = d / 8;
  s.tpr = 32;
  while (s.tpr < dv && s.tpr < 512) s.tpr *= 2;
  s.nv = cdiv(dv, s.tpr);
  s.nv = s.nv > 2 ? 4 : s.nv;
  s.threads = std::max(s.tpr, 256);
  s.rpc = s.threads / s.tpr;
  return s;
}

constexpr int kNormBwdCtas = 296;
int norm_bwd_ctas(const NormShape& s, int T) { return std::min(cdiv(T, s.rpc), kNormBwdCtas); }

sffn_status norm_validate(const sffn_rmsnorm_desc* d) {
  if (!d || !d->weight || !aligned16(d->weight)) return SFFN_ERR_INVALID_ARG;
  if (d->d <= 0 || !(d->eps >= 0.0f) || std::isinf(d->eps)) return SFFN_ERR_INVALID_ARG;
  if (!is_value_type(d->weight_dtype) || !is_value_type(d->x_dtype) || !is_value_type(d->residual_dtype) ||
      (!is_value_type(d->y_dtype) && d->y_dtype != SFFN_E4M3))
    return SFFN_ERR_INVALID_ARG;
  if (d->d % 8 || d->d > NORM_MAX_D) return SFFN_ERR_UNSUPPORTED;
  return SFFN_OK;
}

template <bool XF32, int RES, int OUT>
cudaError_t norm_launch(const NormArgs& a, const NormShape& s, cudaStream_t st) {
  const dim3 grid(cdiv(a.T, s.rpc)), block(s.threads);
  switch (s.nv) {
    case 1: return launch_pdl(k_rmsnorm<XF32, RES, OUT, 1>, grid, block, 0, st, 1, a);
    case 2: return launch_pdl(k_rmsnorm<XF32, RES, OUT, 2>, grid, block, 0, st, 1, a);
    default: return launch_pdl(k_rmsnorm<XF32, RES, OUT, 4>, grid, block, 0, st, 1, a);
  }
}
template <bool XF32, int RES>
cudaError_t norm_launch_out(int out, const NormArgs& a, const NormShape& s, cudaStream_t st) {
  return out == SFFN_BF16   ? norm_launch<XF32, RES, 0>(a, s, st)
         : out == SFFN_FP32 ? norm_launch<XF32, RES, 1>(a, s, st)
                            : norm_launch<XF32, RES, 2>(a, s, st);
}
template <bool XF32>
cudaError_t norm_launch_res(int res, int out, const NormArgs& a, const NormShape& s, cudaStream_t st) {
  return res == 0   ? norm_launch_out<XF32, 0>(out, a, s, st)
         : res == 1 ? norm_launch_out<XF32, 1>(out, a, s, st)
                    : norm_launch_out<XF32, 2>(out, a, s, st);
}

template <bool SF32, bool DYF32, bool DS>
cudaError_t norm_bwd_launch(const NormBwdArgs& a, const NormShape& s, int ctas, cudaStream_t st) {
  const dim3 grid(ctas), block(s.threads);
  switch (s.nv) {
    case 1: return launch_pdl(k_rmsnorm_bwd<SF32, DYF32, DS, 1>, grid, block, 0, st, 1, a);
    case 2: return launch_pdl(k_rmsnorm_bwd<SF32, DYF32, DS, 2>, grid, block, 0, st, 1, a);
    default: return launch_pdl(k_rmsnorm_bwd<SF32, DYF32, DS, 4>, grid, block, 0, st, 1, a);
  }
}
template <bool SF32, bool DYF32>
cudaError_t norm_bwd_launch_ds(const NormBwdArgs& a, const NormShape& s, int ctas, cudaStream_t st) {
  return a.ds ? norm_bwd_launch<SF32, DYF32, true>(a, s, ctas, st) : norm_bwd_launch<SF32, DYF32, false>(a, s, ctas, st);
}

}  // namespace

extern "C" sffn_status sffn_rmsnorm_forward(const sffn_rmsnorm_desc* desc, const void* x, const void* residual, int T,
                                            void* residual_out, void* y, float* scale, void* cuda_stream) {
  const sffn_status vs = norm_validate(desc);
  if (vs != SFFN_OK) return vs;
  if (T < 0 || T > kMaxRows) return SFFN_ERR_INVALID_ARG;
  if (T == 0) return SFFN_OK;
  if (!x || !y || !aligned16(x) || !aligned16(y) || !aligned16(residual) || !aligned16(residual_out))
    return SFFN_ERR_INVALID_ARG;
  if ((residual == nullptr) != (residual_out == nullptr)) return SFFN_ERR_INVALID_ARG;
  if ((desc->y_dtype == SFFN_E4M3) != (scale != nullptr)) return SFFN_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.res = residual;
  a.w = desc->weight;
  a.s = residual_out;
  a.y = y;
  a.scale = scale;
  a.T = T;
  a.d = desc->d;
  a.w_f32 = desc->weight_dtype == SFFN_FP32;
  a.eps = desc->eps;
  const NormShape s = norm_shape(desc->d);
  a.tpr = s.tpr;
  const int res = !residual ? 0 : desc->residual_dtype == SFFN_FP32 ? 2 : 1;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return launched(desc->x_dtype == SFFN_FP32 ? norm_launch_res<true>(res, desc->y_dtype, a, s, st)
                                             : norm_launch_res<false>(res, desc->y_dtype, a, s, st));
}

extern "C" sffn_status sffn_rmsnorm_workspace_bytes(int d, int T, size_t* bytes) {
  if (!bytes || d <= 0 || T < 0 || T > kMaxRows) return SFFN_ERR_INVALID_ARG;
  if (d % 8 || d > NORM_MAX_D) return SFFN_ERR_UNSUPPORTED;
  const NormShape s = norm_shape(d);
  *bytes = (size_t)norm_bwd_ctas(s, T) * s.rpc * d * sizeof(float);
  return SFFN_OK;
}

extern "C" sffn_status sffn_rmsnorm_backward(const sffn_rmsnorm_desc* desc, const void* dy, const void* s_in,
                                             const void* ds, int T, void* dx, float* dweight, void* workspace,
                                             size_t workspace_bytes, void* cuda_stream) {
  const sffn_status vs = norm_validate(desc);
  if (vs != SFFN_OK) return vs;
  if (T < 0 || T > kMaxRows || !is_value_type(desc->y_dtype)) return SFFN_ERR_INVALID_ARG;
  if (!dweight || !aligned16(dweight)) return SFFN_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !s_in || !dx || !aligned16(dy) || !aligned16(s_in) || !aligned16(ds) || !aligned16(dx)))
    return SFFN_ERR_INVALID_ARG;
  size_t need = 0;
  sffn_rmsnorm_workspace_bytes(desc->d, T, &need);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SFFN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const NormShape s = norm_shape(desc->d);
  const int ctas = norm_bwd_ctas(s, T);
  NormBwdArgs a{};
  a.dy = dy;
  a.s = s_in;
  a.ds = ds;
  a.w = desc->weight;
  a.dx = dx;
  a.part = static_cast<float*>(workspace);
  a.T = T;
  a.d = desc->d;
  a.tpr = s.tpr;
  a.w_f32 = desc->weight_dtype == SFFN_FP32;
  a.eps = desc->eps;
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    const bool sf = desc->residual_dtype == SFFN_FP32, yf = desc->y_dtype == SFFN_FP32;
    e = sf ? (yf ? norm_bwd_launch_ds<true, true>(a, s, ctas, st) : norm_bwd_launch_ds<true, false>(a, s, ctas, st))
           : (yf ? norm_bwd_launch_ds<false, true>(a, s, ctas, st) : norm_bwd_launch_ds<false, false>(a, s, ctas, st));
  }
  e = e ? e
        : launch_pdl(k_rmsnorm_dw, dim3(cdiv(desc->d, 32)), dim3(256), 0, st, 1, (const float*)workspace, ctas * s.rpc,
                     desc->d, dweight);
  return launched(e);
}

// ---------------------------------------------------------------------------
// 8-bit codes with scales
extern "C" sffn_status sffn_quantize_rows(const void* x, sffn_dtype x_dtype, int T, int d, void* codes, float* scale,
                                          void* cuda_stream) {
  if (T < 0 || T > kMaxRows || d <= 0 || !is_value_type(x_dtype)) return SFFN_ERR_INVALID_ARG;
  if (d % 8) return SFFN_ERR_UNSUPPORTED;
  if (T == 0) return SFFN_OK;
  if (!x || !codes || !scale || !aligned16(x) || !aligned16(codes) || !aligned16(scale)) return SFFN_ERR_INVALID_ARG;
  const long long groups = (long long)T * cdiv(d, Q_GROUP);
  const dim3 grid((unsigned)std::min<long long>((groups + 15) / 16, 1 << 16)), block(256);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint8_t* q = static_cast<uint8_t*>(codes);
  return launched(x_dtype == SFFN_FP32 ? launch_pdl(k_quant_rows<true>, grid, block, 0, st, 1, x, T, d, q, scale)
                                       : launch_pdl(k_quant_rows<false>, grid, block, 0, st, 1, x, T, d, q, scale));
}

extern "C" sffn_status sffn_quantize_blocks(const void* W, sffn_dtype w_dtype, int n, int k, void* codes, float* scale,
                                            void* cuda_stream) {
  if (n <= 0 || k <= 0 || !is_value_type(w_dtype)) return SFFN_ERR_INVALID_ARG;
  if (k % 8 || cdiv(n, Q_GROUP) > 65535) return SFFN_ERR_UNSUPPORTED;
  if (!W || !codes || !scale || !aligned16(W) || !aligned16(codes) || !aligned16(scale)) return SFFN_ERR_INVALID_ARG;
  const dim3 grid(cdiv(k, Q_GROUP), cdiv(n, Q_GROUP)), block(256);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint8_t* q = static_cast<uint8_t*>(codes);
  return launched(w_dtype == SFFN_FP32 ? launch_pdl(k_quant_blocks<true>, grid, block, 0, st, 1, W, n, k, q, scale)
                                       : launch_pdl(k_quant_blocks<false>, grid, block, 0, st, 1, W, n, k, q, scale));
}

// ---------------------------------------------------------------------------
// 8-bit linear layer
struct sffn_qlinear_handle {
  sffn_qlinear_desc desc;
  int dev = 0, n_sm = 0;
  uint32_t* status = nullptr;   // [4]
};

extern "C" sffn_status sffn_qlinear_create(const sffn_qlinear_desc* desc, void* cuda_stream, sffn_qlinear_handle** out) {
  if (!out) return SFFN_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || !desc->Wq || !desc->Ws || !aligned16(desc->Wq) || !aligned16(desc->Ws)) return SFFN_ERR_INVALID_ARG;
  if (desc->d_in <= 0 || desc->d_out <= 0) return SFFN_ERR_INVALID_ARG;
  if (desc->d_in % 16 || desc->d_out % 8 || desc->d_in > (1 << 20) || desc->d_out > (1 << 20)) return SFFN_ERR_UNSUPPORTED;
  int dev = 0, n_sm = 0;
  const sffn_status ds = pick_device(&dev, &n_sm);
  if (ds != SFFN_OK) return ds;
  sffn_qlinear_handle* h = new (std::nothrow) sffn_qlinear_handle();
  if (!h) return SFFN_ERR_ALLOC;
  h->desc = *desc;
  h->dev = dev;
  h->n_sm = n_sm;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (!dalloc(&h->status, 16)) {
    delete h;
    return SFFN_ERR_ALLOC;
  }
  cudaError_t e = cudaMemsetAsync(h->status, 0, 16, st);
  e = e ? e : cudaStreamSynchronize(st);
  if (e) {
    free_on(dev, h->status);
    delete h;
    return SFFN_ERR_CUDA;
  }
  *out = h;
  return SFFN_OK;
}

extern "C" sffn_status sffn_qlinear_forward(sffn_qlinear_handle* h, const void* xq, const float* xs, int T, void* y,
                                            sffn_dtype y_dtype, void* cuda_stream) {
  if (!h || T < 0 || T > kMaxRows || !is_value_type(y_dtype)) return SFFN_ERR_INVALID_ARG;
  if (T == 0) return SFFN_OK;
  if (!xq || !xs || !y || !aligned16(xq) || !aligned16(xs) || !aligned16(y)) return SFFN_ERR_INVALID_ARG;
  if (!on_device(h->dev)) return SFFN_ERR_INVALID_ARG;
  QlinArgs a{};
  a.xq = static_cast<const uint8_t*>(xq);
  a.xs = xs;
  a.Wq = static_cast<const uint8_t*>(h->desc.Wq);
  a.Ws = h->desc.Ws;
  a.y = y;
  a.T = T;
  a.n = h->desc.d_out;
  a.k = h->desc.d_in;
  a.kb = cdiv(a.k, Q_GROUP);
  a.y_f32 = y_dtype == SFFN_FP32;
  a.status = h->status;
  return launched(launch_pdl(k_qlinear, dim3(cdiv(a.n, 32), cdiv(T, 8)), dim3(256), 0,
                             static_cast<cudaStream_t>(cuda_stream), 1, a));
}

extern "C" sffn_status sffn_qlinear_read_status(sffn_qlinear_handle* h, void* cuda_stream) {
  return h ? read_status_word(h->status, static_cast<cudaStream_t>(cuda_stream)) : SFFN_ERR_INVALID_ARG;
}

extern "C" sffn_status sffn_qlinear_destroy(sffn_qlinear_handle* h) {
  if (!h) return SFFN_OK;
  free_on(h->dev, h->status);
  delete h;
  return SFFN_OK;
}

// ---------------------------------------------------------------------------
// Experts' grouped products
struct sffn_grouped_handle {
  sffn_grouped_desc desc;
  int dev = 0, n_sm = 0;
  uint32_t* status = nullptr;   // [4]
};

extern "C" sffn_status sffn_grouped_create(const sffn_grouped_desc* desc, void* cuda_stream, sffn_grouped_handle** out) {
  if (!out) return SFFN_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || !desc->W || !aligned16(desc->W)) return SFFN_ERR_INVALID_ARG;
  if (desc->n_experts <= 0 || desc->d_in <= 0 || desc->d_out <= 0) return SFFN_ERR_INVALID_ARG;
  if (desc->n_experts > SFFN_GROUPED_MAX_EXPERTS || desc->d_in % 8 || desc->d_out % 8 || desc->d_in > (1 << 20) ||
      desc->d_out > (1 << 20))
    return SFFN_ERR_UNSUPPORTED;
  int dev = 0, n_sm = 0;
  const sffn_status ds = pick_device(&dev, &n_sm);
  if (ds != SFFN_OK) return ds;
  sffn_grouped_handle* h = new (std::nothrow) sffn_grouped_handle();
  if (!h) return SFFN_ERR_ALLOC;
  h->desc = *desc;
  h->dev = dev;
  h->n_sm = n_sm;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (!dalloc(&h->status, 16)) {
    delete h;
    return SFFN_ERR_ALLOC;
  }
  cudaError_t e = cudaMemsetAsync(h->status, 0, 16, st);
  e = e ? e : cudaStreamSynchronize(st);
  if (e) {
    free_on(dev, h->status);
    delete h;
    return SFFN_ERR_CUDA;
  }
  *out = h;
  return SFFN_OK;
}

namespace {

sffn_status grouped_check(const sffn_grouped_handle* h, const void* a, const int32_t* offsets, int R, const void* out,
                          int out_dtype) {
  if (!h || R < 0 || R > kMaxRows || !is_value_type(out_dtype) || !offsets) return SFFN_ERR_INVALID_ARG;
  if (R > 0 && (!a || !out || !aligned16(a) || !aligned16(out))) return SFFN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(offsets) & 3u) return SFFN_ERR_INVALID_ARG;
  return on_device(h->dev) ? SFFN_OK : SFFN_ERR_INVALID_ARG;
}

GroupedArgs grouped_args(const sffn_grouped_handle* h, const int32_t* offsets, int R, void* out, int out_dtype) {
  GroupedArgs g{};
  g.off = offsets;
  g.out = out;
  g.E = h->desc.n_experts;
  g.R = R;
  g.k = h->desc.d_in;
  g.n = h->desc.d_out;
  g.out_f32 = out_dtype == SFFN_FP32;
  g.status = h->status;
  return g;
}

}  // namespace

extern "C" sffn_status sffn_grouped_forward(sffn_grouped_handle* h, const void* x, const int32_t* offsets, int R,
                                            void* y, sffn_dtype y_dtype, void* cuda_stream) {
  const sffn_status s = grouped_check(h, x, offsets, R, y, y_dtype);
  if (s != SFFN_OK || R == 0) return s;
  GroupedArgs g = grouped_args(h, offsets, R, y, y_dtype);
  g.a = static_cast<const __nv_bfloat16*>(x);
  g.b = static_cast<const __nv_bfloat16*>(h->desc.W);
  return launched(launch_pdl(k_grouped_rows<0>, dim3(cdiv(g.n, 32), g.E), dim3(256), 0,
                             static_cast<cudaStream_t>(cuda_stream), 1, g));
}

extern "C" sffn_status sffn_grouped_backward_input(sffn_grouped_handle* h, const void* dy, const int32_t* offsets, int R,
                                                   void* dx, sffn_dtype dx_dtype, void* cuda_stream) {
  const sffn_status s = grouped_check(h, dy, offsets, R, dx, dx_dtype);
  if (s != SFFN_OK || R == 0) return s;
  GroupedArgs g = grouped_args(h, offsets, R, dx, dx_dtype);
  g.a = static_cast<const __nv_bfloat16*>(dy);
  g.b = static_cast<const __nv_bfloat16*>(h->desc.W);
  return launched(launch_pdl(k_grouped_rows<1>, dim3(cdiv(g.k, 32), g.E), dim3(256), 0,
                             static_cast<cudaStream_t>(cuda_stream), 1, g));
}

extern "C" sffn_status sffn_grouped_backward_weight(sffn_grouped_handle* h, const void* x, const void* dy,
                                                    const int32_t* offsets, int R, void* dW, sffn_dtype dw_dtype,
                                                    void* cuda_stream) {
  const sffn_status s = grouped_check(h, x, offsets, R, dW, dw_dtype);
  if (s != SFFN_OK) return s;
  if (!dW || !aligned16(dW) || (R > 0 && (!dy || !aligned16(dy)))) return SFFN_ERR_INVALID_ARG;
  GroupedArgs g = grouped_args(h, offsets, R, dW, dw_dtype);
  g.a = static_cast<const __nv_bfloat16*>(dy);
  g.b = static_cast<const __nv_bfloat16*>(x);
  return launched(launch_pdl(k_grouped_weight, dim3(cdiv(g.k, 32), cdiv(g.n, 8), g.E), dim3(256), 0,
                             static_cast<cudaStream_t>(cuda_stream), 1, g));
}

extern "C" sffn_status sffn_grouped_read_status(sffn_grouped_handle* h, void* cuda_stream) {
  return h ? read_status_word(h->status, static_cast<cudaStream_t>(cuda_stream)) : SFFN_ERR_INVALID_ARG;
}

extern "C" sffn_status sffn_grouped_destroy(sffn_grouped_handle* h) {
  if (!h) return SFFN_OK;
  free_on(h->dev, h->status);
  delete h;
  return SFFN_OK;
}
