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
constexpr long long kMaxTiles = 1 << 30;   // tiles of a launch are counted in 32 bits

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
  int shift;                   // thread index >> shift: row within the CTA
};

NormShape norm_shape(int d) {
  NormShape s;
  const int dv = d / 8;
  if (dv <= 128) {
    s.nv = 1;
    s.shift = dv <= 32 ? 5 : dv <= 64 ? 6 : 7;
    s.tpr = 1 << s.shift;
    s.threads = 256;
  } else {
    s.nv = dv <= 512 ? 1 : dv <= 1024 ? 2 : 4;
    s.shift = 10;
    s.tpr = s.threads = cdiv(cdiv(dv, s.nv), 32) * 32;
  }
  s.rpc = s.threads / s.tpr;
  return s;
}

// CTAs of the gradient: as many as the SMs' registers hold, at most four an SM,
// since each leaves a partial sum of dw; with T and d alone, for the workspace
// (148 SMs: on a device with another number the rounds are uneven, no more).
int norm_bwd_ctas(const NormShape& s, int T, int per_sm) {
  const int most = s.nv == 4 ? 1 : std::min(4, 1024 / s.threads);
  return std::min(cdiv(T, s.rpc), 148 * std::min(most, per_sm));
}

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

template <bool SF32, bool DYF32, bool DS, int NV>
cudaError_t norm_bwd_launch_nv(const NormBwdArgs& a, const NormShape& s, int& ctas, cudaStream_t st) {
  const int smem = NormBwdCfg<SF32, DYF32, DS, NV>::smem(s.threads);
  ctas = norm_bwd_ctas(s, a.T, 227 * 1024 / (smem + 2048));
  const auto kernel = k_rmsnorm_bwd<SF32, DYF32, DS, NV>;
  // set on every call: it belongs to the current device, and costs little
  const cudaError_t e =
      smem > 40 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
  if (e) {
    cudaGetLastError();
    return e;
  }
  return launch_pdl(kernel, dim3(ctas), dim3(s.threads), (size_t)smem, st, 1, a);
}
template <bool SF32, bool DYF32, bool DS>
cudaError_t norm_bwd_launch(const NormBwdArgs& a, const NormShape& s, int& ctas, cudaStream_t st) {
  switch (s.nv) {
    case 1: return norm_bwd_launch_nv<SF32, DYF32, DS, 1>(a, s, ctas, st);
    case 2: return norm_bwd_launch_nv<SF32, DYF32, DS, 2>(a, s, ctas, st);
    default: return norm_bwd_launch_nv<SF32, DYF32, DS, 4>(a, s, ctas, st);
  }
}
template <bool SF32, bool DYF32>
cudaError_t norm_bwd_launch_ds(const NormBwdArgs& a, const NormShape& s, int& ctas, cudaStream_t st) {
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
  a.shift = s.shift;
  a.rpc = s.rpc;
  const int res = !residual ? 0 : desc->residual_dtype == SFFN_FP32 ? 2 : 1;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return launched(desc->x_dtype == SFFN_FP32 ? norm_launch_res<true>(res, desc->y_dtype, a, s, st)
                                             : norm_launch_res<false>(res, desc->y_dtype, a, s, st));
}

extern "C" sffn_status sffn_rmsnorm_workspace_bytes(int d, int T, size_t* bytes) {
  if (!bytes || d <= 0 || T < 0 || T > kMaxRows) return SFFN_ERR_INVALID_ARG;
  if (d % 8 || d > NORM_MAX_D) return SFFN_ERR_UNSUPPORTED;
  const NormShape s = norm_shape(d);
  *bytes = (size_t)norm_bwd_ctas(s, T, 4) * d * sizeof(float);
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
  int ctas = 0;   // as launched
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
  a.shift = s.shift;
  a.rpc = s.rpc;
  a.w_f32 = desc->weight_dtype == SFFN_FP32;
  a.eps = desc->eps;
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    const bool sf = desc->residual_dtype == SFFN_FP32, yf = desc->y_dtype == SFFN_FP32;
    e = sf ? (yf ? norm_bwd_launch_ds<true, true>(a, s, ctas, st) : norm_bwd_launch_ds<true, false>(a, s, ctas, st))
           : (yf ? norm_bwd_launch_ds<false, true>(a, s, ctas, st) : norm_bwd_launch_ds<false, false>(a, s, ctas, st));
  }
  e = e ? e
        : launch_pdl(k_rmsnorm_dw, dim3(cdiv(desc->d, 32)), dim3(512), 0, st, 1, (const float*)workspace, ctas,
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
  // clusters of 1, 2, 4 and 8 CTAs that the GPU holds at once, one CTA per SM
  int cols_slots[4] = {0, 0, 0, 0}, rows_slots[4] = {0, 0, 0, 0};
  uint32_t* status = nullptr;   // [4]
};

namespace {

// Tensor map of e4m3 codes [rows][inner], box 128 x box_rows, 128-byte swizzle.
bool code_map(CUtensorMap* m, const void* base, long long inner, long long rows, int box_rows) {
  const EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)inner};
  const cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map of an output [rows][cols], stored 64 bytes x 32 rows at a time.
bool out_map(CUtensorMap* m, void* base, int f32, long long cols, long long rows) {
  const EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 16u : 32u, 32u};
  const cuuint32_t es[2] = {1u, 1u};
  return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN>
cudaError_t qlinear_cols_attr() {
  return cudaFuncSetAttribute(k_qlinear_cols<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, QcCfg<BN>::SMEM);
}

template <int BN>
sffn_status qlinear_cols(const sffn_qlinear_handle* h, const void* xq, QlinArgs a, cudaStream_t st) {
  // How many CTAs share a tile's k, and how many weight rows a tile has: the
  // least time by a model of it, in cycles.  Every cluster that fits gets one
  // tile of even height, or several.  A block of k costs its bytes at 25 per
  // cycle and SM (the SMs' share of the memory bandwidth), and no less than its
  // MMAs and its pass through the epilogue; a sum over a cluster costs 3000.
  // Measured with d_in 14336, d_out 4096: 13 tokens by 1, 2, 4, 8 CTAs 18.5, 14.6,
  // 14.4, 24.6 us, 32 tokens 23.5, 17.0, 14.4, 27.1; d_in 4096, d_out 14336, 13
  // tokens 12.8, 18.3, 25.8, 47.2.
  constexpr int LEAST = BN <= 16 ? 220 : 300;
  long long best = -1;
  for (int i = 0; i < 4; ++i) {
    const int split = 1 << i, c = h->cols_slots[i];
    if (c <= 0 || (split > 1 && a.kb < 4 * split)) continue;
    const int rows = std::min(128, std::max(8, cdiv(cdiv(a.n, c), 8) * 8)), tiles = cdiv(a.n, rows);
    const long long cost =
        (long long)cdiv(tiles, c) * cdiv(a.kb, split) * std::max(rows * 128 / 25, LEAST) + (split > 1 ? 3000 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      a.split = split;
      a.h = rows;
    }
  }
  CUtensorMap mW, mX;
  if (!code_map(&mW, h->desc.Wq, a.k, a.n, a.h) || !code_map(&mX, xq, a.k, a.T, cdiv(a.T, 16) * 16)) return SFFN_ERR_CUDA;
  return launched(launch_pdl(k_qlinear_cols<BN>, dim3(cdiv(a.n, a.h) * a.split), dim3(QL_THREADS), (size_t)QcCfg<BN>::SMEM,
                             st, a.split, mW, mX, a));
}

template <int BN>
cudaError_t qlinear_rows_attr() {
  return cudaFuncSetAttribute(k_qlinear_rows<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, QrCfg<BN>::SMEM);
}

template <int BN>
sffn_status qlinear_rows_launch(const sffn_qlinear_handle* h, const void* xq, const QlinArgs& a, long long ctas,
                                cudaStream_t st) {
  CUtensorMap mX, mW, mY;
  if (!code_map(&mX, xq, a.k, a.T, 128) || !code_map(&mW, h->desc.Wq, a.k, a.n, BN) ||
      !out_map(&mY, a.y, a.y_f32, a.n, a.T))
    return SFFN_ERR_CUDA;
  return launched(launch_pdl(k_qlinear_rows<BN>, dim3((unsigned)ctas), dim3(QR_THREADS), (size_t)QrCfg<BN>::SMEM, st,
                             a.split, mX, mW, mY, a));
}

sffn_status qlinear_rows(const sffn_qlinear_handle* h, const void* xq, QlinArgs a, cudaStream_t st) {
  // Tiles of 128 or 256 columns, and how many CTAs share a tile's k where all
  // of the tiles fit at once: the least time by a model of it, in ns.  A block
  // of k takes 360 with 128 columns and 565 with 256; a sum over a cluster costs
  // 5000.  Measured in us, 128 and 256 columns: d_in 2048, d_out 8192, 256 tokens
  // 9.8 and 13.3, 333 tokens (two rounds and one) 15.9 and 13.4, 4096 tokens 89 and
  // 74; d_in 14336, d_out 4096, 768 tokens 81 and 60, 64 tokens by 1, 2, 4 CTAs
  // 42, 26.7, 17.8; d_in 2048, d_out 8192, 128 tokens by 1 and 2 CTAs 9.3 and 11.3.
  const long long mt = cdiv(a.T, 128), narrow = mt * cdiv(a.n, 128), wide = mt * cdiv(a.n, 256);
  if (narrow > kMaxTiles) return SFFN_ERR_UNSUPPORTED;
  a.split = 1;
  const long long cost_wide = cdiv(wide, h->n_sm) * (a.kb * 565ll + 1500);
  long long best = cdiv(narrow, h->n_sm) * (a.kb * 360ll + 400);
  for (int i = 1; i < 4; ++i) {
    const int split = 1 << i;
    if (narrow > h->rows_slots[i] || a.kb < 4 * split) continue;
    const long long cost = cdiv(a.kb, split) * 360ll + 5000;
    if (cost < best) {
      best = cost;
      a.split = split;
    }
  }
  if (cost_wide >= best)
    return qlinear_rows_launch<128>(h, xq, a, a.split > 1 ? narrow * a.split : std::min<long long>(narrow, h->n_sm), st);
  a.split = 1;
  return qlinear_rows_launch<256>(h, xq, a, std::min<long long>(wide, h->n_sm), st);
}

// Clusters of 2, 4 and 8 CTAs of a kernel that the GPU holds at once.
template <typename Kernel>
cudaError_t count_clusters(Kernel kernel, int threads, int smem, int (&slots)[4]) {
  cudaError_t e = cudaSuccess;
  for (int i = 1; i < 4 && !e; ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1 << i;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(1 << i);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&slots[i], kernel, &cfg);
  }
  return e;
}

}  // namespace

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
  e = e ? e : qlinear_cols_attr<16>();
  e = e ? e : qlinear_cols_attr<32>();
  e = e ? e : qlinear_rows_attr<128>();
  e = e ? e : qlinear_rows_attr<256>();
  e = e ? e : cudaStreamSynchronize(st);
  h->cols_slots[0] = h->rows_slots[0] = n_sm;
  e = e ? e : count_clusters(k_qlinear_cols<16>, QL_THREADS, QcCfg<16>::SMEM, h->cols_slots);
  e = e ? e : count_clusters(k_qlinear_rows<128>, QR_THREADS, QrCfg<128>::SMEM, h->rows_slots);
  if (e || !get_encode()) {
    cudaGetLastError();
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
  a.xs = xs;
  a.Ws = h->desc.Ws;
  a.y = y;
  a.T = T;
  a.n = h->desc.d_out;
  a.k = h->desc.d_in;
  a.kb = cdiv(a.k, Q_GROUP);
  a.y_f32 = y_dtype == SFFN_FP32;
  a.status = h->status;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  // Up to 32 tokens cost less as the MMA's columns than as a quarter of its rows:
  // measured at 16 / 32 / 40 tokens, d_in 4096, d_out 14336, 16 columns 12.8, 32
  // columns 13.9 / 14.3, 64 columns 15.4 / 16.1 / 16.4 (taken out), rows 15.9 us at
  // all three; d_in 2048, d_out 8192: 5.7, 6.7 / 7.2, 9.8 / 10.2 / 10.3, rows 9.8.
  if (T <= 16) return qlinear_cols<16>(h, xq, a, st);
  if (T <= 32) return qlinear_cols<32>(h, xq, a, st);
  return qlinear_rows(h, xq, a, st);
}

extern "C" sffn_status sffn_qlinear_quantize_forward(sffn_qlinear_handle* h, const void* x, sffn_dtype x_dtype, int T,
                                                     void* y, sffn_dtype y_dtype, void* workspace,
                                                     size_t workspace_bytes, void* cuda_stream) {
  if (!h || T < 0 || T > kMaxRows || !is_value_type(x_dtype) || !is_value_type(y_dtype)) return SFFN_ERR_INVALID_ARG;
  if (T == 0) return SFFN_OK;
  const size_t codes = ((size_t)T * h->desc.d_in + 15) & ~(size_t)15;
  const size_t scales = (size_t)T * cdiv(h->desc.d_in, Q_GROUP) * sizeof(float);
  if (!x || !y || !workspace || !aligned16(x) || !aligned16(y) || !aligned16(workspace) ||
      workspace_bytes < codes + scales)
    return SFFN_ERR_INVALID_ARG;
  if (!on_device(h->dev)) return SFFN_ERR_INVALID_ARG;
  float* xs = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + codes);
  const sffn_status s = sffn_quantize_rows(x, x_dtype, T, h->desc.d_in, workspace, xs, cuda_stream);
  return s != SFFN_OK ? s : sffn_qlinear_forward(h, workspace, xs, T, y, y_dtype, cuda_stream);
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
  int slots[4] = {0, 0, 0, 0};  // clusters of 1, 2, 4 and 8 CTAs that the GPU holds at once, one CTA per SM
  uint32_t* status = nullptr;   // [4]
  CUtensorMap mW, mWT;          // W as the forward's (K-major) and the input gradient's (M-major) operand
};

namespace {

// Tensor map of bf16 [planes][rows][inner] (planes 0: two dimensions), box 64 x
// box_rows, 128-byte swizzle.
bool grouped_map(CUtensorMap* m, const void* base, long long inner, long long rows, int planes, int box_rows) {
  const EncodeTiledFn enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)inner * 2, (cuuint64_t)inner * rows * 2};
  const cuuint32_t box[3] = {64u, (cuuint32_t)box_rows, 1u};
  const cuuint32_t es[3] = {1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 3 : 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int CTAS, int BN>
cudaError_t grouped_attr() {
  return cudaFuncSetAttribute(k_grouped<MODE, CTAS, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              GtCfg<CTAS, BN>::SMEM);
}

// One launch: the columns' operand map(s) of this call, then the kernel.
template <int MODE, int CTAS, int BN>
sffn_status grouped_launch(const sffn_grouped_handle* h, const CUtensorMap& mA, const void* cols, long long inner,
                           const GroupedArgs& g, long long tiles, cudaStream_t st) {
  CUtensorMap mB;
  if (!grouped_map(&mB, cols, inner, g.R, 0, MODE == GROUPED_DW ? 64 : GtCfg<CTAS, BN>::BOX)) return SFFN_ERR_CUDA;
  const int cluster = CTAS * g.split;
  const int grid = (int)std::min<long long>(tiles, h->n_sm / CTAS) * cluster;   // a split has no more tiles than fit
  return launched(launch_pdl(k_grouped<MODE, CTAS, BN>, dim3(grid), dim3(GT_THREADS), (size_t)GtCfg<CTAS, BN>::SMEM, st,
                             cluster, mA, mB, g));
}

// Products over the rows of every group (forward, input gradient).
template <int MODE>
sffn_status grouped_rows(const sffn_grouped_handle* h, const CUtensorMap& mA, const void* rows, GroupedArgs g,
                         cudaStream_t st) {
  const long long tiles = (long long)cdiv(g.M, 128) * (g.R / 32 + g.E);
  if (tiles > kMaxTiles) return SFFN_ERR_UNSUPPORTED;
  // Columns per tile, by the mean rows of an expert, since a second tile of
  // columns reads the expert's weight again.  Measured in us with 32, 128, 256
  // columns (256: CTA pairs), 8 experts of 4096 x 14336 | 32 of 2048 x 1024:
  //   mean rows    forward                               input gradient
  //       2        129 138 141  |  25.0 25.6 26.5        137 133 136  |  21.2 20.8 22.3
  //      16        154 164 167  |  25.3 25.7 27.2        149 141 148  |  25.7 25.6 27.2
  //      32                     |  29.2 27.1 28.7                     |  30.5 26.4 28.5
  //     104        391 171 179  |  61.4 28.7 30.8        396 152 153  |  65.0 28.6 30.9
  //     120        419 192 178  |  68.4 35.9 31.2        446 193 159  |  68.7 32.6 31.4
  //     256                     |   126 49.7 43.1                     |   133 47.9 43.2
  if (g.R >= 112ll * g.E) return grouped_launch<MODE, 2, 256>(h, mA, rows, g.K, g, tiles, st);
  if (g.R >= (MODE == GROUPED_FWD ? 24ll : 8ll) * g.E) return grouped_launch<MODE, 1, 128>(h, mA, rows, g.K, g, tiles, st);
  // A few rows: no more tiles than this, since no more groups have a row.  Where
  // they leave SMs idle, clusters share a tile's k, by a model of the time in ns:
  // a block of k takes 240, a sum over the cluster 3000.  Measured without and
  // with: 2 rows of 14336 to 4096 57 and 32 us, 4 rows (of 4 groups) of 8192 to 2048
  // 34 and 20.5, 1 row of 4096 to 1024 18.5 and 7.6.
  const long long few = (long long)cdiv(g.M, 128) * (g.R / 32 + std::min(g.E, g.R));
  const int kb = cdiv(g.K, GT_BK);
  long long best = kb * 240ll;
  for (int i = 1; i < 4; ++i) {
    const int split = 1 << i;
    if (few > h->slots[i] || kb < 4 * split) continue;
    const long long cost = cdiv(kb, split) * 240ll + 3000;
    if (cost < best) {
      best = cost;
      g.split = split;
    }
  }
  return grouped_launch<MODE, 1, 32>(h, mA, rows, g.K, g, few, st);
}

}  // namespace

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
  const int E = desc->n_experts;
  cudaError_t e = cudaMemsetAsync(h->status, 0, 16, st);
  if (!e && (!grouped_map(&h->mW, desc->W, desc->d_in, desc->d_out, E, 128) ||
             !grouped_map(&h->mWT, desc->W, desc->d_in, desc->d_out, E, 64)))
    e = cudaErrorInvalidValue;
  e = e ? e : grouped_attr<GROUPED_FWD, 2, 256>();
  e = e ? e : grouped_attr<GROUPED_FWD, 1, 128>();
  e = e ? e : grouped_attr<GROUPED_FWD, 1, 32>();
  e = e ? e : grouped_attr<GROUPED_DX, 2, 256>();
  e = e ? e : grouped_attr<GROUPED_DX, 1, 128>();
  e = e ? e : grouped_attr<GROUPED_DX, 1, 32>();
  e = e ? e : grouped_attr<GROUPED_DW, 2, 256>();
  h->slots[0] = n_sm;
  e = e ? e : count_clusters(k_grouped<GROUPED_FWD, 1, 32>, GT_THREADS, GtCfg<1, 32>::SMEM, h->slots);
  e = e ? e : cudaStreamSynchronize(st);
  if (e) {
    cudaGetLastError();
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

// The tensor core drops what lies below its sum's 24 bits at each step of 16
// terms, up to 2^-22 of the sum and always towards zero, so runs of blocks are
// added up in fp32 registers.  For an fp32 output 512 terms (8 blocks), with which
// 512 to 4096 terms of one sign came out at most 2.7e-7 off; for a bf16 output
// 16384 terms (256 blocks), whose 1024 steps stay below 2^-12, at most an eighth
// of the output's rounding.  2^20 terms in one run came out 6e-3 low.
GroupedArgs grouped_args(const sffn_grouped_handle* h, const int32_t* offsets, int R, void* out, int out_dtype) {
  GroupedArgs g{};
  g.off = offsets;
  g.out = out;
  g.E = h->desc.n_experts;
  g.R = R;
  g.out_f32 = out_dtype == SFFN_FP32;
  g.split = 1;
  g.kchunk = g.out_f32 ? 8 : 256;
  g.status = h->status;
  return g;
}

}  // namespace

extern "C" sffn_status sffn_grouped_forward(sffn_grouped_handle* h, const void* x, const int32_t* offsets, int R,
                                            void* y, sffn_dtype y_dtype, void* cuda_stream) {
  const sffn_status s = grouped_check(h, x, offsets, R, y, y_dtype);
  if (s != SFFN_OK || R == 0) return s;
  GroupedArgs g = grouped_args(h, offsets, R, y, y_dtype);
  g.M = h->desc.d_out;
  g.K = h->desc.d_in;
  return grouped_rows<GROUPED_FWD>(h, h->mW, x, g, static_cast<cudaStream_t>(cuda_stream));
}

extern "C" sffn_status sffn_grouped_backward_input(sffn_grouped_handle* h, const void* dy, const int32_t* offsets, int R,
                                                   void* dx, sffn_dtype dx_dtype, void* cuda_stream) {
  const sffn_status s = grouped_check(h, dy, offsets, R, dx, dx_dtype);
  if (s != SFFN_OK || R == 0) return s;
  GroupedArgs g = grouped_args(h, offsets, R, dx, dx_dtype);
  g.M = h->desc.d_in;
  g.K = h->desc.d_out;
  return grouped_rows<GROUPED_DX>(h, h->mWT, dy, g, static_cast<cudaStream_t>(cuda_stream));
}

extern "C" sffn_status sffn_grouped_backward_weight(sffn_grouped_handle* h, const void* x, const void* dy,
                                                    const int32_t* offsets, int R, void* dW, sffn_dtype dw_dtype,
                                                    void* cuda_stream) {
  const sffn_status s = grouped_check(h, x, offsets, R, dW, dw_dtype);
  if (s != SFFN_OK) return s;
  if (!dW || !aligned16(dW) || (R > 0 && (!dy || !aligned16(dy)))) return SFFN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  GroupedArgs g = grouped_args(h, offsets, R, dW, dw_dtype);
  g.M = h->desc.d_in;
  g.N = h->desc.d_out;
  if (R == 0)
    return launched(cudaMemsetAsync(dW, 0, (size_t)g.E * g.M * g.N * (g.out_f32 ? 4 : 2), st));
  CUtensorMap mx;
  if (!grouped_map(&mx, x, g.M, R, 0, 64)) return SFFN_ERR_CUDA;
  const long long tiles = (long long)g.E * cdiv(g.M, 256) * cdiv(g.N, 256);
  if (tiles > kMaxTiles) return SFFN_ERR_UNSUPPORTED;
  return grouped_launch<GROUPED_DW, 2, 256>(h, mx, dy, g.N, g, tiles, st);
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
