// Linear layer with both operands in e4m3: per 128-wide block b of the inner
// dimension,
//
//   y[t][n] = sum_b xs[t][b] · Ws[n/128][b] · sum_{k in b} xq[t][k] · Wq[n][k]
//
// The tensor core adds up one block (four MMAs of 32) in TMEM; each block's
// sums are then scaled and added in fp32 registers, while the MMAs of the next
// blocks run in other TMEM columns.
//
// k_qlinear_cols: few tokens.  Weight rows are the MMA's 128 rows (TMEM
// lanes), tokens its columns, so that a token costs little and W is read
// once.  Bound by W's bytes.  A CTA takes `h` weight rows (a multiple of 8, up
// to 128) over all of k, with h chosen to give every SM one tile: a tile of
// fewer rows leaves lanes of the MMA unused, which costs nothing here, and
// needs no sum over CTAs.
#pragma once

#include "ptx_pair.cuh"
#include "vec8.cuh"

namespace sffn {

constexpr int QL_SMEM = 227 * 1024;
constexpr int QL_EPI_WARPS = 8;
constexpr int QL_PRODUCER = QL_EPI_WARPS, QL_MMA = QL_EPI_WARPS + 1, QL_SCALE = QL_EPI_WARPS + 2;
constexpr int QL_THREADS = (QL_EPI_WARPS + 3) * 32;

// Instruction descriptor, kind::f8f6f4: e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Two fp32 lanes at a time.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

struct QlinArgs {
  const float* xs;      // [T][kb]
  const float* Ws;      // [ceil(n/128)][kb]
  void* y;              // [T][n], bf16 or fp32
  int T, n, k, kb;
  int h;                // k_qlinear_cols: weight rows per CTA
  int each;             // k_qlinear_cols: tokens per CTA (a multiple of 16)
  int y_f32;
  uint32_t* status;
};

template <int BN>
struct QcCfg {
  static constexpr int KS = BN <= 64 ? 2 : 1;            // 128-wide blocks per stage
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = KS * (A_BYTES + B_BYTES);
  static constexpr int SCALES = KS * BN * 4;             // a stage's xs, [KS][BN]
  static constexpr int FIXED = 1024 + 512;
  static constexpr int RAW = (QL_SMEM - FIXED) / (STAGE + SCALES);
  static constexpr int STAGES = RAW > 8 ? 8 : RAW;
  static constexpr int SMEM = FIXED + STAGES * (STAGE + SCALES);
  static constexpr int NBUF = BN <= 64 ? 4 : 2;          // TMEM accumulators
  // Up to 64 columns the two epilogue warpgroups take every other block, above
  // that they halve the columns.
  static constexpr bool ALT = BN <= 64;
  static constexpr int COLS = ALT ? BN : BN / 2;         // columns per epilogue thread
};

template <int BN>
__global__ void __launch_bounds__(QL_THREADS, 1)
k_qlinear_cols(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const QlinArgs a) {
  using Cfg = QcCfg<BN>;
  constexpr int STAGES = Cfg::STAGES, KS = Cfg::KS, NBUF = Cfg::NBUF;
  constexpr uint32_t NCOLS = NBUF * BN;
  static_assert(NCOLS >= 32 && NCOLS <= 512 && (NCOLS & (NCOLS - 1)) == 0, "TMEM columns");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_xs = reinterpret_cast<float*>(smem + STAGES * Cfg::STAGE);   // [STAGES][KS][BN]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * (Cfg::STAGE + Cfg::SCALES));
  uint64_t* empty = full + STAGES;
  uint64_t* sfull = empty + STAGES;     // a stage's scales are there / have been used
  uint64_t* sempty = sfull + STAGES;
  uint64_t* accfull = sempty + STAGES;  // [NBUF]
  uint64_t* accfree = accfull + NBUF;   // [NBUF]
  uint64_t* mma_done = accfree + NBUF;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((4 * STAGES + 2 * NBUF + 1) * 8 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = blockIdx.x * a.h, n0 = blockIdx.y * a.each;
  const int cols = min(a.each, a.T - n0), bn = (cols + 15) & ~15;
  const int KB = a.kb, ns = (KB + KS - 1) / KS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], QL_EPI_WARPS);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accfree[b], Cfg::ALT ? 4 : QL_EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == QL_MMA) {
    tmem_alloc(tmem_slot, NCOLS);
    tmem_relinquish();
  }
  if (warp == QL_PRODUCER && lane == 0) {
    tma_prefetch_desc(&mW);
    tma_prefetch_desc(&mX);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();   // operands and outputs belong to the stream order

  if (warp == QL_PRODUCER) {
    // --------------------------------------------------------- TMA producer
    // Weight rows past the end and columns of k past the end arrive as zeros.
    bool ok = true;
    for (int i = 0; i < ns; ++i) {
      const int s = i % STAGES, f = i / STAGES;
      if (f > 0) ok = mbar_wait_warp(&empty[s], (f - 1) & 1, abort_flag, a.status);
      if (!ok) break;
      if (elect_one()) {
        uint8_t* st = smem + (size_t)s * Cfg::STAGE;
        const int nb = min(KS, KB - i * KS);
        mbar_expect_tx(&full[s], (uint32_t)(nb * (a.h + a.each) * 128));
        for (int j = 0; j < nb; ++j) {
          tma_2d<1>(st + j * Cfg::A_BYTES, &mW, smem_u32(&full[s]), (i * KS + j) * 128, m0);
          tma_2d<1>(st + KS * Cfg::A_BYTES + j * Cfg::B_BYTES, &mX, smem_u32(&full[s]), (i * KS + j) * 128, n0);
        }
      }
      __syncwarp();
    }
    if (!ok) {   // a CTA must not exit before its copies have landed: wait far longer than they take
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 1000000ull) __nanosleep(1000);
    }
  } else if (warp == QL_SCALE) {
    // --------------------------------------------- the tokens' scales, by stage
    for (int i = 0; i < ns; ++i) {
      const int s = i % STAGES, f = i / STAGES;
      if (f > 0 && !mbar_wait_warp(&sempty[s], (f - 1) & 1, abort_flag, a.status)) break;
      float v[KS][(BN + 31) / 32];
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int c = 0; c < (BN + 31) / 32; ++c) {
          const int kb = i * KS + j, col = c * 32 + lane;
          v[j][c] = kb < KB && col < cols ? a.xs[(size_t)(n0 + col) * KB + kb] : 0.0f;
        }
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int c = 0; c < (BN + 31) / 32; ++c)
          if (c * 32 + lane < BN) s_xs[(s * KS + j) * BN + c * 32 + lane] = v[j][c];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[s]);
    }
  } else if (warp == QL_MMA) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t idesc = idesc_e4m3_f32(128, bn);
    bool ok = true;
    for (int i = 0; i < ns && ok; ++i) {
      const int s = i % STAGES, f = i / STAGES;
      ok = mbar_wait_warp(&full[s], f & 1, abort_flag, a.status);
      if (!ok) break;
      for (int j = 0; j < KS; ++j) {
        const int kb = i * KS + j;
        if (kb >= KB) break;
        const int b = kb % NBUF;
        if (kb >= NBUF) ok = mbar_wait_warp(&accfree[b], (kb / NBUF - 1) & 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + (size_t)s * Cfg::STAGE + j * Cfg::A_BYTES);
        const uint32_t sb = smem_u32(smem + (size_t)s * Cfg::STAGE + KS * Cfg::A_BYTES + j * Cfg::B_BYTES);
        const uint64_t ad = sdesc_k_sw128(sa), bd = sdesc_k_sw128(sb);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pair_mma<1, true>(tmem + (uint32_t)(b * BN), ad + 2u * k, bd + 2u * k, idesc, k ? 1u : 0u);
          tc_commit(&accfull[b]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&empty[s]);
      __syncwarp();
    }
    if (elect_one()) tc_commit(mma_done);
    __syncwarp();
    if (lane == 0) {   // every MMA is complete before TMEM is freed
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(mma_done, 0)) {
        if (globaltimer() - t0 > SFFN_WAIT_LIMIT_NS) {
          atomicOr(a.status, DEV_ERR_TIMEOUT);
          break;
        }
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    constexpr int COLS = Cfg::COLS, P = COLS / 2;
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane, m = m0 + row;
    const int c0 = Cfg::ALT ? 0 : wg * COLS;            // first column of this thread
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool in = row < a.h && m < a.n;
    const float* ws = a.Ws + (size_t)(in ? m / Q_GROUP : 0) * KB;
    uint64_t acc[P];
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] = 0;
    bool ok = true;
    float w_next = ws[0];
    for (int i = 0; i < ns && ok; ++i) {
      const int s = i % STAGES, f = i / STAGES;
      ok = mbar_wait_warp(&sfull[s], f & 1, abort_flag, a.status);
      for (int j = 0; j < KS && ok; ++j) {
        const int kb = i * KS + j;
        if (kb >= KB) break;
        const float w = w_next;
        if (kb + 1 < KB) w_next = ws[kb + 1];
        if (Cfg::ALT && (kb & 1) != wg) continue;
        const int b = kb % NBUF;
        ok = mbar_wait_warp(&accfull[b], (kb / NBUF) & 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const float4* xs = reinterpret_cast<const float4*>(s_xs + (s * KS + j) * BN + c0);
        const uint64_t w2 = pack2(w, w);
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
          if (c0 + c < cols) {
            float v[16];
            tmem_ld16(tlane + (uint32_t)(b * BN + c0 + c), v);
#pragma unroll
            for (int u = 0; u < 16; u += 4) {
              const float4 x = xs[(c + u) / 4];
              acc[(c + u) / 2] = fma2(pack2(v[u], v[u + 1]), mul2(pack2(x.x, x.y), w2), acc[(c + u) / 2]);
              acc[(c + u) / 2 + 1] = fma2(pack2(v[u + 2], v[u + 3]), mul2(pack2(x.z, x.w), w2), acc[(c + u) / 2 + 1]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&accfree[b]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sempty[s]);
    }
    if (Cfg::ALT) {
      // The odd blocks' sums join the even blocks', through the ring's memory:
      // once both warpgroups have seen their last block, every copy and MMA of
      // this CTA has completed.
      named_bar_sync(1, QL_EPI_WARPS * 32);
      float* ex = reinterpret_cast<float*>(smem);       // [COLS][128]
      if (wg == 1)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float u, v;
          unpack2(acc[i], u, v);
          ex[(2 * i) * 128 + row] = u;
          ex[(2 * i + 1) * 128 + row] = v;
        }
      named_bar_sync(1, QL_EPI_WARPS * 32);
      if (wg == 0)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float u, v;
          unpack2(acc[i], u, v);
          acc[i] = pack2(u + ex[(2 * i) * 128 + row], v + ex[(2 * i + 1) * 128 + row]);
        }
    }
    if (in && !*abort_flag && !(Cfg::ALT && wg == 1)) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float u, v;
        unpack2(acc[i], u, v);
        const int c = c0 + 2 * i;
        const size_t at = (size_t)(n0 + c) * a.n + m;
        if (a.y_f32) {
          if (c < cols) reinterpret_cast<float*>(a.y)[at] = u;
          if (c + 1 < cols) reinterpret_cast<float*>(a.y)[at + a.n] = v;
        } else {
          if (c < cols) reinterpret_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16(u);
          if (c + 1 < cols) reinterpret_cast<__nv_bfloat16*>(a.y)[at + a.n] = __float2bfloat16(v);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == QL_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, NCOLS);
  }
}

}  // namespace sffn
