// Linear layer with both operands in e4m3: per 128-wide block b of the inner
// dimension,
//
//   y[t][n] = sum_b xs[t][b] · Ws[n/128][b] · sum_{k in b} xq[t][k] · Wq[n][k]
//
// The tensor core adds up one block (four MMAs of 32) in TMEM; each block's
// sums are then scaled and added in fp32 registers, two columns at a time,
// while the MMAs of the next blocks run in other TMEM columns.
//
// k_qlinear_cols: up to 32 tokens.  Weight rows are the MMA's 128 rows (TMEM
// lanes), tokens its columns, so that a token costs little and W is read
// once.  Bound by W's bytes: one token, d_in 4096, d_out 14336, 59 MB, 12 to 13 us
// of which some 4 are launch and set-up.  An MMA of 128 x 16 x 32 takes 45 cycles
// however many of its rows are used, and looking at a barrier 50 to 100, so a
// stage is two blocks with one barrier each way, and a narrow weight (few rows,
// long k) is cut along k over the CTAs of a cluster, which add their sums up
// through distributed shared memory in a fixed order: 13 tokens, d_in 14336,
// d_out 4096, 18.5 us without and 14.4 with.
//
// k_qlinear_rows: more tokens.  Tokens are the MMA's rows, so that a token's
// scale is one register per thread.  4096 tokens, d_in 4096, d_out 14336: 253 us,
// 1.9 PFLOP/s.  A block of 128 x 256 takes about 1000 cycles: 512 are MMAs, 768
// the least that shared memory needs at 128 bytes a cycle (48 KB in by copies, 48
// KB out to the MMAs), and the sums' way from TMEM takes 560.  CTA pairs, which
// halve the weights' part, took 259 us (the second CTA's epilogue has to signal
// the first); halves of 128 columns with barriers of their own 277 (the tokens
// are read from shared memory twice).  From 129 to some 1000 tokens whole rounds of
// tiles bound it, with SMs idle in the last: 333 tokens, 4096 to 14336, 39 us, 14336
// to 4096 42 us.
#pragma once

#include "ptx_pair.cuh"
#include "vec8.cuh"

namespace sffn {

constexpr int QL_SMEM = 227 * 1024;
constexpr int QL_EPI_WARPS = 8;
constexpr int QL_PRODUCER = QL_EPI_WARPS, QL_SCALE = QL_EPI_WARPS + 1, QL_MMA = QL_EPI_WARPS + 2;   // QL_MMA, + 1
constexpr int QL_THREADS = (QL_EPI_WARPS + 4) * 32;

// Instruction descriptor, kind::f8f6f4: e4m3 x e4m3 -> fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

struct QlinArgs {
  const float* xs;      // [T][kb]
  const float* Ws;      // [ceil(n/128)][kb]
  void* y;              // [T][n], bf16 or fp32
  int T, n, k, kb;
  int h;                // k_qlinear_cols: weight rows per CTA
  int split;            // CTAs of a cluster, each with a part of k
  int y_f32;
  uint32_t* status;
};

__device__ __forceinline__ void put_y(void* y, int f32, size_t at, float v) {
  if (f32) reinterpret_cast<float*>(y)[at] = v;
  else reinterpret_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16(v);
}

template <int BN>
struct QcCfg {
  static constexpr int KS = 2;                           // 128-wide blocks per stage
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = KS * (A_BYTES + B_BYTES);
  static constexpr int SLOT = BN + 4;                    // scales of a block: tokens, two weight blocks
  static constexpr int SCALES = KS * SLOT * 4;
  static constexpr int FIXED = 1024 + 512;
  // An even number: the MMA threads and the epilogue warpgroups take every
  // other stage, and each may only ever wait on barriers whose every phase it
  // waits for: a phase's parity says nothing about the phases it has not seen.
  static constexpr int RAW = (QL_SMEM - FIXED) / (STAGE + SCALES);
  static constexpr int STAGES = (RAW > 8 ? 8 : RAW) & ~1;
  static constexpr int SMEM = FIXED + STAGES * (STAGE + SCALES);
  static constexpr int NBUF = 4;                         // TMEM accumulators, KS · BN columns each
};

template <int BN>
__global__ void __launch_bounds__(QL_THREADS, 1)
k_qlinear_cols(const __grid_constant__ CUtensorMap mW, const __grid_constant__ CUtensorMap mX, const QlinArgs a) {
  using Cfg = QcCfg<BN>;
  constexpr int STAGES = Cfg::STAGES, KS = Cfg::KS, NBUF = Cfg::NBUF;
  constexpr uint32_t NCOLS = NBUF * KS * BN;
  static_assert(NCOLS >= 32 && NCOLS <= 512 && (NCOLS & (NCOLS - 1)) == 0, "TMEM columns");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* slots = reinterpret_cast<float*>(smem + STAGES * Cfg::STAGE);  // [STAGES][KS][SLOT]
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
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  const int m0 = (blockIdx.x / a.split) * a.h, cols = a.T, bn = (cols + 15) & ~15;
  // this CTA's blocks of k
  const int kb0 = (int)((long long)a.kb * rank / a.split), kb1 = (int)((long long)a.kb * (rank + 1) / a.split);
  const int ns = (kb1 - kb0 + KS - 1) / KS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 32);
      mbar_init(&sempty[s], QL_EPI_WARPS / 2);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accfree[b], QL_EPI_WARPS / 2);
    }
    mbar_init(mma_done, 2);
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
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < ns; ++i) {
      if (!mbar_wait_warp(&empty[s], ph, abort_flag, a.status)) break;   // the first round passes
      if (elect_one()) {
        uint8_t* st = smem + (size_t)s * Cfg::STAGE;
        const int kb = kb0 + i * KS, nb = min(KS, kb1 - kb);
        const uint32_t bar = smem_u32(&full[s]);
        mbar_expect_tx(&full[s], (uint32_t)(nb * (a.h + bn) * 128));
        for (int j = 0; j < nb; ++j) {
          tma_2d<1>(st + j * Cfg::A_BYTES, &mW, bar, (kb + j) * 128, m0);
          tma_2d<1>(st + KS * Cfg::A_BYTES + j * Cfg::B_BYTES, &mX, bar, (kb + j) * 128, 0);
        }
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
  } else if (warp == QL_SCALE) {
    // ----------------------------------------------------- scales, by stage
    int s = 0;
    uint32_t ph = 1;
    const int nblk = (a.n + Q_GROUP - 1) / Q_GROUP;
    const float* ws = a.Ws + (size_t)min(m0 / Q_GROUP + (lane & 1), nblk - 1) * a.kb;
    for (int i = 0; i < ns; ++i) {
      if (!mbar_wait_warp(&sempty[s], ph, abort_flag, a.status)) break;   // the first round passes
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int kb = min(kb0 + i * KS + j, kb1 - 1);
        float* slot = slots + (s * KS + j) * Cfg::SLOT;
#pragma unroll
        for (int col = lane; col < BN; col += 32)
          copy4_async(slot + col, a.xs + (size_t)min(col, cols - 1) * a.kb + kb, col < cols);
        if (lane < 2) copy4_async(slot + BN + lane, ws + kb, true);
      }
      copies_arrive(&sfull[s]);
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    copies_wait_all();
  } else if (warp >= QL_MMA) {
    // ---------------------------------------------------------- MMA issuers
    // One thread of each of two warps, every other stage each: an MMA's issue
    // waits for the one before it, so what a thread does between its MMAs
    // (looking at barriers, mostly) leaves the tensor core idle unless another
    // thread's are there.
    const uint32_t idesc = idesc_e4m3_f32(128, bn);
    const uint64_t desc0 = sdesc_k_sw128(smem_u32(smem));
    if (elect_one()) {
      for (int i = warp - QL_MMA; i < ns; i += 2) {
        const int s = i % STAGES, b = i % NBUF;
        if (!mbar_wait(&full[s], (i / STAGES) & 1, abort_flag, a.status) ||
            !mbar_wait(&accfree[b], (i / NBUF + 1) & 1, abort_flag, a.status))   // free in the first round
          break;
        tc_fence_after();
        const uint64_t ad = desc0 + (uint32_t)(s * (Cfg::STAGE / 16)), bd = ad + KS * (Cfg::A_BYTES / 16);
        const int nb = min(KS, kb1 - kb0 - i * KS);
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (j < nb) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pair_mma<1, true>(tmem + (uint32_t)((b * KS + j) * BN), ad + j * (Cfg::A_BYTES / 16) + 2 * k,
                                bd + j * (Cfg::B_BYTES / 16) + 2 * k, idesc, k ? 1u : 0u);
          }
        tc_commit(&accfull[b]);
        tc_commit(&empty[s]);
      }
      tc_commit(mma_done);
    }
    __syncwarp();
    mbar_drain(mma_done, 0, a.status);   // every MMA is complete before TMEM is freed
  } else {
    // ------------------------------------------------------------- epilogue
    // Two warpgroups, every other stage each.
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane, m = m0 + row;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool in = row < a.h && m < a.n;
    const int blk = in ? m / Q_GROUP - m0 / Q_GROUP : 0;   // h <= 128: one of two weight blocks
    uint64_t sum[BN / 2];   // of two columns each
#pragma unroll
    for (int i = 0; i < BN / 2; ++i) sum[i] = 0;
    for (int i = wg; i < ns; i += 2) {
      const int s = i % STAGES, b = i % NBUF, kb = kb0 + i * KS;
      // A failed wait is not acted on (nothing is stored then, by any CTA that
      // shares the tile): leaving the loop from its middle would cost a select
      // per sum.
      mbar_wait_warp(&sfull[s], (i / STAGES) & 1, abort_flag, a.status);
      mbar_wait_warp(&accfull[b], (i / NBUF) & 1, abort_flag, a.status);
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        if (kb + j < kb1) {
          const float* slot = slots + (s * KS + j) * Cfg::SLOT;
          const float4* xs = reinterpret_cast<const float4*>(slot);
          const uint64_t w = pack2(slot[BN + blk], slot[BN + blk]);
#pragma unroll
          for (int c = 0; c < BN; c += 16) {
            uint64_t v[8];
            tmem_get16x2(tlane + (uint32_t)((b * KS + j) * BN + c), v);
#pragma unroll
            for (int u = 0; u < 8; u += 2) {
              const float4 x = xs[c / 4 + u / 2];
              sum[c / 2 + u] = fma2(v[u], mul2(pack2(x.x, x.y), w), sum[c / 2 + u]);
              sum[c / 2 + u + 1] = fma2(v[u + 1], mul2(pack2(x.z, x.w), w), sum[c / 2 + u + 1]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&accfree[b]);
        mbar_arrive(&sempty[s]);
      }
    }
    float acc[BN];
#pragma unroll
    for (int i = 0; i < BN / 2; ++i) unpack2(sum[i], acc[2 * i], acc[2 * i + 1]);
    float* ex = reinterpret_cast<float*>(smem);       // [BN][128], in the ring's memory (see below)
    // Once both warpgroups have seen their last stage, every copy and MMA of
    // this CTA has completed and the ring is free.
    named_bar_sync(1, QL_EPI_WARPS * 32);
    if (wg == 1)
#pragma unroll
      for (int i = 0; i < BN; ++i) ex[i * 128 + row] = acc[i];
    named_bar_sync(1, QL_EPI_WARPS * 32);
    if (wg == 0) {   // the odd stages' sums join the even stages'
#pragma unroll
      for (int i = 0; i < BN; ++i) acc[i] += ex[i * 128 + row];
      if (a.split > 1) {
#pragma unroll
        for (int i = 0; i < BN; ++i) ex[i * 128 + row] = acc[i];
      } else if (in && !*abort_flag) {
#pragma unroll
        for (int i = 0; i < BN; ++i)
          if (i < cols) put_y(a.y, a.y_f32, (size_t)i * a.n + m, acc[i]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (a.split > 1) {
    spread_abort(abort_flag, a.split);
    cluster_sync();   // every CTA's sums are in its ex
    // CTA `rank` adds up and stores every split-th column
    const int row = threadIdx.x & 127, m = m0 + row;
    if (threadIdx.x < QL_EPI_WARPS * 32 && row < a.h && m < a.n && !*abort_flag) {
      const uint32_t ex = smem_u32(smem);
      const int step = 2 * a.split;
      for (int c = rank + a.split * (threadIdx.x >> 7); c < cols; c += 4 * step) {   // up to cols + 3 steps < BN + 64
        float v[4];
        cluster_sums<4>(ex + (uint32_t)(c * 128 + row) * 4, (uint32_t)step * 512, a.split, v);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + step * q < cols) put_y(a.y, a.y_f32, (size_t)(c + step * q) * a.n + m, v[q]);
      }
    }
    __syncwarp();
    cluster_sync();   // nobody leaves while its sums are read
  }
  __syncthreads();
  if (*abort_flag) drain_copies();
  if (warp == QL_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, NCOLS);
  }
}

// ---------------------------------------------------------------- many tokens
// Every block's sums (128 x BN per CTA) pass from TMEM through registers, while
// the next block's MMAs (four of 128 cycles at 256 columns) run.  A warp spends
// most of that in latencies (a barrier, its scales, its reads of TMEM), so
// sixteen warps share it, a quarter of the columns each: a block of 128 columns
// took 540 ns with eight warps that read 256 whatever the tile, 360 so.
constexpr int QR_EPI_WARPS = 16;
constexpr int QR_PRODUCER = QR_EPI_WARPS, QR_SCALE = QR_EPI_WARPS + 1, QR_MMA = QR_EPI_WARPS + 2;
constexpr int QR_THREADS = (QR_EPI_WARPS + 3) * 32;
// Scales of four blocks: 128 tokens' and 2 weight blocks', four values
// each.  Every token's come from another line, with the latency of L2: 16
// blocks of them are in flight.  The MMAs' operands and the copies that bring
// them take most of shared memory's bandwidth, so a thread fetches four
// blocks' scales with three loads.
constexpr int QR_SLOTS = 4, QR_SLOT = 4 * 130;
// y leaves through shared memory, 64 bytes of 32 rows per warp at a time, as
// tiled copies: a thread's own stores (16 bytes of 32 rows each) took as long
// as ten blocks of MMAs.
constexpr int QR_OUT = 32 * 64;
// BN: weight rows per tile, 128 or 256.
template <int BN>
struct QrCfg {
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int FIXED = 1024 + 512 + QR_SLOTS * QR_SLOT * 4 + QR_EPI_WARPS * QR_OUT;
  static constexpr int RAW = (QL_SMEM - FIXED) / STAGE;
  static constexpr int STAGES = RAW > 6 ? 6 : RAW;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
  static constexpr int NBUF = 512 / BN;                 // TMEM accumulators
  static constexpr int COLS = BN / 4;                   // columns per epilogue thread
};

// A warp's 32 rows of 64 bytes leave; rows and columns past the end are not written.
__device__ __forceinline__ void store_rows(const CUtensorMap* map, const uint8_t* src, int col, int row) {
  fence_proxy_async_smem();
  __syncwarp();
  if (elect_one()) {
    tma_store_2d(map, src, col, row);
    bulk_commit();
  }
  __syncwarp();
}

// Tile w: 128 tokens (fastest) and BN weight rows, each by the CTAs of a cluster
// that share k (split > 1: one tile per cluster).
template <int BN>
__global__ void __launch_bounds__(QR_THREADS, 1)
k_qlinear_rows(const __grid_constant__ CUtensorMap mX, const __grid_constant__ CUtensorMap mW,
               const __grid_constant__ CUtensorMap mY, const QlinArgs a) {
  using Cfg = QrCfg<BN>;
  constexpr int STAGES = Cfg::STAGES, NBUF = Cfg::NBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage_out = smem + STAGES * Cfg::STAGE;                       // [QR_EPI_WARPS][QR_OUT]
  float* slots = reinterpret_cast<float*>(stage_out + QR_EPI_WARPS * QR_OUT);   // [QR_SLOTS][QR_SLOT]
  uint64_t* full = reinterpret_cast<uint64_t*>(slots + QR_SLOTS * QR_SLOT);
  uint64_t* empty = full + STAGES;
  uint64_t* accfull = empty + STAGES;   // [NBUF]
  uint64_t* accfree = accfull + NBUF;   // [NBUF]
  uint64_t* sfull = accfree + NBUF;     // [QR_SLOTS] scales
  uint64_t* sfree = sfull + QR_SLOTS;
  uint64_t* mma_done = sfree + QR_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * STAGES + 2 * NBUF + 1 + 2 * QR_SLOTS) * 8 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = (a.T + 127) / 128, n_tiles = mt * ((a.n + BN - 1) / BN);
  const int walk0 = blockIdx.x / a.split, n_walk = gridDim.x / a.split;
  const int rank = a.split > 1 ? (int)cluster_rank() : 0;
  // this CTA's blocks of k
  const int kb0 = (int)((long long)a.kb * rank / a.split);
  const int KB = (int)((long long)a.kb * (rank + 1) / a.split) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accfree[b], QR_EPI_WARPS);
    }
    for (int j = 0; j < QR_SLOTS; ++j) {
      mbar_init(&sfull[j], 32);
      mbar_init(&sfree[j], QR_EPI_WARPS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == QR_MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == QR_PRODUCER && lane == 0) {
    tma_prefetch_desc(&mX);
    tma_prefetch_desc(&mW);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();   // operands and outputs belong to the stream order

  if (warp >= QR_EPI_WARPS) {
    if (warp == QR_PRODUCER) {
      // ------------------------------------------------------- TMA producer
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int w = walk0; w < n_tiles && ok; w += n_walk) {
        const int m0 = w % mt * 128, n0 = w / mt * BN;
        for (int kb = 0; kb < KB; ++kb) {
          ok = mbar_wait_warp(&empty[s], ph, abort_flag, a.status);   // the first round passes
          if (!ok) break;
          if (elect_one()) {
            uint8_t* st = smem + (size_t)s * Cfg::STAGE;
            const uint32_t bar = smem_u32(&full[s]);
            mbar_expect_tx(&full[s], Cfg::STAGE);
            tma_2d<1>(st, &mX, bar, (kb0 + kb) * 128, m0);
            tma_2d<1>(st + Cfg::A_BYTES, &mW, bar, (kb0 + kb) * 128, n0);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp == QR_SCALE) {
      // ------------------------------------------------------------- scales
      const int nblk = (a.n + Q_GROUP - 1) / Q_GROUP;
      int j = 0;
      uint32_t jph = 1;
      bool ok = true;
      for (int w = walk0; w < n_tiles && ok; w += n_walk) {
        const int m0 = w % mt * 128, nb0 = w / mt * (BN / Q_GROUP);
        const float* x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = a.xs + (size_t)min(m0 + i * 32 + lane, a.T - 1) * a.kb + kb0;
        const float* ws = a.Ws + (size_t)min(nb0 + (lane & 1), nblk - 1) * a.kb + kb0;
        for (int kb = 0; kb < KB; kb += 4) {
          ok = mbar_wait_warp(&sfree[j], jph, abort_flag, a.status);   // the first round passes
          if (!ok) break;
          float* slot = slots + j * QR_SLOT;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int k = min(kb + q, KB - 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) copy4_async(slot + (i * 32 + lane) * 4 + q, x[i] + k, true);
            if (lane < 2) copy4_async(slot + (128 + lane) * 4 + q, ws + k, true);
          }
          copies_arrive(&sfull[j]);
          if (++j == QR_SLOTS) {
            j = 0;
            jph ^= 1;
          }
        }
      }
      copies_wait_all();
    } else {
      // --------------------------------------------------------- MMA issuer
      if (elect_one()) {
        const uint32_t idesc = idesc_e4m3_f32(128, BN);
        const uint64_t desc0 = sdesc_k_sw128(smem_u32(smem));
        bool ok = true;
        int s = 0, b = 0;
        uint32_t ph = 0, bph = 1;        // phase of full[s]; of accfree[b] (free in the first round)
        for (int w = walk0; w < n_tiles && ok; w += n_walk) {
          for (int kb = 0; kb < KB; ++kb) {
            ok = mbar_wait(&full[s], ph, abort_flag, a.status) && mbar_wait(&accfree[b], bph, abort_flag, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = desc0 + (uint32_t)(s * (Cfg::STAGE / 16)), bd = ad + Cfg::A_BYTES / 16;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pair_mma<1, true>(tmem + (uint32_t)(b * BN), ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
            tc_commit(&accfull[b]);
            tc_commit(&empty[s]);
            b = (b + 1) & (NBUF - 1);
            if (!b) bph ^= 1;
            if (++s == STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        tc_commit(mma_done);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue
    // A thread has one token and a quarter of the tile's columns.
    constexpr int COLS = Cfg::COLS;
    const int quarter = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(quarter * COLS);
    const int blk = quarter * COLS / Q_GROUP;   // these columns' weight block, counted from the tile's first
    int b = 0, j = 0;
    uint32_t bph = 0, jph = 0;
    float sc[4];
        // the next four blocks' scales
    auto scales = [&]() -> bool {
      if (!mbar_wait_warp(&sfull[j], jph, abort_flag, a.status)) return false;
      const float4* slot = reinterpret_cast<const float4*>(slots + j * QR_SLOT);
      const float4 x = slot[row], u = slot[128 + blk];
      sc[0] = x.x * u.x, sc[1] = x.y * u.y, sc[2] = x.z * u.z, sc[3] = x.w * u.w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfree[j]);
      if (++j == QR_SLOTS) {
        j = 0;
        jph ^= 1;
      }
      return true;
    };
    // Left at once when a wait fails: going on to the end of a loop from the
    // middle would keep both sides' sums alive.
    auto run = [&]() {
      if (walk0 < n_tiles && !scales()) return;
      for (int w = walk0; w < n_tiles; w += n_walk) {
        const int t0 = w % mt * 128 + (warp & 3) * 32, n0 = w / mt * BN + quarter * COLS;
        uint64_t acc[COLS / 2];
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i) acc[i] = 0;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait_warp(&accfull[b], bph, abort_flag, a.status)) return;
          tc_fence_after();
          const uint32_t src = tlane + (uint32_t)(b * BN);
          const uint64_t u = pack2(sc[0], sc[0]);
#pragma unroll
          for (int c = 0; c < COLS; c += 16) {
            uint64_t v[8];
            tmem_get16x2(src + c, v);
            if (c == COLS - 16) {   // all read: the next MMAs may have the columns
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&accfree[b]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[c / 2 + i] = fma2(v[i], u, acc[c / 2 + i]);
          }
          b = (b + 1) & (NBUF - 1);
          if (!b) bph ^= 1;
#pragma unroll
          for (int q = 0; q < 3; ++q) sc[q] = sc[q + 1];
          if (kb + 1 == KB ? w + n_walk < n_tiles : (kb & 3) == 3)
            if (!scales()) return;
        }
        if (BN == 128 && a.split > 1) {
          // This warp saw the CTA's last block: all copies and MMAs have
          // completed, and the ring holds the sums now.
          float* ex = reinterpret_cast<float*>(smem);   // [128 columns][128 rows]
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) {
            float u, v;
            unpack2(acc[i], u, v);
            ex[(quarter * COLS + 2 * i) * 128 + row] = u;
            ex[(quarter * COLS + 2 * i + 1) * 128 + row] = v;
          }
          return;
        }
        uint8_t* out = stage_out + warp * QR_OUT;
        const int step = a.y_f32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < COLS; c += 16) {
          if ((c & (step - 1)) == 0 && n0 + c < a.n && t0 < a.T) {
            if (elect_one()) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // 16 bytes each, in the copy's 64-byte swizzle
              uint8_t* to = out + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16;
              if (a.y_f32) {
                float4 f;
                unpack2(acc[c / 2 + 2 * i], f.x, f.y);
                unpack2(acc[c / 2 + 2 * i + 1], f.z, f.w);
                *reinterpret_cast<float4*>(to) = f;
              } else if ((c & 31) == 0) {
                float f[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) unpack2(acc[(c & ~31) / 2 + 4 * i + q], f[2 * q], f[2 * q + 1]);
                store8_bf16(to, 0, f);
              }
            }
            store_rows(&mY, out, n0 + c, t0);
          }
        }
      }
    };
    run();
    __syncwarp();
    if (elect_one()) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  if (BN == 128 && a.split > 1) {
    spread_abort(abort_flag, a.split);
    cluster_sync();   // every CTA's sums are in its ring
    // CTA `rank` adds up and stores its part of every warp's 32 columns
    const int each = 32 / a.split, c0 = (warp >> 2) * 32 + rank * each;
    const int row = (warp & 3) * 32 + lane, t = walk0 % mt * 128 + row, n0 = walk0 / mt * BN + c0;
    if (warp < QR_EPI_WARPS && t < a.T && !*abort_flag)
      for (int c = 0; c < each; c += 4) {
        if (n0 + c >= a.n) break;       // n is a multiple of 8
        float v[4];
        cluster_sums<4>(smem_u32(smem) + (uint32_t)((c0 + c) * 128 + row) * 4, 512, a.split, v);
        const size_t at = ((size_t)t * a.n + n0 + c) / 4;
        if (a.y_f32) reinterpret_cast<float4*>(a.y)[at] = make_float4(v[0], v[1], v[2], v[3]);
        else reinterpret_cast<uint2*>(a.y)[at] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      }
    __syncwarp();
    cluster_sync();   // nobody leaves while its sums are read
  }
  __syncthreads();
  if (*abort_flag) drain_copies();
  if (warp == QR_MMA) {
    mbar_drain(mma_done, 0, a.status);   // every MMA is complete before TMEM is freed
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace sffn
