// Products grouped by expert with ragged groups: expert e owns the rows
// off[e] .. off[e+1] of x.  With W [E][n][k],
//
//   forward   y[r]  = W[e] x[r]
//   input     dx[r] = W[e]^T dy[r]
//   weight    dW[e] = sum_{r in e} dy[r] x[r]^T
//
// bf16 operands, fp32 sums.  All three are one tile kernel, D[m][c] = sum_k
// A[m][k] B[c][k] on the tensor cores, with the weight side as the MMA's rows m
// (128 TMEM lanes per CTA) and the ragged side as its columns c:
//
//             m          c               k               A            B
//   forward   n          e's rows        k               W, K-major   x, K-major
//   input     k          e's rows        n               W, M-major   dy, K-major
//   weight    k          n               e's rows        x, M-major   dy, N-major
//
// so that a group costs columns rounded up to 16 or 32, not to 128 rows, and
// an M- or N-major operand is read as it lies, without a transposed copy.  D's
// column c is a row of the output and its lanes are consecutive there, so
// every store of a warp is one run of 32 values.
//
// Persistent CTAs (or CTA pairs: 256 rows, each CTA holding half of the
// columns' operand) walk the tiles of all experts; two accumulators in TMEM
// let the MMAs of a tile run beside the stores of the tile before.
//
// With many rows the tensor cores bound it: 8192 rows in 8 groups, 2048 to 8192,
// forward 194 to 203 us (1.4 PFLOP/s, where the power limit holds the clock at about
// 1.5 GHz), input gradient 200 to 208; the weight gradient, whose 537 MB leave beside
// the MMAs, 260 (207 without its stores).  One shape of tile serves all groups of a
// call, and rows that are no multiple of 128 bytes cross lines: 4426 rows in 19
// groups of 85 to 856, forward, 1152 to 2304 31 us, 1192 to 2360 47.  With few rows the weights' bytes do: 16
// rows in 8 groups, 4096 to 14336, 128 us (6.4 TB/s).  There a tile is 32 columns
// and 128 rows m, and where tiles are fewer than SMs a cluster shares each tile's
// k and adds the parts up through distributed shared memory, in a fixed order.
#pragma once

#include "ptx_pair.cuh"
#include "vec8.cuh"

namespace sffn {

enum { GROUPED_FWD = 0, GROUPED_DX = 1, GROUPED_DW = 2 };
constexpr int GROUPED_MAX_E = 1024;
constexpr int GT_EPI_WARPS = 8;                        // two warpgroups, every other 32 columns each
constexpr int GT_PRODUCER = GT_EPI_WARPS;
constexpr int GT_FIX = GT_EPI_WARPS + 1;              // clears what lies behind a group's end (weight gradient)
constexpr int GT_MMA = GT_EPI_WARPS + 2;
constexpr int GT_THREADS = (GT_EPI_WARPS + 3) * 32;
constexpr int GT_BK = 64;                              // bf16 values of k per stage
constexpr int GT_SMEM = 227 * 1024;

// BN: columns per tile.
template <int CTAS, int BN>
struct GtCfg {
  static constexpr int B_ROWS = BN / CTAS;             // columns whose operand a CTA holds
  static constexpr int A_BYTES = 128 * GT_BK * 2;
  static constexpr int B_BYTES = B_ROWS * GT_BK * 2;
  static constexpr int BOX = BN >= 128 ? 64 : 32;      // columns per copy
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int TABLE = (3 * (GROUPED_MAX_E + 1) * 4 + 127) & ~127;
  static constexpr int FIXED = 1024 /*align*/ + 384 /*barriers*/ + TABLE;
  static constexpr int RAW = (GT_SMEM - FIXED) / STAGE;
  static constexpr int STAGES = RAW > 10 ? 10 : RAW;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
};

struct GroupedArgs {
  const int* off;       // [E + 1]
  void* out;
  int E, R;
  int M, N, K;          // rows m; columns c (weight gradient); inner size k (forward and input gradient)
  int out_f32;
  int split;            // 32 columns: CTAs of a cluster, each with a part of k; one tile per cluster then
  int kchunk;           // k blocks that the tensor core adds up before they join the fp32 sum in registers
  uint32_t* status;
};

// Group e's rows [a, b), clamped to [0, R]; false if the offsets are out of
// range or run backwards (the group is then what the clamping leaves).
__device__ __forceinline__ bool group_rows(const int* off, int e, int R, int* a, int* b) {
  const int u = off[e], v = off[e + 1];
  *a = min(max(u, 0), R);
  *b = max(min(max(v, 0), R), *a);
  return u >= 0 && v >= u && v <= R;
}

// a / b and the remainder, a >= 0, b > 0.  Every role of a CTA does this between
// two tiles; an integer division there takes several times as long.
__device__ __forceinline__ int div_rem(int a, int b, int* rem) {
  int q = (int)((float)a * __frcp_rn((float)b));   // off by one step or two at most for a / b < 2^21
  int r = a - q * b;
  while (r < 0) {
    --q;
    r += b;
  }
  while (r >= b) {
    ++q;
    r -= b;
  }
  *rem = r;
  return q;
}

// The tiles of all experts in order, one role's walk over them.
template <int MODE, int CTAS, int BN>
struct GtWalk {
  const int *ra, *rb, *first;   // group rows, first tile of each expert ([E] the total)
  int M, N, K, e;
  int split, rank;              // this CTA's part of k
  // the current tile
  int m0;                       // first row m of the tile (of the pair)
  int c0, cols, bn;             // first column, columns stored, columns computed
  int krow;                     // weight gradient: first row of the group
  int kb0, kbs, ktail;          // first k block, k blocks, and values in the last one
  size_t orow;                  // output row of column 0

  __device__ __forceinline__ void set(int w) {
    while (w >= first[e + 1]) ++e;
    const int t = w - first[e], a = ra[e], rows = rb[e] - a;
    constexpr int STEP = 16 * CTAS;
    if (MODE == GROUPED_DW) {
      const int nt = (N + BN - 1) / BN;
      int j;
      m0 = div_rem(t, nt, &j) * (128 * CTAS);
      c0 = j * BN;
      cols = min(BN, N - c0);
      krow = a;
      kbs = (rows + GT_BK - 1) / GT_BK;
      ktail = rows - (kbs - 1) * GT_BK;
      orow = (size_t)e * N + c0;
    } else {
      // the fewest tiles of at most BN columns, even ones
      const int nt = (rows + BN - 1) / BN;
      int j;
      const int each = (div_rem(rows + nt - 1, nt, &j) + STEP - 1) / STEP * STEP;
      m0 = div_rem(t, nt, &j) * (128 * CTAS);
      c0 = a + j * each;
      cols = min(each, a + rows - c0);
      kbs = (K + GT_BK - 1) / GT_BK;
      ktail = K - (kbs - 1) * GT_BK;
      orow = (size_t)c0;
    }
    bn = (cols + STEP - 1) / STEP * STEP;
    kb0 = 0;
    if (BN == 32 && split > 1) {
      const int all = kbs;
      kb0 = all * rank / split;
      kbs = all * (rank + 1) / split - kb0;
      if (rank + 1 < split) ktail = GT_BK;
    }
  }
};

template <int MODE, int CTAS, int BN>
__global__ void __launch_bounds__(GT_THREADS, 1)
k_grouped(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
          const GroupedArgs args) {
  using Cfg = GtCfg<CTAS, BN>;
  using Walk = GtWalk<MODE, CTAS, BN>;
  constexpr int STAGES = Cfg::STAGES;
  constexpr uint32_t NCOLS = BN <= 16 ? 32 : 2 * BN;     // two accumulators, a power of two of at least 32
  constexpr bool A_MN = MODE != GROUPED_FWD, B_MN = MODE == GROUPED_DW;
  constexpr int BOX = Cfg::BOX;
  static_assert(NCOLS <= 512 && (NCOLS & (NCOLS - 1)) == 0, "TMEM columns");
  static_assert(!B_MN || Cfg::B_ROWS % 64 == 0, "N-major columns come in boxes of 64");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * Cfg::STAGE);
  uint64_t* empty = full + STAGES;
  uint64_t* accfull = empty + STAGES;   // [2]
  uint64_t* accfree = accfull + 2;      // [2]
  uint64_t* tailbar = accfree + 2;      // [STAGES] a group's last block has landed, not yet cleared
  uint64_t* mma_done = tailbar + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((3 * STAGES + 5) * 8 + 8 <= 384, "barrier area");
  int* ra = reinterpret_cast<int*>(smem + STAGES * Cfg::STAGE + 384);
  int* rb = ra + GROUPED_MAX_E + 1;
  int* first = rb + GROUPED_MAX_E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0u;
  const int split = BN == 32 ? args.split : 1;
  const int n_walk = gridDim.x / (CTAS * split), walk0 = blockIdx.x / (CTAS * split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], CTAS);        // one arrival per CTA's producer
      mbar_init(&empty[s], 1);
      mbar_init(&tailbar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accfree[b], GT_EPI_WARPS * CTAS);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == GT_MMA) pair_tmem_alloc<CTAS>(tmem_slot, NCOLS);
  if (warp == GT_PRODUCER && lane == 0) {
    tma_prefetch_desc(&mA);
    tma_prefetch_desc(&mB);
  }
  griddep_wait();   // offsets, operands and outputs belong to the stream order
  for (int e = threadIdx.x; e < args.E; e += GT_THREADS) {
    if (!group_rows(args.off, e, args.R, &ra[e], &rb[e]) && blockIdx.x == 0) atomicOr(args.status, DEV_ERR_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {   // first tile of each expert: a running sum over experts, 32 at a time
    const int mt = (args.M + 128 * CTAS - 1) / (128 * CTAS);
    int base = 0, end = 0;
    for (int e0 = 0; e0 < args.E; e0 += 32) {
      const int e = e0 + lane;
      // A group starts no earlier than any before it ends: with offsets that run
      // back and forth the rows, and so the tiles, would count many times.
      const int b = e < args.E ? rb[e] : 0;
      int last = b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, last, o);
        if (lane >= o) last = max(last, u);
      }
      last = max(last, end);
      int before = __shfl_up_sync(0xFFFFFFFFu, last, 1);
      if (lane == 0) before = end;
      end = __shfl_sync(0xFFFFFFFFu, last, 31);
      int n = 0;
      if (e < args.E) {
        ra[e] = max(ra[e], before);
        rb[e] = max(b, ra[e]);
        n = mt * (MODE == GROUPED_DW ? (args.N + BN - 1) / BN : (rb[e] - ra[e] + BN - 1) / BN);
      }
      int s = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
      }
      if (e < args.E) first[e] = base + s - n;
      base += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) first[args.E] = base;
  }
  if (CTAS == 2) cluster_sync();   // the barriers of both CTAs are ready
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = first[args.E];
  Walk t;
  t.ra = ra;
  t.rb = rb;
  t.first = first;
  t.M = args.M;
  t.N = args.N;
  t.K = args.K;
  t.e = 0;
  t.split = split;
  t.rank = split > 1 ? (int)cluster_rank() : 0;

  if (warp == GT_PRODUCER) {
    // --------------------------------------------------------- TMA producer
    int it = 0;
    bool ok = true;
    for (int w = walk0; w < n_tiles && ok; w += n_walk) {
      t.set(w);
      const int m0 = t.m0 + (int)rank * 128;
      const int half = t.bn / CTAS, b0 = t.c0 + (int)rank * half, nbox = (half + BOX - 1) / BOX;   // this CTA's columns
      const uint32_t bytes = Cfg::A_BYTES + nbox * (BOX * GT_BK * 2);
      for (int kb = 0; kb < t.kbs; ++kb, ++it) {
        const int s = it % STAGES, f = it / STAGES;
        if (f > 0) ok = mbar_wait_warp(&empty[s], (f - 1) & 1, abort_flag, args.status);
        if (!ok) break;
        uint8_t* sa = smem + (size_t)s * Cfg::STAGE;
        uint8_t* sb = sa + Cfg::A_BYTES;
        const bool tail = B_MN && kb == t.kbs - 1 && (t.ktail & 15);
        const uint32_t leader_full = CTAS == 2 ? cluster_addr(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
        if (elect_one()) {
          const uint32_t bar = tail ? smem_u32(&tailbar[s]) : leader_full;
          if (tail) mbar_expect_tx(&tailbar[s], bytes);
          else if (CTAS == 2) mbar_expect_cluster(bar, bytes);
          else mbar_expect_tx(&full[s], bytes);
          const int k0 = (t.kb0 + kb) * GT_BK;
          if (MODE == GROUPED_FWD) {
            tma_3d<CTAS>(sa, &mA, bar, k0, m0, t.e);
          } else if (MODE == GROUPED_DX) {
            tma_3d<CTAS>(sa, &mA, bar, m0, k0, t.e);
            tma_3d<CTAS>(sa + 8192, &mA, bar, m0 + 64, k0, t.e);
          } else {
            tma_2d<CTAS>(sa, &mA, bar, m0, t.krow + k0);
            tma_2d<CTAS>(sa + 8192, &mA, bar, m0 + 64, t.krow + k0);
          }
          for (int i = 0; i < nbox; ++i) {
            uint8_t* dst = sb + i * (BOX * GT_BK * 2);
            if (B_MN) tma_2d<CTAS>(dst, &mB, bar, b0 + BOX * i, t.krow + k0);
            else tma_2d<CTAS>(dst, &mB, bar, k0, b0 + BOX * i);
          }
        }
      }
    }
  } else if (warp == GT_FIX) {
    // --------------------------------------------------- weight gradient only
    // The last MMA of a group takes k up to the next multiple of 16: what lies
    // there belongs to other groups and may hold anything, so both operands
    // are cleared from ktail on before the MMA warp sees the stage.
    int it = 0;
    uint32_t used = 0;                  // parity of tailbar[s] in bit s
    for (int w = walk0; B_MN && w < n_tiles; w += n_walk) {
      t.set(w);
      it += t.kbs;
      if (t.kbs == 0 || !(t.ktail & 15)) continue;
      const int s = (it - 1) % STAGES;
      if (!mbar_wait_warp(&tailbar[s], (used >> s) & 1, abort_flag, args.status)) break;
      used ^= 1u << s;
      uint8_t* sa = smem + (size_t)s * Cfg::STAGE;
      uint8_t* sb = sa + Cfg::A_BYTES;
      const int nbox = (t.bn / CTAS + 63) / 64;
      const int k1 = (t.ktail + 15) & ~15;
      for (int i = lane; i < (k1 - t.ktail) * 8; i += 32) {
        const int at = t.ktail * 128 + i * 16;   // whole rows of 128 bytes: the swizzle permutes within a row
        for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4*>(sa + c * 8192 + at) = make_uint4(0, 0, 0, 0);
        for (int c = 0; c < nbox; ++c) *reinterpret_cast<uint4*>(sb + c * 8192 + at) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 2) mbar_release_cluster(cluster_addr(smem_u32(&full[s]), 0));
        else mbar_arrive(&full[s]);
      }
    }
  } else if (warp == GT_MMA) {
    // ----------------------------------------------------------- MMA issuer
    // One thread (of the pair's first CTA).
    if (rank == 0 && elect_one()) {
      const uint32_t sa0 = smem_u32(smem), sb0 = sa0 + Cfg::A_BYTES;
      const uint64_t ad0 = A_MN ? sdesc_mn_sw128(sa0, 8192) : sdesc_k_sw128(sa0);
      const uint64_t bd0 = B_MN ? sdesc_mn_sw128(sb0, 8192) : sdesc_k_sw128(sb0);
      constexpr uint32_t AK = A_MN ? 128u : 2u, BK = B_MN ? 128u : 2u;   // 16 values of k further
      int s = 0, b = 0;
      uint32_t ph = 0, bph = 1;          // phase of full[s]; of accfree[b] (free in the first round)
      bool ok = true;
      for (int w = walk0; w < n_tiles && ok; w += n_walk) {
        t.set(w);
        const uint32_t idesc = idesc_bf16_f32(128 * CTAS, t.bn) | ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16);
        for (int kc = 0; kc < t.kbs && ok; kc += args.kchunk) {
          ok = mbar_wait(&accfree[b], bph, abort_flag, args.status);
          if (!ok) break;
          const uint32_t d = tmem + (uint32_t)(b * BN);
          const int k1 = min(kc + args.kchunk, t.kbs);
          for (int kb = kc; kb < k1; ++kb) {
            // a block that the other CTA's threads cleared has to be seen as they left it
            ok = CTAS == 2 && B_MN && kb == t.kbs - 1 && (t.ktail & 15)
                     ? mbar_wait_cluster(&full[s], ph, abort_flag, args.status)
                     : mbar_wait(&full[s], ph, abort_flag, args.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = ad0 + (uint32_t)(s * (Cfg::STAGE / 16)), bd = bd0 + (uint32_t)(s * (Cfg::STAGE / 16));
            const int nk = kb == t.kbs - 1 ? (t.ktail + 15) / 16 : GT_BK / 16;
#pragma unroll
            for (int k = 0; k < GT_BK / 16; ++k)
              if (k < nk) pair_mma<CTAS, false>(d, ad + AK * k, bd + BK * k, idesc, (kb == kc && k == 0) ? 0u : 1u);
            pair_commit<CTAS>(&empty[s]);
            if (++s == STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
          if (ok) pair_commit<CTAS>(&accfull[b]);
          b ^= 1;
          if (!b) bph ^= 1;
        }
      }
      pair_commit<CTAS>(mma_done);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue
    constexpr int NCH = (BN + 63) / 64;   // 32-column pieces per warpgroup
    const int wg = warp >> 2;
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (BN >= 64 ? 32u * wg : 0u);
    const uint32_t free0 = CTAS == 2 ? cluster_addr(smem_u32(&accfree[0]), 0) : smem_u32(&accfree[0]);
    int ci = 0;
    // this warp has read accumulator b: the MMAs may refill it
    auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 2) mbar_arrive_cluster(free0 + 8 * b);
        else mbar_arrive(&accfree[b]);
      }
    };
    // columns c .. c + 31 of the tile, this thread's row m; by whole warps
    auto store = [&](const float (&v)[32], int c) {
      const int m = t.m0 + (int)rank * 128 + (warp & 3) * 32 + lane;
      const int n = m < t.M ? t.cols - c : 0;   // M is a multiple of 8: both lanes of a pair store, or neither
      if (args.out_f32) {
        float* o = reinterpret_cast<float*>(args.out) + (t.orow + c) * (size_t)t.M + m;
        if (n >= 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i, o += t.M) *o = v[i];
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i, o += t.M)
            if (i < n) *o = v[i];
        }
      } else {
        // two columns at a time: even lanes store two rows m of the first one,
        // odd lanes of the second
        const int odd = lane & 1;
        const uint32_t sel = odd ? 0x3276u : 0x5410u;
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(args.out) + (t.orow + c + odd) * (size_t)t.M + (m - odd);
#pragma unroll
        for (int i = 0; i < 32; i += 2, o += 2 * (size_t)t.M) {
          const uint32_t p = pack_bf16(v[i], v[i + 1]);
          const uint32_t q = __shfl_xor_sync(0xFFFFFFFFu, p, 1);
          if (i + odd < n) *reinterpret_cast<uint32_t*>(o) = __byte_perm(p, q, sel);
        }
      }
    };
    // k shared by a cluster: this CTA's sums into the ring's memory, which the
    // tile's last accumulator shows to be free
    auto put = [&](const float (&v)[32]) {
      float* ex = reinterpret_cast<float*>(smem) + (warp & 3) * 32 + lane;   // [32 columns][128 rows]
#pragma unroll
      for (int i = 0; i < 32; ++i) ex[i * 128] = v[i];
    };
    // Left at once when a wait fails: leaving a loop from its middle would keep
    // both sides' sums alive, a select for each of them.
    auto run = [&]() {
      for (int w = walk0; w < n_tiles; w += n_walk) {
        t.set(w);
        const int pieces = (t.cols - 32 * wg + 63) / 64;   // this warpgroup's, possibly none
        if (t.kbs <= args.kchunk) {
          // one sum in TMEM: from there to the output, a piece at a time
          if (MODE == GROUPED_DW && t.kbs == 0) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
#pragma unroll 1
            for (int j = 0; j < pieces; ++j) {
              store(v, 64 * j + 32 * wg);
              __syncwarp();
            }
            continue;
          }
          const int b = ci & 1;
          if (!mbar_wait_warp(&accfull[b], (uint32_t)((ci >> 1) & 1), abort_flag, args.status)) return;
          ++ci;
          tc_fence_after();
          if (pieces <= 0) release(b);
#pragma unroll 1
          for (int j = 0; j < pieces; ++j) {
            float v[32];
            tmem_get32(tlane + (uint32_t)(b * BN + 64 * j), v);
            if (j == pieces - 1) release(b);
            if (BN == 32 && split > 1) put(v);
            else store(v, 64 * j + 32 * wg);
            __syncwarp();
          }
        } else {
          // several: added up in registers, all of the tile's columns, computed
          // or not (what the others hold is never stored, and a test would cost
          // a select per value)
          float acc[NCH][32];
#pragma unroll
          for (int j = 0; j < NCH; ++j)
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[j][i] = 0.0f;
          for (int kc = 0; kc < t.kbs; kc += args.kchunk, ++ci) {
            const int b = ci & 1;
            if (!mbar_wait_warp(&accfull[b], (uint32_t)((ci >> 1) & 1), abort_flag, args.status)) return;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < NCH; ++j)
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                float v[16];
                tmem_get16(tlane + (uint32_t)(b * BN + 64 * j + h), v);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][h + i] += v[i];
              }
            release(b);
          }
#pragma unroll
          for (int j = 0; j < NCH; ++j)
            if (j < pieces) {
              if (BN == 32 && split > 1) put(acc[j]);
              else store(acc[j], 64 * j + 32 * wg);
              __syncwarp();
            }
        }
      }
    };
    run();
  }
  __syncwarp();
  tc_fence_before();
  if (BN == 32 && split > 1) {
    spread_abort(abort_flag, split);
    cluster_sync();   // every CTA's sums are in its ring
    if (walk0 < n_tiles && warp < GT_EPI_WARPS) {
      // CTA `rank` adds up and stores every split-th column
      t.set(walk0);
      const int row = threadIdx.x & 127, m = t.m0 + row, step = 2 * split;
      if (m < t.M && !*abort_flag)
        for (int c = t.rank + split * (threadIdx.x >> 7); c < t.cols; c += 4 * step) {   // reads on to column 31 + 48
          float v[4];
          cluster_sums<4>(smem_u32(smem) + (uint32_t)(c * 128 + row) * 4, (uint32_t)step * 512, split, v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const size_t at = (t.orow + c + step * q) * (size_t)t.M + m;
            if (c + step * q >= t.cols) break;
            if (args.out_f32) reinterpret_cast<float*>(args.out)[at] = v[q];
            else reinterpret_cast<__nv_bfloat16*>(args.out)[at] = __float2bfloat16(v[q]);
          }
        }
    }
    __syncwarp();
    cluster_sync();   // nobody leaves while its sums are read
  }
  __syncthreads();
  // every MMA of this CTA (pair) is complete before TMEM is freed
  if (warp == GT_MMA) mbar_drain(mma_done, 0, args.status);
  __syncwarp();
  if (CTAS == 2) {   // neither CTA leaves while the other may still signal or read it
    spread_abort(abort_flag, 2);
    cluster_sync();
  }
  if (*abort_flag) {
    drain_copies();
    if (CTAS == 2) cluster_sync();
  }
  if (warp == GT_MMA) {
    tc_fence_after();
    pair_tmem_dealloc<CTAS>(tmem, NCOLS);
  }
}

}  // namespace sffn
