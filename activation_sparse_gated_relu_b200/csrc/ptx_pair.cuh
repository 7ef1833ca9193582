// PTX wrappers for CTA pairs (clusters of two whose tcgen05.mma spans both
// SMs) next to the one-CTA forms of ptx.cuh.  CTAS is 1 or 2; with 1 each
// wrapper is the one-CTA instruction.  No load here is a multicast.
#pragma once

#include "ptx.cuh"

namespace sffn {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared-memory address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Every thread of the cluster arrives and waits.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrivals on a barrier given by its cluster address.  What they order is
// read and written by copies and MMAs; mbar_release_cluster is for the writes
// of threads.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_release_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void mbar_expect_cluster(uint32_t addr, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(addr), "r"(bytes) : "memory");
}
// True in one lane of a converged warp.  Copies and MMAs take their operands
// from uniform registers; behind this predicate (rather than a lane number)
// the compiler knows that a single lane is active and needs no loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p)::"memory");
  return p != 0;
}
// mbar_wait of a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                               uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, status));
}
// mbar_wait for a phase that threads of another CTA of the cluster arrived on
// with mbar_release_cluster: what they wrote is seen.  The acquire is a second
// look at the phase, which is complete by then and stays until the caller hands
// its stage back; a wait that acquires at cluster scope at every try is slow.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                  uint32_t* status) {
  if (!mbar_wait(bar, parity, abort_flag, status)) return false;
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Where a wait failed in this CTA, the other CTAs of its cluster learn of it.  By
// every warp before the cluster barrier behind which they use each other's
// results, so that behind it all of them find the flag set, or none.  (A wait
// takes seconds to fail: every CTA has cleared its flag long before.)
__device__ __forceinline__ void spread_abort(volatile int* abort_flag, int n_ctas) {
  if (__any_sync(0xFFFFFFFFu, *abort_flag)) {
    const uint32_t at = smem_u32(const_cast<const int*>(abort_flag));
    for (int r = 0; r < n_ctas; ++r)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(at, (uint32_t)r)), "r"(1) : "memory");
  }
  __syncwarp();
}
// What a CTA that leaves, TMEM freed, must not have under way, also where a wait
// has failed in any of its roles: MMAs (`bar` is committed to behind the last of
// them; a bounded wait that goes on where another has failed) ...
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity, uint32_t* status) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > SFFN_WAIT_LIMIT_NS) {
      atomicOr(status, DEV_ERR_TIMEOUT);
      break;
    }
  }
}
// ... and copies.  Their barriers may be another CTA's, or half-armed, so this
// waits many times as long as any copy takes.
__device__ __forceinline__ void drain_copies() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000ull) __nanosleep(1000);
}

// Four bytes from global to shared memory, asynchronously; zero where `in` is false.
__device__ __forceinline__ void copy4_async(void* dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
// Groups of this thread's copies, and the wait until at most N are under way.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// One arrival on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Tiled loads into this CTA's shared memory; `bar` is a cluster address, with
// a pair possibly in the other CTA.  c0 · element size is a multiple of 16.
template <int CTAS>
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  if (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  if (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Tiled store from shared memory (a bulk group of the issuing thread); what
// lies outside the map is not written.  c0 >= 0, c0 · element size a multiple of 16.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}

template <int CTAS>
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  if (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  }
}
template <int CTAS>
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if (CTAS == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
  else
    tmem_dealloc(taddr, ncols);
}
// D (+)= A · B^T; kind::f16 (bf16 operands) or kind::f8f6f4 (e4m3 operands), fp32 D.
template <int CTAS, bool F8>
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
#define SFFN_PAIR_MMA(group, kind)                                                              \
  asm volatile(                                                                                 \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                         \
      "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)                                       \
      : "memory")
  if (CTAS == 2 && F8) SFFN_PAIR_MMA("2", "f8f6f4");
  else if (CTAS == 2) SFFN_PAIR_MMA("2", "f16");
  else if (F8) SFFN_PAIR_MMA("1", "f8f6f4");
  else SFFN_PAIR_MMA("1", "f16");
#undef SFFN_PAIR_MMA
}
// Arrive on `bar` (with a pair: on that barrier in both CTAs) once the MMAs
// issued so far are complete.
template <int CTAS>
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  if (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    tc_commit(bar);
}

// 16 or 32 consecutive fp32 columns of this warp's TMEM lanes, one lane per
// thread.  Load and wait are one statement, so that no use of the values can
// come before the wait and no copies are made around it.
__device__ __forceinline__ void tmem_get16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_get32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
      "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
        "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
        "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
        "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}

// 16 columns as eight pairs, for the two-lane arithmetic below.
__device__ __forceinline__ void tmem_get16x2(uint32_t taddr, uint64_t (&v)[8]) {
  asm volatile(
      "{\n\t.reg .b32 r<16>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {r0,r1,r2,r3,r4,r5,r6,r7,r8,r9,r10,r11,r12,r13,r14,r15}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {r0, r1};\n\t"
      "mov.b64 %1, {r2, r3};\n\t"
      "mov.b64 %2, {r4, r5};\n\t"
      "mov.b64 %3, {r6, r7};\n\t"
      "mov.b64 %4, {r8, r9};\n\t"
      "mov.b64 %5, {r10, r11};\n\t"
      "mov.b64 %6, {r12, r13};\n\t"
      "mov.b64 %7, {r14, r15};\n\t"
      "}"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]), "=l"(v[7])
      : "r"(taddr)
      : "memory");
}
// Two fp32 values in a register pair: one multiply-add instruction for both.
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Shared-memory descriptor of an MN-major operand staged by TMA with
// SWIZZLE_128B: rows of 64 values along M or N (128 bytes), one row per k;
// 8-row groups 1024 bytes apart, the next 64 values of M or N `chunk` bytes
// further.  Stepping K by 16 adds 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t chunk) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(chunk >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// v[q] = the sum over the cluster's CTAs, in order, of their shared memory's
// float at addr + q · step.  All loads go out before the first sum.
template <int N>
__device__ __forceinline__ void cluster_sums(uint32_t addr, uint32_t step, int split, float (&v)[N]) {
  float u[8][N];
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < split) {
      const uint32_t from = cluster_addr(addr, (uint32_t)r);
#pragma unroll
      for (int q = 0; q < N; ++q)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u[r][q]) : "r"(from + (uint32_t)q * step) : "memory");
    }
#pragma unroll
  for (int q = 0; q < N; ++q) v[q] = 0.0f;
#pragma unroll
  for (int r = 0; r < 8; ++r)
    if (r < split)
#pragma unroll
      for (int q = 0; q < N; ++q) v[q] += u[r][q];
}

}  // namespace sffn
