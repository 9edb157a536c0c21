// Device-side building blocks of kernels that run on CTA pairs (tcgen05 cta_group::2): one
// 256-row tensor-core tile over two SMs, each SM holding half of either operand.
#pragma once

#include <cuda.h>

#include "mx_device.cuh"

namespace fs4 {

// Like mbar_try_wait / mbar_wait, for barriers that threads of the other CTA arrive on.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* status, volatile int* abort) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (*abort) return false;
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      *abort = 1;
      return false;
    }
  }
}

// Arrive on a barrier given by its cluster address (cluster_map), to hand TMEM back: the tcgen05
// fences order the accesses and no memory is published, so the release stays at the default
// (CTA) scope.  At cluster scope it takes about 1200 cycles.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// A producer that gives up (a wait of its ran out) may have issued fewer or more stages than the
// other CTA's.  The leader's barriers count the copies of both, so each says how far it got:
// CTA 1 tells the leader before they meet, and the leader expects and awaits what CTA 1 issued
// alone, before either may leave.  `stage` is the bytes of one CTA's part of a stage.
__device__ __forceinline__ void tell_issued(uint32_t* slot, uint32_t issued) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_map(smem_addr(slot), 0)), "r"(issued) : "memory");
}
__device__ __forceinline__ void await_issued(uint64_t* full, uint32_t stages, uint32_t stage, uint32_t own, uint32_t other, uint32_t* status) {
  for (uint32_t i = own; i < other; ++i) {
    volatile int never = 0;
    mbar_arrive_expect_tx(&full[i % stages], stage);
    if (!mbar_wait_cluster(&full[i % stages], (i / stages) & 1u, status, &never)) break;
  }
}
// The leader's own stages, before that.  A stage that CTA 1 did not issue never completes: its wait
// runs out, and the copies of later stages had that time to land.
__device__ __forceinline__ void await_own(uint64_t* full, uint32_t stages, uint32_t issued, uint32_t* status) {
  for (uint32_t i = issued > stages ? issued - stages : 0u; i < issued; ++i) {
    volatile int never = 0;
    if (!mbar_wait(&full[i % stages], (i / stages) & 1u, status, &never)) break;
  }
}

// Copy of `rows` (the map's box) 128-byte rows from row `row` on to this CTA's shared memory; the
// bytes are counted on `bar`, a cluster address in either CTA of the pair.  x is always 0.
__device__ __forceinline__ void tma_rows_pair(uint32_t dst, const CUtensorMap* map, int32_t row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(0), "r"(row)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Arrive on the barrier at this address in both CTAs once every tcgen05 operation this thread
// issued so far has completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// FP16 operands: instruction descriptor (kind::f16, FP32 accumulate, M x N; a_mn / b_mn: the
// operand's M or N index runs fastest in shared memory) ...
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// ... the MMA of a CTA pair (K = 16) ...
__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// ... and the descriptor of an operand with the M or N index fastest: 128-byte swizzled rows of
// 64 elements, one row per k, 8-row groups 1024 bytes apart; the next 64 elements of M or N
// start `next64` bytes on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t next64) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(next64 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// MXFP4 operands: scale atoms to both CTAs' TMEM, each from its own shared memory ...
__device__ __forceinline__ void tc_copy_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// ... the arrival of a thread's tcgen05 operations on one barrier of this CTA ...
__device__ __forceinline__ void tc_commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// ... and the MMA of a CTA pair (K = 64).
__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa_tmem,
                                                 uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// ------------------------------------------------------------------ 32-byte global accesses
struct Pair {
  uint32_t w[8];
};
// Loads bypass L1: the data may have been written by other SMs earlier in the launch.
__device__ __forceinline__ Pair load_pair(const void* p) {
  Pair r;
  asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void store_pair(void* p, const Pair& r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3]),
               "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

// Transpose a warp's 32 x 32 words: v[i] of lane l becomes v[l] of lane i.
__device__ __forceinline__ void turn32(uint32_t* v, int lane) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & s) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, (lane & s) ? v[i] : v[i + s], s);
      if (lane & s) v[i] = got;
      else v[i + s] = got;
    }
  }
}

}  // namespace fs4
