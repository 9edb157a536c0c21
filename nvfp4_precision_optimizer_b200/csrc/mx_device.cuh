// Device-side building blocks of the MXFP4 kernels: the E8M0 block scale, its TILED
// placement and the random stream.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs4_device.cuh"

namespace fs4 {

// Scale byte of a block from the largest |x|'s float bits.  The exponent field of amax is
// floor(log2 amax) + 127, so the floor rule's byte is that field less 2; the ceil rule adds
// 1 where the significand passes 1.5 (6 = 1.5 2^2).  A subnormal amax has field 0.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, bool ceil_rule) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int32_t e = (int32_t)(amax_bits >> 23) - 2 + ((ceil_rule && (amax_bits & 0x7FFFFFu) > 0x400000u) ? 1 : 0);
  return (uint32_t)max(e, 0);
}

// 2^-e of scale byte e + 127 (0 <= byte <= 253: a normal number).
__device__ __forceinline__ float mx_inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Byte offset of the scale of row r, column block kb = c / 32, in the TILED layout of a
// view with Cp padded columns: 512-byte atoms of 128 rows x 4 blocks.
__host__ __device__ __forceinline__ int64_t mx_scale_offset(int64_t r, int64_t kb, int64_t Cp) {
  const int64_t atom = (r >> 7) * (Cp >> 7) + (kb >> 2);
  return atom * kAtomBytes + 16 * (r & 31) + 4 * ((r & 127) >> 5) + (kb & 3);
}

// SplitMix64 (Steele, Lea and Flood, OOPSLA 2014) at count i of a generator started at `seed`.
__device__ __forceinline__ uint64_t splitmix64(uint64_t seed, uint64_t i) {
  uint64_t z = seed + (i + 1ull) * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// ------------------------------------------------------------------ element types
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void put_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put_as(__half* p, float v) { *p = __float2half_rn(v); }

// ------------------------------------------------------------------ tensor core, kind::mxf4
// Instruction descriptor: E2M1 x E2M1, UE8M0 scales, K-major A and B, FP32 accumulate, M x N,
// K = 64.  A 32-bit scale column holds a row's four blocks of 128 elements; `half` selects
// the two of the first or the second 64 (sub-column byte 0 or 2).
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int half) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
         ((uint32_t)(2 * half) << 4) | ((uint32_t)(2 * half) << 29);
}

// D (TMEM) (+)= A(smem) * B(smem)^T with per-32 UE8M0 scales from TMEM; K = 64.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
      : "memory");
}

// ------------------------------------------------------------------ dependent launches
// A product launched behind the quantisation of its operand starts while that still runs; the
// quantise kernel lets it (every CTA, at its start), and the product's producer waits for its
// end before the first load.
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_quantize(bool after) {
  if (after) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Shared-memory address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

}  // namespace fs4
