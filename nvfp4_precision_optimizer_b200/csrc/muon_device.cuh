// Element access shared by the Muon kernels: values of any of the three types, the update
// direction, and the owner of a work unit.
#pragma once

#include "muon_internal.h"
#include "mx_device.cuh"

namespace fs4 {

__device__ __forceinline__ int owner_of(const int32_t* prefix, int count, int32_t u) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Round to the type and back: what a later read sees.
__device__ __forceinline__ float put1(void* p, int64_t i, int type, float v) {
  if (type == kTypeF32) {
    static_cast<float*>(p)[i] = v;
    return v;
  }
  if (type == kTypeBf16) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    static_cast<__nv_bfloat16*>(p)[i] = h;
    return __bfloat162float(h);
  }
  const __half h = __float2half_rn(v);
  static_cast<__half*>(p)[i] = h;
  return __half2float(h);
}

__device__ __forceinline__ bool aligned16(const void* p, int64_t ld, int type) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * (type == kTypeF32 ? 4 : 2))) & 15) == 0;
}

// Eight consecutive elements from index i (16-byte aligned) as they are in memory, and their
// values: apart, so that several loads are in flight before the first is unpacked.
struct Raw8 {
  uint4 a, b;
};
__device__ __forceinline__ Raw8 load8(const void* p, int64_t i, int type) {
  Raw8 r;
  if (type == kTypeF32) {
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.a = f[0];
    r.b = f[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    r.b = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8& r, int type, float* v) {
  const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  if (type == kTypeF32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]);
  } else if (type == kTypeBf16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(u[k] << 16);
      v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = half_lo(u[k]);
      v[2 * k + 1] = half_hi(u[k]);
    }
  }
}
// Eight elements at[i], absent where it is negative (0): the loads are in flight together.
template <typename T>
__device__ __forceinline__ void gather8_as(const void* p, const int64_t* at, float* v) {
  const T* q = static_cast<const T*>(p);
  T raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at[i] >= 0) raw[i] = q[at[i]];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = at[i] >= 0 ? to_f32(raw[i]) : 0.0f;
}
__device__ __forceinline__ void gather8(const void* p, int type, const int64_t* at, float* v) {
  if (type == kTypeF32) gather8_as<float>(p, at, v);
  else if (type == kTypeBf16) gather8_as<__nv_bfloat16>(p, at, v);
  else gather8_as<__half>(p, at, v);
}

// Store and replace by what was stored.
__device__ __forceinline__ void put8(void* p, int64_t i, int type, float* v) {
  if (type == kTypeF32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (type == kTypeBf16) {
      u[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
      v[2 * k] = __uint_as_float(u[k] << 16);
      v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
      v[2 * k] = half_lo(u[k]);
      v[2 * k + 1] = half_hi(u[k]);
    }
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float direction(const MuonCall& p, float mom, float g) {
  return p.nesterov ? fmaf(p.beta, mom, p.rest * g) : mom;
}

// FP16 parts of eight values: value = high + low, to 22 significand bits or 2^-25, whichever is
// more (values are scaled: X by 2^12, A by 2^8).
__device__ __forceinline__ uint32_t two_halves(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void join8(uint4 hi, uint4 lo, float* v) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = half_lo(l[i]) + half_lo(h[i]);
    v[2 * i + 1] = half_hi(l[i]) + half_hi(h[i]);
  }
}
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = two_halves(v[2 * i], v[2 * i + 1]);
    l[i] = two_halves(v[2 * i] - half_lo(h[i]), v[2 * i + 1] - half_hi(h[i]));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

}  // namespace fs4
