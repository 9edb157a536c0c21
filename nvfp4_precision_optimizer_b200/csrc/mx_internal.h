// Internal definitions shared by the MXFP4 and Muon kernels and their C entry points.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fs4.h"

namespace fs4 {

// Element types of the C ABI (fs4_dtype).
constexpr int kTypeF32 = 0, kTypeBf16 = 1, kTypeF16 = 2;
inline int64_t type_bytes(int dtype) { return dtype == kTypeF32 ? 4 : 2; }

// The bytes of a matrix or a buffer: [lo, hi), of which rows of `width` bytes, `pitch` apart, are its
// own (pitch 0: all of them).
struct Span {
  uintptr_t lo, hi;
  uint64_t pitch, width;
};
inline Span bytes_at(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)(p ? bytes : 0), 0, (uint64_t)(p ? bytes : 0)};
}
inline Span matrix_at(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t type) {
  Span s = bytes_at(p, ((rows - 1) * ld + cols) * type_bytes(type));
  if (rows > 1) s.pitch = (uint64_t)(ld * type_bytes(type));
  s.width = (uint64_t)(cols * type_bytes(type));
  return s;
}
// Whether two of them share a byte.  Matrices of one pitch may lie side by side, as column slices of
// one buffer do: modulo the pitch a's rows are [0, a.width) and b's start at d.  Different pitches
// count as overlapping where their ranges do.
inline bool meet(const Span& a, const Span& b) {
  if (!(a.lo < b.hi && b.lo < a.hi)) return false;
  const uint64_t pitch = a.pitch ? a.pitch : b.pitch;
  if (pitch == 0 || (b.pitch != 0 && b.pitch != pitch)) return true;
  const uint64_t d = b.lo >= a.lo ? (b.lo - a.lo) % pitch : (pitch - (a.lo - b.lo) % pitch) % pitch;
  return !(d >= a.width && d + b.width <= pitch);
}

// The current device's SM count; FS4_ERR_ARCH off sm_100 (api.cu).
fs4_status current_device(int* num_sms);

// ---------------------------------------------------------------- launchers (mxfp4.cu)
cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* row_codes,
                                  uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, bool tiled, bool ceil_rule,
                                  bool stochastic, uint64_t seed, cudaStream_t st);
cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* y, int dtype,
                                    int64_t ld, bool tiled, cudaStream_t st, int num_sms);

// ---------------------------------------------------------------- launchers (mxfp4_gemm.cu)
struct MxGemmArgs {
  const uint8_t* a_codes;
  const uint8_t* a_scales;
  const uint8_t* b_codes;
  const uint8_t* b_scales;
  int64_t M, N, K;
  void* d;
  int64_t ldd;
  int32_t dtype;
  int32_t accumulate;
  uint32_t* status;
  int32_t after_quantize;   // the launch before quantises A: overlap its end
  int32_t stall;            // test only: the MMA issuer waits on a barrier nothing arrives on
};
cudaError_t launch_mxfp4_pair(const MxGemmArgs& a, cudaStream_t st);   // mxfp4_pair.cu
// A few rows of x times W in one launch that quantises x on its way; false where x does not fit.
struct MxLinearArgs {
  const void* x;
  const uint8_t* w_codes;
  const uint8_t* w_scales;
  int64_t M, N, K, ldx;
  void* d;
  int64_t ldd;
  int32_t x_dtype, d_dtype;
  int32_t accumulate, ceil_rule;
  uint32_t* status;
  int32_t stall;
};
bool mxfp4_linear_fused(const MxLinearArgs& a, cudaStream_t st, int num_sms, cudaError_t* error);
cudaError_t launch_mxfp4_gemm(const MxGemmArgs& a, cudaStream_t st, int num_sms);

}  // namespace fs4
