// C entry points of the MXFP4 operators (declared in include/fs4.h): argument checks and launches.
#include "mx_internal.h"

using namespace fs4;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline fs4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FS4_OK : FS4_ERR_CUDA; }
inline bool known_type(int32_t t) { return t == FS4_F32 || t == FS4_BF16 || t == FS4_F16; }
inline int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// Codes and scales of a rows x K view.
Span code_range(const void* p, int64_t rows, int64_t K, bool tiled) {
  return bytes_at(p, tiled ? up(rows, 128) * up(K, 256) / 2 : rows * ((K + 1) / 2));
}
Span scale_range(const void* p, int64_t rows, int64_t K, bool tiled) {
  return bytes_at(p, tiled ? up(rows, 128) * up(K, 256) / 32 : rows * ((K + 31) / 32));
}

constexpr int64_t kMxMaxDim = int64_t(1) << 31;
constexpr int64_t kMxMaxGemm = int64_t(1) << 20;    // rows, columns and K of a product
constexpr int64_t kMxHeader = 256;                  // the workspace's status word

fs4_status check_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales, int64_t M,
                      int64_t N, int64_t K, const void* d, int32_t d_dtype, int64_t ldd, const void* workspace,
                      size_t workspace_bytes) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !d || !known_type(d_dtype)) return FS4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1 || M > kMxMaxGemm || N > kMxMaxGemm || K > kMxMaxGemm) return FS4_ERR_SHAPE;
  if (ldd < N || ldd > INT64_MAX / 4 / M) return FS4_ERR_INVALID_ARG;
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(b_codes, 16) || !aligned(b_scales, 16) ||
      !aligned(d, type_bytes(d_dtype)))
    return FS4_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kMxHeader) return FS4_ERR_WORKSPACE;
  const Span out = matrix_at(d, M, N, ldd, d_dtype), header = bytes_at(workspace, kMxHeader);
  if (meet(out, code_range(a_codes, M, K, true)) || meet(out, scale_range(a_scales, M, K, true)) ||
      meet(out, code_range(b_codes, N, K, true)) || meet(out, scale_range(b_scales, N, K, true)) || meet(out, header))
    return FS4_ERR_ALIAS;
  return FS4_OK;
}

}  // namespace

extern "C" {

fs4_status fs4_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* row_codes,
                              uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, uint32_t flags, uint64_t seed,
                              void* stream) {
  const bool row = row_codes != nullptr, col = col_codes != nullptr;
  if (!x || (!row && !col) || row != (row_scales != nullptr) || col != (col_scales != nullptr)) return FS4_ERR_INVALID_ARG;
  if (!known_type(dtype)) return FS4_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(FS4_LAYOUT_TILED | FS4_MX_SCALE_CEIL | FS4_MX_STOCHASTIC)) return FS4_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1 || rows > kMxMaxDim || cols > kMxMaxDim) return FS4_ERR_SHAPE;
  if (ld < cols || ld > INT64_MAX / 4 / rows) return FS4_ERR_INVALID_ARG;
  if (!aligned(x, type_bytes(dtype)) || !aligned(row_codes, 16) || !aligned(row_scales, 16) || !aligned(col_codes, 16) ||
      !aligned(col_scales, 16))
    return FS4_ERR_INVALID_ARG;
  const bool tiled = (flags & FS4_LAYOUT_TILED) != 0;
  const Span r[5] = {matrix_at(x, rows, cols, ld, dtype), code_range(row_codes, rows, cols, tiled),
                      scale_range(row_scales, rows, cols, tiled), code_range(col_codes, cols, rows, tiled),
                      scale_range(col_scales, cols, rows, tiled)};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (meet(r[i], r[j])) return FS4_ERR_ALIAS;
  int sms = 0;
  const fs4_status ds = current_device(&sms);
  if (ds != FS4_OK) return ds;
  return cuda_status(launch_mxfp4_quantize(x, dtype, rows, cols, ld, row_codes, row_scales, col_codes, col_scales, tiled,
                                           (flags & FS4_MX_SCALE_CEIL) != 0, (flags & FS4_MX_STOCHASTIC) != 0, seed,
                                           static_cast<cudaStream_t>(stream)));
}

fs4_status fs4_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* y, int32_t dtype,
                                int64_t ld, uint32_t flags, void* stream) {
  if (!codes || !scales || !y || !known_type(dtype)) return FS4_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)FS4_LAYOUT_TILED) return FS4_ERR_INVALID_ARG;
  if (rows < 1 || cols < 1 || rows > kMxMaxDim || cols > kMxMaxDim) return FS4_ERR_SHAPE;
  if (ld < cols || ld > INT64_MAX / 4 / rows) return FS4_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(y, type_bytes(dtype))) return FS4_ERR_INVALID_ARG;
  const bool tiled = (flags & FS4_LAYOUT_TILED) != 0;
  const Span out = matrix_at(y, rows, cols, ld, dtype);
  if (meet(out, code_range(codes, rows, cols, tiled)) || meet(out, scale_range(scales, rows, cols, tiled))) return FS4_ERR_ALIAS;
  int sms = 0;
  const fs4_status ds = current_device(&sms);
  if (ds != FS4_OK) return ds;
  return cuda_status(launch_mxfp4_dequantize(codes, scales, rows, cols, y, dtype, ld, tiled, static_cast<cudaStream_t>(stream), sms));
}

fs4_status fs4_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                          int64_t M, int64_t N, int64_t K, void* d, int32_t d_dtype, int64_t ldd, uint32_t flags, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (flags & ~(uint32_t)(FS4_MX_ACCUMULATE | FS4_TEST_STALL)) return FS4_ERR_INVALID_ARG;
  const fs4_status s = check_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, d, d_dtype, ldd, workspace, workspace_bytes);
  if (s != FS4_OK) return s;
  int sms = 0;
  const fs4_status ds = current_device(&sms);
  if (ds != FS4_OK) return ds;
  MxGemmArgs g{a_codes, a_scales, b_codes, b_scales, M, N, K, d, ldd, d_dtype, (flags & FS4_MX_ACCUMULATE) ? 1 : 0,
               static_cast<uint32_t*>(workspace), 0, (flags & FS4_TEST_STALL) ? 1 : 0};
  return cuda_status(launch_mxfp4_gemm(g, static_cast<cudaStream_t>(stream), sms));
}

size_t fs4_mxfp4_linear_workspace_size(int64_t M, int64_t K) {
  if (M < 1 || K < 1 || M > kMxMaxGemm || K > kMxMaxGemm) return 0;
  return (size_t)(kMxHeader + up(M, 128) * up(K, 256) / 32 * 17);
}

fs4_status fs4_mxfp4_linear(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t* w_codes,
                            const uint8_t* w_scales, int64_t N, void* d, int32_t d_dtype, int64_t ldd, uint32_t flags,
                            void* workspace, size_t workspace_bytes, void* stream) {
  return fs4_mxfp4_linear_ex(x, x_dtype, M, K, ldx, w_codes, w_scales, N, d, d_dtype, ldd, flags, workspace, workspace_bytes, workspace,
                             stream);
}

fs4_status fs4_mxfp4_linear_ex(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t* w_codes,
                               const uint8_t* w_scales, int64_t N, void* d, int32_t d_dtype, int64_t ldd, uint32_t flags,
                               void* workspace, size_t workspace_bytes, void* status, void* stream) {
  if (!x || !w_codes || !w_scales || !d || !known_type(x_dtype) || !known_type(d_dtype)) return FS4_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(FS4_MX_SCALE_CEIL | FS4_MX_ACCUMULATE | FS4_TEST_STALL)) return FS4_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1 || M > kMxMaxGemm || N > kMxMaxGemm || K > kMxMaxGemm) return FS4_ERR_SHAPE;
  if (ldx < K || ldx > INT64_MAX / 4 / M) return FS4_ERR_INVALID_ARG;
  const size_t need = fs4_mxfp4_linear_workspace_size(M, K);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return FS4_ERR_WORKSPACE;
  if (!status || !aligned(status, 256)) return FS4_ERR_WORKSPACE;
  uint8_t* codes = static_cast<uint8_t*>(workspace) + kMxHeader;
  uint8_t* scales = codes + up(M, 128) * up(K, 256) / 2;
  const Span ws = bytes_at(workspace, (int64_t)need), xr = matrix_at(x, M, K, ldx, x_dtype);
  if (meet(ws, xr) || meet(ws, code_range(w_codes, N, K, true)) || meet(ws, scale_range(w_scales, N, K, true))) return FS4_ERR_ALIAS;
  if (ldd >= N && ldd <= INT64_MAX / 4 / M) {
    const Span out = matrix_at(d, M, N, ldd, d_dtype);
    if (meet(out, ws) || meet(out, xr)) return FS4_ERR_ALIAS;
  }
  if (status != workspace) {
    const Span word = bytes_at(status, kMxHeader);
    if (meet(word, ws) || meet(word, xr) || meet(word, code_range(w_codes, N, K, true)) || meet(word, scale_range(w_scales, N, K, true)))
      return FS4_ERR_ALIAS;
  }
  // the product's checks come before the quantisation is enqueued
  fs4_status s = check_gemm(codes, scales, w_codes, w_scales, M, N, K, d, d_dtype, ldd, status, kMxHeader);
  if (s != FS4_OK) return s;
  if (!aligned(x, type_bytes(x_dtype))) return FS4_ERR_INVALID_ARG;
  int sms = 0;
  if ((s = current_device(&sms)) != FS4_OK) return s;
  MxLinearArgs l{x, w_codes, w_scales, M, N, K, ldx, d, ldd, x_dtype, d_dtype, (flags & FS4_MX_ACCUMULATE) ? 1 : 0,
                 (flags & FS4_MX_SCALE_CEIL) ? 1 : 0, static_cast<uint32_t*>(status), (flags & FS4_TEST_STALL) ? 1 : 0};
  cudaError_t e = cudaSuccess;
  if (mxfp4_linear_fused(l, static_cast<cudaStream_t>(stream), sms, &e)) return cuda_status(e);
  s = fs4_mxfp4_quantize(x, x_dtype, M, K, ldx, codes, scales, nullptr, nullptr, FS4_LAYOUT_TILED | (flags & FS4_MX_SCALE_CEIL), 0,
                         stream);
  if (s != FS4_OK) return s;
  MxGemmArgs g{codes, scales, w_codes, w_scales, M, N, K, d, ldd, d_dtype, (flags & FS4_MX_ACCUMULATE) ? 1 : 0,
               static_cast<uint32_t*>(status), 1, l.stall};
  return cuda_status(launch_mxfp4_gemm(g, static_cast<cudaStream_t>(stream), sms));
}

}  // extern "C"
