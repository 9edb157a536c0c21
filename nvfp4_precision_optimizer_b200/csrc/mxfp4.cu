// MXFP4 quantisation and dequantisation (sm_100a): E2M1 codes, one E8M0 scale per 32
// elements along a row of the view.
//
// Block rule, amax = max |x_i| over the block's elements (absent ones count as 0):
//   floor:  e = floor(log2 amax) - 2            (amax 2^-e in [4, 8): codes saturate at 6)
//   ceil:   e = min { e : amax <= 6 2^e }       (nothing saturates)
//   e >= -127 (also for amax = 0); scale byte e + 127; code_i = sign_i | E2M1(|x_i| 2^-e).
// The product with 2^-e is exact wherever the result is at least 2^-126 (below that the
// code is 0), so nearest rounding is the conversion instruction's, ties to even.
// Stochastic rounding: |x| 2^-e in [lo, hi) goes up iff u <= (v - lo) / (hi - lo), with
// u = (f + 1/2) 2^-16 and f a 16-bit field of SplitMix64 at the count of the element's
// group of four.  The kernel keeps the top 22 bits of the fraction: f' = 64 f + 32 is an
// integer, so f' <= fraction 2^22 decides the same with the fraction cut to its integer part.
// A block that holds NaN or Inf: scale byte 255 (NaN), codes 0.
//
// One pass: each CTA reads a 128 x 128 tile once (eight elements a thread and step, four
// threads a 32-element block) and writes the row view from registers; the column view
// reads the tile back from shared memory, one thread a column (FP32) or a pair of columns
// (16-bit types), and both views' scales leave as whole 512-byte atoms.  Bound by HBM: in
// bytes per element the input's size plus 17/32 for each view.
#include <cstdint>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace fs4 {
namespace {

constexpr int kMxThreads = 256;
constexpr int kMxTile = 128;                            // rows and columns of one CTA's tile
constexpr uint64_t kMxColumnSeed = 0xD1B54A32D192ED03ull;

template <typename T> struct MxIo;
template <> struct MxIo<float> {
  static constexpr int kVec = 2;                        // 16-byte loads for 8 elements
  static __device__ __forceinline__ float get(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void unpack(const uint4* w, float* x) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
  }
  static __device__ __forceinline__ void pack(const float* x, uint4* w) {
    w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  }
  static __device__ __forceinline__ float cast(float v) { return v; }
};
template <> struct MxIo<__nv_bfloat16> {
  static constexpr int kVec = 1;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }
  static __device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
  static __device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t two(float a, float b) { return pack_bf16x2(a, b); }
  static __device__ __forceinline__ void unpack(const uint4* w, float* x) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = lo(u[i]); x[2 * i + 1] = hi(u[i]); }
  }
  static __device__ __forceinline__ void pack(const float* x, uint4* w) {
    w[0] = make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
  }
  static __device__ __forceinline__ __nv_bfloat16 cast(float v) { return __float2bfloat16_rn(v); }
};
template <> struct MxIo<__half> {
  static constexpr int kVec = 1;
  static __device__ __forceinline__ float get(const __half* p) { return __half2float(__ldg(p)); }
  static __device__ __forceinline__ float lo(uint32_t u) { return half_lo(u); }
  static __device__ __forceinline__ float hi(uint32_t u) { return half_hi(u); }
  static __device__ __forceinline__ uint32_t two(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4* w, float* x) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = lo(u[i]); x[2 * i + 1] = hi(u[i]); }
  }
  static __device__ __forceinline__ void pack(const float* x, uint4* w) {
    w[0] = make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
  }
  static __device__ __forceinline__ __half cast(float v) { return __float2half_rn(v); }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight codes of x[0..7], nearest.
__device__ __forceinline__ uint32_t mx_codes8(const float* x, float inv) {
  return pack8_e2m1(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv, x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
}

// One code, stochastic.  Adding 1 (towards zero) to v < 1 gives every interval of the grid
// below 1 the form 1.m, so bit 22 upwards of the float counts grid points and the 22 bits
// below are the fraction of the interval.
__device__ __forceinline__ uint32_t mx_code_sr(float x, float inv, uint32_t f) {
  const float v = fminf(fabsf(x * inv), 6.0f);
  const bool small = v < 1.0f;
  const uint32_t b = __float_as_uint(small ? __fadd_rz(v, 1.0f) : v);
  uint32_t code = (b >> 22) - (small ? 254u : 252u);
  code += (64u * f + 32u <= (b & 0x3FFFFFu)) ? 1u : 0u;
  return code | ((__float_as_uint(x) >> 31) << 3);
}

// Eight codes of view elements (r, c) .. (r, c + 7), stochastic; c % 8 == 0.
__device__ __forceinline__ uint32_t mx_codes8_sr(const float* x, float inv, uint64_t seed, int64_t group) {
  uint32_t w = 0u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t z = splitmix64(seed, (uint64_t)(group + h));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w |= mx_code_sr(x[4 * h + j], inv, (uint32_t)(z >> (16 * j)) & 0xFFFFu) << (4 * (4 * h + j));
  }
  return w;
}

struct MxQuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  uint8_t* row_codes;
  uint8_t* row_scales;
  uint8_t* col_codes;
  uint8_t* col_scales;
  uint64_t seed;
  int32_t tiled;
  int32_t ceil_rule;
  int32_t vec;        // rows start on 16-byte boundaries
};

// `bytes` (4 or 16) code bytes of row r of a PLAIN view at byte b0, cut at the row's end.
template <int kBytes>
__device__ __forceinline__ void plain_store(uint8_t* codes, int64_t r, int64_t b0, int64_t row_bytes, const uint32_t* w) {
  uint8_t* p = codes + r * row_bytes + b0;
  if (b0 + kBytes <= row_bytes && (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0) {
    if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kBytes; ++i)
    if (b0 + i < row_bytes) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

template <typename T, bool kRow, bool kCol, bool kSr>
__global__ void __launch_bounds__(kMxThreads) mxfp4_quantize_kernel(const __grid_constant__ MxQuantArgs a,
                                                                    int32_t tiles_x) {
  extern __shared__ __align__(16) uint8_t mx_smem[];
  allow_dependents();
  __shared__ __align__(16) uint8_t row_atom[kAtomBytes];
  __shared__ __align__(16) uint8_t col_atom[kAtomBytes];
  T* tile = reinterpret_cast<T*>(mx_smem);
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_x) * kMxTile, c0 = (int64_t)(blockIdx.x % tiles_x) * kMxTile;
  const T* x = static_cast<const T*>(a.x);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool ceil_rule = a.ceil_rule != 0;
  const int64_t row_cp = (a.cols + 255) & ~int64_t(255), col_cp = (a.rows + 255) & ~int64_t(255);
  // the row view's padding ends at rows % 128, the column view's at cols % 128
  const bool row_in = kRow && (a.tiled ? r0 < ((a.rows + 127) & ~int64_t(127)) && c0 < row_cp : true);
  const int rr = lane >> 4, ch = lane & 15;    // two rows a warp and step, eight columns a lane
  const int64_t c = c0 + 8 * ch;
  const int64_t groups = (a.cols + 3) >> 2;
#pragma unroll 1
  for (int s0 = 0; s0 < 8; s0 += 4) {
    if (!a.tiled && r0 + 16 * s0 >= a.rows && !kCol) break;
    float xv[4][8];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t r = r0 + 16 * (s0 + s) + 2 * warp + rr;
      const T* p = x + r * a.ld + c;
      if (r < a.rows && c + 8 <= a.cols && a.vec) {
        uint4 w[MxIo<T>::kVec];
#pragma unroll
        for (int q = 0; q < MxIo<T>::kVec; ++q) w[q] = __ldg(reinterpret_cast<const uint4*>(p) + q);
        MxIo<T>::unpack(w, xv[s]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[s][i] = (r < a.rows && c + i < a.cols) ? MxIo<T>::get(p + i) : 0.0f;
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int tr = 16 * (s0 + s) + 2 * warp + rr;
      const int64_t r = r0 + tr;
      if constexpr (kCol) {
        uint4 w[MxIo<T>::kVec];
        MxIo<T>::pack(xv[s], w);                // exact: the values came from T
#pragma unroll
        for (int q = 0; q < MxIo<T>::kVec; ++q) reinterpret_cast<uint4*>(tile + tr * kMxTile + 8 * ch)[q] = w[q];
      }
      if constexpr (kRow) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, abs_bits(xv[s][i]));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t byte = mx_scale_byte(m, ceil_rule);
        uint32_t w = 0u;
        if (byte != 255u) {
          const float inv = mx_inverse_scale(byte);
          w = kSr ? mx_codes8_sr(xv[s], inv, a.seed, r * groups + (c >> 2)) : mx_codes8(xv[s], inv);
        }
        if (a.tiled) {
          if (row_in)
            *reinterpret_cast<uint32_t*>(a.row_codes + tiled_chunk_offset(r, c & ~int64_t(31), row_cp) + ((c & 31) >> 1)) = w;
          if ((lane & 3) == 0) row_atom[16 * (tr & 31) + 4 * (tr >> 5) + (ch >> 2)] = (uint8_t)byte;
        } else if (r < a.rows && c < a.cols) {
          // an odd row's last nibble is 0: its element was read as 0
          plain_store<4>(a.row_codes, r, c >> 1, (a.cols + 1) >> 1, &w);
          if ((lane & 3) == 0) a.row_scales[r * ((a.cols + 31) >> 5) + (c >> 5)] = (uint8_t)byte;
        }
      }
    }
  }
  if (kCol || a.tiled) __syncthreads();
  if constexpr (kCol) {
    // column pass: lanes take consecutive 32-bit words of a tile row
    constexpr int kPair = sizeof(T) == 4 ? 1 : 2;               // columns per word
    constexpr int kTasks = kMxTile / kPair * 4 / kMxThreads;     // (column word, 32-row block) a thread
    const bool col_in = a.tiled ? c0 < ((a.cols + 127) & ~int64_t(127)) && r0 < col_cp : true;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(tile);
    const int64_t cgroups = (a.rows + 3) >> 2;
    const uint64_t cseed = a.seed ^ kMxColumnSeed;
#pragma unroll
    for (int t = 0; t < kTasks; ++t) {
      const int task = threadIdx.x + t * kMxThreads;
      const int cw = task % (kMxTile / kPair), blk = task / (kMxTile / kPair);
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = words[(32 * blk + i) * (kMxTile / kPair) + cw];
#pragma unroll
      for (int h = 0; h < kPair; ++h) {
        auto value = [&](int i) -> float {
          if constexpr (kPair == 1) return __uint_as_float(w[i]);
          else return h ? MxIo<T>::hi(w[i]) : MxIo<T>::lo(w[i]);
        };
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, abs_bits(value(i)));
        const uint32_t byte = mx_scale_byte(m, ceil_rule);
        uint32_t q[4] = {0u, 0u, 0u, 0u};
        const int tc = kPair * cw + h;
        const int64_t vr = c0 + tc, vc = r0 + 32 * blk;          // row and column in the view
        if (byte != 255u) {
          const float inv = mx_inverse_scale(byte);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = value(8 * g + i);
            q[g] = kSr ? mx_codes8_sr(v, inv, cseed, vr * cgroups + ((vc + 8 * g) >> 2)) : mx_codes8(v, inv);
          }
        }
        if (a.tiled) {
          if (col_in)
            *reinterpret_cast<uint4*>(a.col_codes + tiled_chunk_offset(vr, vc, col_cp)) = make_uint4(q[0], q[1], q[2], q[3]);
          col_atom[16 * (tc & 31) + 4 * (tc >> 5) + blk] = (uint8_t)byte;
        } else if (vr < a.cols && vc < a.rows) {
          plain_store<16>(a.col_codes, vr, vc >> 1, (a.rows + 1) >> 1, q);
          a.col_scales[vr * ((a.rows + 31) >> 5) + (vc >> 5)] = (uint8_t)byte;
        }
      }
    }
    if (a.tiled) {
      __syncthreads();
      if (col_in && threadIdx.x >= 32 && threadIdx.x < 64)
        reinterpret_cast<uint4*>(a.col_scales + ((c0 >> 7) * (col_cp >> 7) + (r0 >> 7)) * kAtomBytes)[lane] =
            reinterpret_cast<const uint4*>(col_atom)[lane];
    }
  }
  if constexpr (kRow) {
    if (a.tiled && row_in && threadIdx.x < 32)
      reinterpret_cast<uint4*>(a.row_scales + ((r0 >> 7) * (row_cp >> 7) + (c0 >> 7)) * kAtomBytes)[lane] =
          reinterpret_cast<const uint4*>(row_atom)[lane];
  }
}

template <typename T, bool kRow, bool kCol, bool kSr>
cudaError_t launch_quant(const MxQuantArgs& a, cudaStream_t st) {
  // extent: what the views' padding has to cover (TILED), or the matrix
  auto up = [](int64_t v, int64_t m) { return (v + m - 1) / m * m; };
  int64_t er = a.rows, ec = a.cols;
  if (a.tiled) {
    er = up(a.rows, kCol ? 256 : 128);
    ec = up(a.cols, kRow ? 256 : 128);
  }
  const int64_t gx = (ec + kMxTile - 1) / kMxTile, gy = (er + kMxTile - 1) / kMxTile;
  if (gx * gy > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;   // over 2^45 elements
  const size_t smem = kCol ? (size_t)kMxTile * kMxTile * sizeof(T) : 0;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(mxfp4_quantize_kernel<T, kRow, kCol, kSr>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  mxfp4_quantize_kernel<T, kRow, kCol, kSr><<<(unsigned)(gx * gy), kMxThreads, smem, st>>>(a, (int32_t)gx);
  return cudaGetLastError();
}

template <typename T, bool kSr>
cudaError_t launch_quant_views(const MxQuantArgs& a, cudaStream_t st) {
  if (a.row_codes && a.col_codes) return launch_quant<T, true, true, kSr>(a, st);
  if (a.col_codes) return launch_quant<T, false, true, kSr>(a, st);
  return launch_quant<T, true, false, kSr>(a, st);
}

template <typename T>
cudaError_t launch_quant_type(const MxQuantArgs& a, bool sr, cudaStream_t st) {
  return sr ? launch_quant_views<T, true>(a, st) : launch_quant_views<T, false>(a, st);
}

struct MxDequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, ld;
  void* y;
  int32_t tiled;
  int32_t vec;      // rows of y start on 16-byte boundaries
  int32_t word;     // rows of PLAIN codes start on 4-byte boundaries
};

// y = code 2^(byte - 127), rounded once to T.  Eight elements a thread, 256 columns a warp,
// four rows a warp at once so that four loads are in flight.  Bound by HBM.
template <typename T>
__global__ void __launch_bounds__(kMxThreads) mxfp4_dequantize_kernel(const __grid_constant__ MxDequantArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cp = (a.cols + 255) & ~int64_t(255);
  const int64_t segs = cp >> 8, groups = (a.rows + 3) >> 2, total = segs * groups;
  const int64_t row_bytes = (a.cols + 1) >> 1, row_blocks = (a.cols + 31) >> 5;
  for (int64_t t = (int64_t)blockIdx.x * (kMxThreads / 32) + warp; t < total; t += (int64_t)gridDim.x * (kMxThreads / 32)) {
    const int64_t rg = 4 * (t / segs), c = (t % segs) * 256 + 8 * lane;
    if (c >= a.cols) continue;
    uint32_t w[4], byte[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = rg + i;
      w[i] = 0u;
      byte[i] = 0u;
      if (r >= a.rows) continue;
      if (a.tiled) {
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(a.codes + tiled_chunk_offset(r, c & ~int64_t(31), cp) + ((c & 31) >> 1)));
        byte[i] = __ldg(a.scales + mx_scale_offset(r, c >> 5, cp));
      } else {
        const uint8_t* p = a.codes + r * row_bytes + (c >> 1);
        if (a.word && c + 8 <= a.cols) {
          w[i] = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((c >> 1) + k < row_bytes) w[i] |= (uint32_t)__ldg(p + k) << (8 * k);
        }
        byte[i] = __ldg(a.scales + r * row_blocks + (c >> 5));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = rg + i;
      if (r >= a.rows) continue;
      // 2^(byte - 127): byte 0 is the subnormal 2^-127, byte 255 NaN
      const float s = byte[i] == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte[i] ? byte[i] << 23 : 0x400000u);
      uint32_t h[4];
      float v[8];
      e2m1_decode8(w[i], h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = half_lo(h[k]) * s;
        v[2 * k + 1] = half_hi(h[k]) * s;
      }
      T* y = static_cast<T*>(a.y) + r * a.ld + c;
      if (a.vec && c + 8 <= a.cols) {
        uint4 o[MxIo<T>::kVec];
        MxIo<T>::pack(v, o);
#pragma unroll
        for (int k = 0; k < MxIo<T>::kVec; ++k) reinterpret_cast<uint4*>(y)[k] = o[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < a.cols) y[k] = MxIo<T>::cast(v[k]);
      }
    }
  }
}

template <typename T>
cudaError_t launch_dequant(const MxDequantArgs& a, cudaStream_t st, int num_sms) {
  const int64_t warps = ((a.cols + 255) / 256) * ((a.rows + 3) / 4);
  const int64_t want = (warps + kMxThreads / 32 - 1) / (kMxThreads / 32), most = (int64_t)num_sms * 16;
  mxfp4_dequantize_kernel<T><<<(unsigned)(want < most ? want : most), kMxThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* row_codes,
                                  uint8_t* row_scales, uint8_t* col_codes, uint8_t* col_scales, bool tiled, bool ceil_rule,
                                  bool stochastic, uint64_t seed, cudaStream_t st) {
  MxQuantArgs a{x, rows, cols, ld, row_codes, row_scales, col_codes, col_scales, seed, tiled, ceil_rule, 0};
  const int64_t size = dtype == kTypeF32 ? 4 : 2;
  a.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (rows == 1 || ld * size % 16 == 0);
  switch (dtype) {
    case kTypeF32: return launch_quant_type<float>(a, stochastic, st);
    case kTypeBf16: return launch_quant_type<__nv_bfloat16>(a, stochastic, st);
    default: return launch_quant_type<__half>(a, stochastic, st);
  }
}

cudaError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* y, int dtype,
                                    int64_t ld, bool tiled, cudaStream_t st, int num_sms) {
  MxDequantArgs a{codes, scales, rows, cols, ld, y, tiled, 0, 0};
  const int64_t size = dtype == kTypeF32 ? 4 : 2;
  a.vec = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (rows == 1 || ld * size % 16 == 0);
  a.word = reinterpret_cast<uintptr_t>(codes) % 4 == 0 && (rows == 1 || (cols + 1) / 2 % 4 == 0);
  switch (dtype) {
    case kTypeF32: return launch_dequant<float>(a, st, num_sms);
    case kTypeBf16: return launch_dequant<__nv_bfloat16>(a, st, num_sms);
    default: return launch_dequant<__half>(a, st, num_sms);
  }
}

}  // namespace fs4
