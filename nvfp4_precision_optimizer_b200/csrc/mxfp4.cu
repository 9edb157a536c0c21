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
// One pass: each CTA reads a 128 x 128 tile once (four pieces of sixteen elements a thread, all
// loads first, two threads a 32-element block) and writes the row view from registers; the column view
// reads the tile back from shared memory, one thread a column (FP32) or a pair of columns
// (16-bit types), and both views' scales leave as whole 512-byte atoms.  The floor is HBM: in
// bytes per element the input's size plus 17/32 for each view.  Measured on BF16, 8192 x 5120: the row view
// 20.6 us (5.1 TB/s); the column view 31.6 us PLAIN and 23.1 TILED, both 39.9 and 27.2 (PLAIN's column
// view is stored in pieces of 16 bytes, half a sector, each in a row of its own); stochastic 49 us a
// view and 94 both, where the random stream's arithmetic keeps 67% of the issue slots busy.
#include <cstdint>
#include <type_traits>

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

// Sixteen consecutive elements of T as they are in memory.
template <typename T>
struct Piece {
  static constexpr int kWords = 4 * (int)sizeof(T);       // 32-bit words
  uint32_t w[kWords];
};

// Largest |x| of the pieces' words, as a running maximum over packed magnitudes ...
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w) {
  if constexpr (sizeof(T) == 4) return max(m, w & 0x7FFFFFFFu);
  else return max_u16x2(m, w & 0x7FFF7FFFu);
}
// ... and float bits of a 16-bit magnitude (Inf and NaN stay Inf or NaN).
template <typename T>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t m16) {
  if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m16)));
  else return m16 << 16;
}
// Element i of packed words.
template <typename T>
__device__ __forceinline__ float element(const uint32_t* w, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
  else return (i & 1) ? MxIo<T>::hi(w[i >> 1]) : MxIo<T>::lo(w[i >> 1]);
}

// Eight codes of x[0..7], nearest.
__device__ __forceinline__ uint32_t mx_codes8(const float* x, float inv) {
  return pack8_e2m1(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv, x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
}

// One code, stochastic.  Adding 1 (towards zero) to v < 1 gives every interval of the grid
// below 1 the form 1.m, so bit 22 upwards of the float counts grid points and the 22 bits
// below are the fraction F of the interval.  64 f + 32 <= F exactly when F + 64 (65535 - f) + 32
// carries into bit 22; `nf` is 65535 - f.
__device__ __forceinline__ uint32_t mx_code_sr(float x, float inv, uint32_t nf) {
  const float v = fminf(fabsf(x * inv), 6.0f);
  const bool small = v < 1.0f;
  const uint32_t b = __float_as_uint(small ? __fadd_rz(v, 1.0f) : v);
  const uint32_t code = ((b + 64u * nf + 32u) >> 22) - (small ? 254u : 252u);
  return code | ((__float_as_uint(x) >> 28) & 8u);
}

// Eight codes of view elements (r, c) .. (r, c + 7), stochastic; group = the first's group of four.
__device__ __forceinline__ uint32_t mx_codes8_sr(const float* x, float inv, uint64_t seed, int64_t group) {
  uint32_t w = 0u;
#pragma unroll
  for (int h = 1; h >= 0; --h) {
    const uint64_t z = ~splitmix64(seed, (uint64_t)(group + h));
    const uint32_t lo = (uint32_t)z, hi = (uint32_t)(z >> 32);
    w = 16u * w + mx_code_sr(x[4 * h + 3], inv, hi >> 16);
    w = 16u * w + mx_code_sr(x[4 * h + 2], inv, hi & 0xFFFFu);
    w = 16u * w + mx_code_sr(x[4 * h + 1], inv, lo >> 16);
    w = 16u * w + mx_code_sr(x[4 * h], inv, lo & 0xFFFFu);
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
  int32_t vec;        // rows start on 32-byte (2) or 16-byte (1) boundaries
};

// `kBytes` (8 or 16) code bytes of row r of a PLAIN view at byte b0, cut at the row's end.
template <int kBytes>
__device__ __forceinline__ void plain_store(uint8_t* codes, int64_t r, int64_t b0, int64_t row_bytes, const uint32_t* w) {
  uint8_t* p = codes + r * row_bytes + b0;
  if (b0 + kBytes <= row_bytes && (reinterpret_cast<uintptr_t>(p) & (kBytes - 1)) == 0) {
    if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
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
  // four rows a warp and step, sixteen columns a lane, two lanes a block
  const int rr = lane >> 3, ch = lane & 7;
  const int64_t c = c0 + 16 * ch;
  const int64_t groups = (a.cols + 3) >> 2;
  uint8_t* const row_tile = a.row_codes + ((r0 >> 7) * (row_cp >> 8) + (c0 >> 8)) * kTileBytes + 8 * (lane & 1);
  const int row_chunk = (int)((c0 & 255) >> 5) + (ch >> 1);
  constexpr int kSteps = 4;
  Piece<T> piece[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t r = r0 + 32 * s + 4 * warp + rr;
    const T* p = x + r * a.ld + c;
    uint32_t* w = piece[s].w;
    if (r < a.rows && c + 16 <= a.cols) {
      if (a.vec == 2) {
#pragma unroll
        for (int q = 0; q < Piece<T>::kWords / 8; ++q)
          asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(w[8 * q]), "=r"(w[8 * q + 1]), "=r"(w[8 * q + 2]), "=r"(w[8 * q + 3]), "=r"(w[8 * q + 4]),
                         "=r"(w[8 * q + 5]), "=r"(w[8 * q + 6]), "=r"(w[8 * q + 7])
                       : "l"(reinterpret_cast<const uint8_t*>(p) + 32 * q));
      } else if (a.vec == 1) {
#pragma unroll
        for (int q = 0; q < Piece<T>::kWords / 4; ++q) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + q);
          w[4 * q] = u.x; w[4 * q + 1] = u.y; w[4 * q + 2] = u.z; w[4 * q + 3] = u.w;
        }
      } else if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
        for (int i = 0; i < Piece<T>::kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
      } else if constexpr (sizeof(T) == 2) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (uint32_t)__ldg(h + 2 * i) | (uint32_t)__ldg(h + 2 * i + 1) << 16;
      }
    } else {
#pragma unroll
      for (int i = 0; i < Piece<T>::kWords; ++i) w[i] = 0u;
      if (r < a.rows) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= a.cols) continue;
          if constexpr (sizeof(T) == 4) w[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
          else w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + i) << (16 * (i & 1));
        }
      }
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int tr = 32 * s + 4 * warp + rr;
    const int64_t r = r0 + tr;
    const uint32_t* w = piece[s].w;
    if constexpr (kCol) {
#pragma unroll
      for (int q = 0; q < Piece<T>::kWords / 4; ++q)
        reinterpret_cast<uint4*>(tile + tr * kMxTile + 16 * ch)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
    if constexpr (kRow) {
      if (!a.tiled && r0 + 32 * s >= a.rows) continue;       // (uniform)
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < Piece<T>::kWords; ++i) m = max_magnitude<T>(m, w[i]);
      if constexpr (sizeof(T) == 2) m = magnitude_bits<T>(max(m & 0xFFFFu, m >> 16));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      const uint32_t byte = mx_scale_byte(m, ceil_rule);
      uint32_t q[2] = {0u, 0u};
      if (byte != 255u) {
        const float inv = mx_inverse_scale(byte);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = element<T>(w, 8 * g + i);
          q[g] = kSr ? mx_codes8_sr(v, inv, a.seed, r * groups + (c >> 2) + 2 * g) : mx_codes8(v, inv);
        }
      }
      if (a.tiled) {
        if (row_in) *reinterpret_cast<uint2*>(row_tile + 128 * tr + ((row_chunk ^ (tr & 7)) << 4)) = make_uint2(q[0], q[1]);
        if ((lane & 1) == 0) row_atom[16 * (tr & 31) + 4 * (tr >> 5) + (ch >> 1)] = (uint8_t)byte;
      } else if (r < a.rows && c < a.cols) {
        // an odd row's last nibble is 0: its element was read as 0
        plain_store<8>(a.row_codes, r, c >> 1, (a.cols + 1) >> 1, q);
        if ((lane & 1) == 0) a.row_scales[r * ((a.cols + 31) >> 5) + (c >> 5)] = (uint8_t)byte;
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
    uint8_t* const col_tile = a.col_codes + ((c0 >> 7) * (col_cp >> 8) + (r0 >> 8)) * kTileBytes;
    const int col_chunk = (int)((r0 & 255) >> 5);
#pragma unroll
    for (int t = 0; t < kTasks; ++t) {
      const int task = threadIdx.x + t * kMxThreads;
      const int cw = task % (kMxTile / kPair), blk = task / (kMxTile / kPair);
      uint32_t w[32], m2 = 0u;
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = words[(32 * blk + i) * (kMxTile / kPair) + cw];
#pragma unroll
      for (int i = 0; i < 32; ++i) m2 = max_magnitude<T>(m2, w[i]);      // both columns of a word
#pragma unroll
      for (int h = 0; h < kPair; ++h) {
        const uint32_t m = kPair == 1 ? m2 : magnitude_bits<T>(h ? m2 >> 16 : m2 & 0xFFFFu);
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
            for (int i = 0; i < 8; ++i) {
              if constexpr (kPair == 1) v[i] = __uint_as_float(w[8 * g + i]);
              else v[i] = h ? MxIo<T>::hi(w[8 * g + i]) : MxIo<T>::lo(w[8 * g + i]);
            }
            q[g] = kSr ? mx_codes8_sr(v, inv, cseed, vr * cgroups + ((vc + 8 * g) >> 2)) : mx_codes8(v, inv);
          }
        }
        if (a.tiled) {
          if (col_in)
            *reinterpret_cast<uint4*>(col_tile + 128 * tc + (((col_chunk + blk) ^ (tc & 7)) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
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
// four rows a warp at once so that four loads are in flight.  Bound by HBM: 8192 x 5120 to BF16
// 21.6 us, 4.9 TB/s.
template <typename T>
__global__ void __launch_bounds__(kMxThreads) mxfp4_dequantize_kernel(const __grid_constant__ MxDequantArgs a) {
  __shared__ __align__(16) float turn[kMxThreads / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cp = (a.cols + 255) & ~int64_t(255);
  const int64_t segs = cp >> 8, groups = (a.rows + 3) >> 2, total = segs * groups;
  const int64_t row_bytes = (a.cols + 1) >> 1, row_blocks = (a.cols + 31) >> 5;
  for (int64_t t = (int64_t)blockIdx.x * (kMxThreads / 32) + warp; t < total; t += (int64_t)gridDim.x * (kMxThreads / 32)) {
    const int64_t rg = 4 * (t / segs), c = (t % segs) * 256 + 8 * lane;
    uint32_t w[4], byte[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = rg + i;
      w[i] = 0u;
      byte[i] = 0u;
      if (r >= a.rows || c >= a.cols) continue;
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
      T* y = static_cast<T*>(a.y) + r * a.ld;
      if (a.vec) {
        if (c + 8 <= a.cols) {
          uint4 o[MxIo<T>::kVec];
          MxIo<T>::pack(v, o);
#pragma unroll
          for (int k = 0; k < MxIo<T>::kVec; ++k) reinterpret_cast<uint4*>(y + c)[k] = o[k];
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.cols) y[c + k] = MxIo<T>::cast(v[k]);
        }
      } else {
        // rows that do not start on 16 bytes: neighbouring lanes store neighbouring elements
        __syncwarp();
        reinterpret_cast<float4*>(turn[warp])[2 * lane] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(turn[warp])[2 * lane + 1] = make_float4(v[4], v[5], v[6], v[7]);
        __syncwarp();
        const int64_t c0 = c - 8 * lane;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c0 + 32 * k + lane < a.cols) y[c0 + 32 * k + lane] = MxIo<T>::cast(turn[warp][32 * k + lane]);
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
  const auto starts_on = [&](uintptr_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0 && (rows == 1 || (uintptr_t)(ld * size) % n == 0); };
  a.vec = starts_on(32) ? 2 : starts_on(16) ? 1 : 0;
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
