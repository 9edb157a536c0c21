// Element-wise kernels of the Muon step (sm_100a):
//   moment   M <- beta M + (1 - beta) G (in FP32, rounded to M's type), and partial sums of
//            squares of the update direction U = M, or beta M + (1 - beta) G with Nesterov
//            (of U = G without a momentum)
//   prepare  X_0 = U / (||U||_F + 1e-7), transposed for a tall matrix, as high and low FP16
//            parts in the tensor core's layout, zero padded
// The norm is a sum of float64 partials in a fixed order (no atomics), so a step repeats bit
// for bit.  A matrix whose norm is not finite gets X_0 = 0 and sets the status word: its
// update is zero.  Both kernels are bound by HBM: moment reads G and M and writes M, prepare
// reads them again and writes 4 bytes an element.
#include <cstdint>

#include "muon_device.cuh"

namespace fs4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

// Unit u of a matrix: `rows` whole rows of G, about kMuonUnit elements.
__global__ void __launch_bounds__(kThreads) muon_moment_kernel(const __grid_constant__ MuonParams p) {
  __shared__ double red[kThreads / 32];
  const int32_t u = blockIdx.x;
  const MuonMat& d = p.mat[owner_of(p.prefix, p.count, u)];
  const int32_t part = u - p.prefix[owner_of(p.prefix, p.count, u)];
  const int64_t grows = d.tall ? d.n : d.m, gcols = d.tall ? d.m : d.n;
  const int64_t per = (grows + d.parts - 1) / d.parts;
  const int64_t r0 = part * per, r1 = r0 + per < grows ? r0 + per : grows;
  const bool vec = gcols % 8 == 0 && aligned16(d.g, d.ldg, d.tg) && (!d.mom || aligned16(d.mom, d.ldm, d.tm));
  double sum = 0.0;
  if (r0 < r1) {
    const int64_t width = vec ? gcols / 8 : gcols, count = (r1 - r0) * width;
    for (int64_t i = threadIdx.x; i < count; i += kThreads) {
      const int64_t r = r0 + i / width, c = i % width;
      if (vec) {
        float g[8], m[8];
        get8(d.g, r * d.ldg + 8 * c, d.tg, g);
        if (d.mom) {
          get8(d.mom, r * d.ldm + 8 * c, d.tm, m);
#pragma unroll
          for (int k = 0; k < 8; ++k) m[k] = fmaf(p.beta, m[k], p.rest * g[k]);
          put8(d.mom, r * d.ldm + 8 * c, d.tm, m);
#pragma unroll
          for (int k = 0; k < 8; ++k) g[k] = direction(p, m[k], g[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += (double)g[k] * (double)g[k];
      } else {
        float g = get1(d.g, r * d.ldg + c, d.tg);
        if (d.mom) {
          const float m = put1(d.mom, r * d.ldm + c, d.tm,
                              fmaf(p.beta, get1(d.mom, r * d.ldm + c, d.tm), p.rest * g));
          g = direction(p, m, g);
        }
        sum += (double)g * (double)g;
      }
    }
  }
  const double s = block_sum(sum, red);
  if (threadIdx.x == 0) p.partials[d.partial + part] = s;
}

// Persistent; one 128 x 64 tile of X_0 at a time.
__global__ void __launch_bounds__(kThreads) muon_prepare_kernel(const __grid_constant__ MuonParams p) {
  __shared__ double red[kThreads / 32];
  __shared__ float turn[64][129];
  const int32_t total = p.prefix[p.count];
  const int32_t per = (total + gridDim.x - 1) / gridDim.x;
  int32_t u = blockIdx.x * per;
  const int32_t end = u + per < total ? u + per : total;
  int cur = -1;
  float inv = 0.0f;
  for (; u < end; ++u) {
    const int mi = owner_of(p.prefix, p.count, u);
    const MuonMat& d = p.mat[mi];
    if (mi != cur) {
      cur = mi;
      double s = 0.0;
      for (int i = threadIdx.x; i < d.parts; i += kThreads) s += p.partials[d.partial + i];
      s = block_sum(s, red);
      const bool fine = isfinite(s);
      inv = fine ? (float)(1.0 / (sqrt(s) + 1e-7)) * kXScale : 0.0f;
      if (!fine && threadIdx.x == 0) atomicOr(p.status, kStatusNonFinite);
      if (!fine) inv = -1.0f;      // the matrix is carried as zeros
    }
    const int32_t t = u - p.prefix[mi], across = d.np / 64;
    const int64_t r0 = (int64_t)(t / across) * 128, c0 = (int64_t)(t % across) * 64;
    const MuonLayout L = muon_layout(d.mp, d.np);
    uint8_t* hi = p.ws + d.base + L.x[0];
    uint8_t* lo = p.ws + d.base + L.xl;
    const bool vec = !d.tall && aligned16(d.g, d.ldg, d.tg) && (!d.mom || aligned16(d.mom, d.ldm, d.tm));
    if (d.tall) {
      __syncthreads();
      // G is n x m: its rows c0.. and columns r0.. land transposed
      for (int i = threadIdx.x; i < 64 * 128; i += kThreads) {
        const int64_t c = c0 + (i >> 7), r = r0 + (i & 127);
        turn[i >> 7][i & 127] = (c < d.n && r < d.m) ? direction_at(p, d, c, r) : 0.0f;
      }
      __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int q = threadIdx.x + s * kThreads;        // 128 rows x 8 chunks
      const int64_t r = r0 + (q >> 3), c = c0 + 8 * (q & 7);
      float x[8];
      if (d.tall) {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = turn[8 * (q & 7) + k][q >> 3];
      } else if (vec && r < d.m && c + 8 <= d.n) {
        get8(d.g, r * d.ldg + c, d.tg, x);
        if (d.mom) {
          float m[8];
          get8(d.mom, r * d.ldm + c, d.tm, m);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = direction(p, m[k], x[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = (r < d.m && c + k < d.n) ? direction_at(p, d, r, c + k) : 0.0f;
      }
      uint32_t h[4], l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = inv < 0.0f ? 0.0f : x[2 * k] * inv, b = inv < 0.0f ? 0.0f : x[2 * k + 1] * inv;
        const __half2 hh = __floats2half2_rn(a, b);
        h[k] = *reinterpret_cast<const uint32_t*>(&hh);
        const __half2 ll = __floats2half2_rn((a - half_lo(h[k])) * kLowScale, (b - half_hi(h[k])) * kLowScale);
        l[k] = *reinterpret_cast<const uint32_t*>(&ll);
      }
      const int64_t off = tiled_chunk_offset_bf16(r, c, d.np);
      *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

}  // namespace

cudaError_t launch_muon_moment(const MuonParams& p, cudaStream_t st, int num_sms) {
  muon_moment_kernel<<<(unsigned)p.prefix[p.count], kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_muon_prepare(const MuonParams& p, cudaStream_t st, int num_sms) {
  const int total = p.prefix[p.count], most = 4 * num_sms;
  muon_prepare_kernel<<<(unsigned)(total < most ? total : most), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace fs4
