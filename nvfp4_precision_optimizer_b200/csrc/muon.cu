// Element-wise kernels of the Muon step (sm_100a):
//   moment   M <- beta M + (1 - beta) G (in FP32, rounded to M's type), and partial sums of
//            squares of the update direction U = M, or beta M + (1 - beta) G with Nesterov
//            (of U = G without a momentum)
//   prepare  X_0 = U / (||U||_F + 1e-7), transposed for a tall matrix, as high and low FP16
//            parts in the tensor core's layout, zero padded
// The norm is a sum of float64 partials in a fixed order (no atomics), so a step repeats bit
// for bit.  A matrix whose norm is not finite gets X_0 = 0 and sets the status word: its
// update is zero.  Both kernels are bound by HBM: moment reads G and M and writes M, prepare
// reads them again and writes 4 bytes an element.  Loads of four 8-element pieces are issued
// before the first is used.  Measured on seven 2048-wide matrices (67 M elements, BF16 gradient, FP32
// momentum): moment 122 us (5.5 TB/s), prepare 140 us (4.8 TB/s).
#include <cstdint>

#include "muon_device.cuh"

namespace fs4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;      // 8-element pieces in flight a thread

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

// Sum of eight squares, in FP64 where FP32 could overflow or lose small ones.
__device__ __forceinline__ double squares8(const float* u) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s = fmaf(u[k], u[k], s);
    m = fmaxf(m, fabsf(u[k]));
  }
  if (m < 1e18f && (m > 1e-15f || m == 0.0f) && s == s) return (double)s;
  double e = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) e += (double)u[k] * (double)u[k];
  return e;
}

// Unit u of a matrix: whole rows of G.  CTA 0 also leaves the table
// in the workspace and resets the status word and the iterate kernel's counts.
template <int N>
__global__ void __launch_bounds__(kThreads, 2) muon_moment_kernel(const __grid_constant__ MuonCall p,
                                                               const __grid_constant__ MuonTableN<N> t) {
  __shared__ double red[kThreads / 32];
  if (blockIdx.x == 0) {
    MuonTable* out = muon_table(p.ws);
    for (int i = threadIdx.x; i < kUnitKinds * (p.count + 1); i += kThreads)
      out->prefix[i / (p.count + 1)][i % (p.count + 1)] = t.prefix[i / (p.count + 1)][i % (p.count + 1)];
    for (int i = threadIdx.x; i < p.count; i += kThreads) out->mat[i] = t.mat[i];
    for (int i = threadIdx.x; i < p.counts; i += kThreads) reinterpret_cast<uint32_t*>(p.ws + p.counts_at)[i] = 0u;
    for (int i = threadIdx.x; i < p.count; i += kThreads) muon_counts(p.ws)[i] = 0u;
    if (threadIdx.x == 0) *muon_status(p.ws) = 0u;
  }
  const int32_t u = blockIdx.x;
  if (u >= t.prefix[kUnitsMoment][p.count]) return;
  const int mi = owner_of(t.prefix[kUnitsMoment], p.count, u);
  const MuonMat& d = t.mat[mi];
  const int32_t part = u - t.prefix[kUnitsMoment][mi];
  const int32_t grows = d.tall ? d.n : d.m, gcols = d.tall ? d.m : d.n;
  const int32_t per = (grows + d.parts - 1) / d.parts;
  const int32_t r0 = part * per, r1 = min(r0 + per, grows);
  const bool vec = gcols % 8 == 0 && aligned16(d.g, d.ldg, d.tg) && (!d.mom || aligned16(d.mom, d.ldm, d.tm));
  double sum = 0.0;
  if (vec) {
    // rows without gaps need no division into rows and columns
    const bool flat = d.ldg == gcols && (!d.mom || d.ldm == gcols);
    const int32_t width = gcols / 8, count = (r1 - r0) * width;
    auto at = [&](int32_t i, int64_t ld) -> int64_t {
      return flat ? (int64_t)r0 * gcols + 8ll * i : (r0 + i / width) * ld + 8 * (i % width);
    };
    for (int32_t i0 = threadIdx.x; i0 < count; i0 += kAhead * kThreads) {
      Raw8 g[kAhead], m[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int32_t i = i0 + s * kThreads;
        if (i < count) {
          g[s] = load8(d.g, at(i, d.ldg), d.tg);
          if (d.mom) m[s] = load8(d.mom, at(i, d.ldm), d.tm);
        }
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int32_t i = i0 + s * kThreads;
        if (i < count) {
          float u[8];
          unpack8(g[s], d.tg, u);
          if (d.mom) {
            float v[8];
            unpack8(m[s], d.tm, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = fmaf(p.beta, v[k], p.rest * u[k]);
            put8(d.mom, at(i, d.ldm), d.tm, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = direction(p, v[k], u[k]);
          }
          sum += squares8(u);
        }
      }
    }
  } else {
    const bool flat = d.ldg == gcols && (!d.mom || d.ldm == gcols);
    const int32_t count = (r1 - r0) * gcols;
    for (int32_t i0 = threadIdx.x; i0 < count; i0 += 8 * kThreads) {
      int64_t ag[8], am[8];
      float g[8], m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int32_t i = i0 + k * kThreads;
        const int64_t r = flat ? r0 : r0 + i / gcols, c = flat ? i : i % gcols;
        ag[k] = i < count ? r * d.ldg + c : -1;
        am[k] = i < count ? r * d.ldm + c : -1;
      }
      gather8(d.g, d.tg, ag, g);
      if (d.mom) {
        gather8(d.mom, d.tm, am, m);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (am[k] < 0) continue;
          m[k] = put1(d.mom, am[k], d.tm, fmaf(p.beta, m[k], p.rest * g[k]));
          g[k] = direction(p, m[k], g[k]);
        }
      }
      sum += squares8(g);
    }
  }
  const double s = block_sum(sum, red);
  if (threadIdx.x == 0) muon_partials(p.ws)[d.partial + part] = s;
}

// Eight elements of U that may be absent or off a 16-byte boundary: out of line, so that its
// registers do not crowd the aligned case.
struct Eight {
  float v[8];
};
__device__ __noinline__ Eight guarded_direction8(const MuonCall& p, const MuonMat& d, int64_t r, int64_t c, int64_t rows, int64_t cols) {
  Eight x;
  int64_t at[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) at[k] = (r < rows && c + k < cols) ? r * d.ldg + c + k : -1;
  gather8(d.g, d.tg, at, x.v);
  if (d.mom) {
    float m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) at[k] = (r < rows && c + k < cols) ? r * d.ldm + c + k : -1;
    gather8(d.mom, d.tm, at, m);
#pragma unroll
    for (int k = 0; k < 8; ++k) x.v[k] = direction(p, m[k], x.v[k]);
  }
  return x;
}

// Persistent, a contiguous range of 128 x 64 tiles of X_0 a CTA.  A tall matrix's tile turns in
// shared memory: element (c, r) of G at word r ^ 4 (c / 8 % 8) of row c, so that the reads of
// eight c at one r take different banks.
__global__ void __launch_bounds__(kThreads, 2) muon_prepare_kernel(const __grid_constant__ MuonCall p) {
  __shared__ double red[kThreads / 32];
  __shared__ __align__(16) float turn[64 * 128];
  const MuonTable& t = *muon_table(p.ws);
  const int32_t* prefix = t.prefix[kUnitsPrepare];
  const int32_t total = prefix[p.count];
  const int32_t per = (total + gridDim.x - 1) / gridDim.x;
  int32_t u = blockIdx.x * per;
  const int32_t end = min(u + per, total);
  if (u >= end) return;
  int mi = owner_of(prefix, p.count, u) - 1;
  MuonMat d{};
  float inv = 0.0f;
  int32_t next = u;
  for (; u < end; ++u) {
    if (u == next) {      // the next matrix (those without tiles here have empty ranges)
      do ++mi; while (prefix[mi + 1] <= u);
      next = prefix[mi + 1];
      d = t.mat[mi];
      const double* part = muon_partials(p.ws) + d.partial;
      double s = 0.0;
      for (int i = threadIdx.x; i < d.parts; i += kThreads) s += part[i];
      s = block_sum(s, red);
      const bool fine = isfinite(s);
      inv = fine ? (float)(kXScale / (sqrt(s) + 1e-7)) : -1.0f;   // -1: carried as zeros
      if (!fine && threadIdx.x == 0) atomicOr(muon_status(p.ws), kStatusNonFinite);
    }
    const int32_t tu = u - prefix[mi], across = d.np / 64;
    const int64_t r0 = (int64_t)(tu / across) * 128, c0 = (int64_t)(tu % across) * 64;
    const MuonLayout L = muon_layout(d.mp, d.np);
    uint8_t* hi = p.ws + d.base + L.x[0];
    uint8_t* lo = p.ws + d.base + L.xl;
    const bool vec = aligned16(d.g, d.ldg, d.tg) && (!d.mom || aligned16(d.mom, d.ldm, d.tm));
    // rows and columns of G that piece s reads: 128 rows x 8 pieces, or, tall (G is n x m: rows
    // c0 .., columns r0 ..), 64 rows x 16 pieces
    const int64_t grows = d.tall ? d.n : d.m, gcols = d.tall ? d.m : d.n;
    auto row_of = [&](int q) -> int64_t { return d.tall ? c0 + (q >> 4) : r0 + (q >> 3); };
    auto col_of = [&](int q) -> int64_t { return d.tall ? r0 + 8 * (q & 15) : c0 + 8 * (q & 7); };
    float x[kAhead][8];
    // tiles inside the matrix, on 16-byte boundaries: all loads first
    if (vec && r0 + 128 <= d.m && c0 + 64 <= d.n) {
      Raw8 g[kAhead], m[kAhead];
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int q = threadIdx.x + s * kThreads;
        g[s] = load8(d.g, row_of(q) * d.ldg + col_of(q), d.tg);
        if (d.mom) m[s] = load8(d.mom, row_of(q) * d.ldm + col_of(q), d.tm);
      }
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        unpack8(g[s], d.tg, x[s]);
        if (d.mom) {
          float v[8];
          unpack8(m[s], d.tm, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[s][k] = direction(p, v[k], x[s][k]);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int q = threadIdx.x + s * kThreads;
        const Eight e = guarded_direction8(p, d, row_of(q), col_of(q), grows, gcols);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[s][k] = e.v[k];
      }
    }
    if (d.tall) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int q = threadIdx.x + s * kThreads, c = q >> 4, r = 8 * (q & 15), sw = 4 * ((c >> 3) & 7);
        *reinterpret_cast<float4*>(turn + 128 * c + (r ^ sw)) = make_float4(x[s][0], x[s][1], x[s][2], x[s][3]);
        *reinterpret_cast<float4*>(turn + 128 * c + ((r + 4) ^ sw)) = make_float4(x[s][4], x[s][5], x[s][6], x[s][7]);
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int q = threadIdx.x + s * kThreads, r = q >> 3, c = 8 * (q & 7);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[s][k] = turn[128 * (c + k) + (r ^ (4 * (q & 7)))];
      }
    }
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int q = threadIdx.x + s * kThreads;
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = inv < 0.0f ? 0.0f : x[s][k] * inv;
      uint4 h, l;
      split8(y, h, l);
      const int64_t off = tiled_chunk_offset_bf16(r0 + (q >> 3), c0 + 8 * (q & 7), d.np);
      *reinterpret_cast<uint4*>(hi + off) = h;
      *reinterpret_cast<uint4*>(lo + off) = l;
    }
  }
}

}  // namespace

cudaError_t launch_muon_moment(const MuonCall& c, const MuonTable& t, cudaStream_t st) {
  const int32_t units = t.prefix[kUnitsMoment][c.count];
  const unsigned grid = (unsigned)(units > 0 ? units : 1);
  if (c.count <= kMuonFew) {
    MuonTableN<kMuonFew> few;
    for (int k = 0; k < kUnitKinds; ++k)
      for (int i = 0; i <= kMuonFew; ++i) few.prefix[k][i] = t.prefix[k][i < c.count ? i : c.count];
    for (int i = 0; i < kMuonFew; ++i) few.mat[i] = t.mat[i < c.count ? i : 0];
    muon_moment_kernel<kMuonFew><<<grid, kThreads, 0, st>>>(c, few);
  } else {
    muon_moment_kernel<kMuonMaxBatch><<<grid, kThreads, 0, st>>>(c, t);
  }
  return cudaGetLastError();
}

cudaError_t launch_muon_prepare(const MuonCall& c, int32_t units, cudaStream_t st, int num_sms) {
  const int most = 4 * num_sms;
  muon_prepare_kernel<<<(unsigned)(units < most ? units : most), kThreads, 0, st>>>(c);
  return cudaGetLastError();
}

}  // namespace fs4
