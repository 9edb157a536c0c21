// Muon's Newton-Schulz step on thin matrices (at most kMuonThin = 32 rows in the working
// orientation: vectors, low-rank factors), sm_100a.
//
// Every iterate is a polynomial in A_0 = U U^T times U, X_k = T_k U, and the m x m matrices
// commute:  A = T U U^T T,  B = b A + c A^2,  S = a I + B,  T <- S T,  A <- S A S.
// So U is read twice whatever K is: once for U U^T (whose trace is ||U||_F^2), once for T U.
// The m x m part is in FP64: the iteration raises small singular values by up to a^K (485 for
// the Muon coefficients), and so the rounding of A_0.  With so few rows the tensor core's
// 256-row tile would be empty, and rounding errors do not average out over few elements: FP16
// operands were up to 5.5e-3 off on 2 x 3 matrices.
// Measured on 16 x 4096, 2000 x 16 and 1 x 513 together: 9.6, 10.3 and 9.5 us, all latency.
// Three launches: Gram matrices of 256-column chunks (summed in order: no atomics), one CTA per
// matrix for the iteration, the products T U.
#include <cstdint>

#include "muon_device.cuh"

namespace fs4 {
namespace {

constexpr int kThreads = 256;
static_assert(kMuonChunk == kThreads, "one column a thread");

// Rows r0 .. r0 + 7 of array element column c of an m x n working matrix (tall: stored n x m);
// absent ones are 0.  The eight loads are in flight together.
template <typename T>
__device__ __forceinline__ void column8(const void* p, int64_t ld, const MuonMat& d, int r0, int64_t c, float* v) {
  const T* q = static_cast<const T*>(p);
  T raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i < d.m && c < d.n) raw[i] = d.tall ? q[c * ld + r0 + i] : q[(int64_t)(r0 + i) * ld + c];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (r0 + i < d.m && c < d.n) ? to_f32(raw[i]) : 0.0f;
}
__device__ __forceinline__ void column8_of(const void* p, int64_t ld, int type, const MuonMat& d, int r0, int64_t c, float* v) {
  if (type == kTypeF32) column8<float>(p, ld, d, r0, c, v);
  else if (type == kTypeBf16) column8<__nv_bfloat16>(p, ld, d, r0, c, v);
  else column8<__half>(p, ld, d, r0, c, v);
}
// The same of U.
__device__ __forceinline__ void direction_column8(const MuonCall& p, const MuonMat& d, int r0, int64_t c, float* v) {
  column8_of(d.g, d.ldg, d.tg, d, r0, c, v);
  if (!d.mom) return;
  float m[8];
  column8_of(d.mom, d.ldm, d.tm, d, r0, c, m);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = direction(p, m[i], v[i]);
}

// Entries in 2 x 2 blocks on and above the diagonal; the threads left over by few blocks share
// the columns.
__global__ void __launch_bounds__(kThreads) muon_thin_gram_kernel(const __grid_constant__ MuonCall p) {
  __shared__ float u[kMuonThin][kMuonChunk + 1];
  __shared__ double sums[kThreads][4];
  const MuonTable& t = *muon_table(p.ws);
  const int mi = owner_of(t.prefix[kUnitsThin], p.count, blockIdx.x);
  const MuonMat& d = t.mat[mi];
  const int32_t chunk = blockIdx.x - t.prefix[kUnitsThin][mi];
  const int m = d.m, mb = (m + 1) / 2, blocks = mb * (mb + 1) / 2, shares = kThreads / blocks;
  for (int r = 0; r < m; r += 8) {
    float v[8];
    direction_column8(p, d, r, (int64_t)chunk * kMuonChunk + threadIdx.x, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[r + i][threadIdx.x] = v[i];      // rows past m are 0
  }
  __syncthreads();
  const int block = threadIdx.x % blocks, share = threadIdx.x / blocks;
  int j = 0, i = block;                       // block (i, j), i <= j
  while (i > j) i -= ++j;
  if (share < shares) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int c = share; c < kMuonChunk; c += shares) {
      const double a0 = u[2 * i][c], a1 = u[2 * i + 1][c], b0 = u[2 * j][c], b1 = u[2 * j + 1][c];
      s[0] += a0 * b0;
      s[1] += a0 * b1;
      s[2] += a1 * b0;
      s[3] += a1 * b1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sums[threadIdx.x][k] = s[k];
  }
  __syncthreads();
  double* out = reinterpret_cast<double*>(p.ws + d.base + thin_gram_offset(m)) + (int64_t)chunk * m * m;
  if (threadIdx.x < blocks) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      double s = 0.0;
      for (int h = 0; h < shares; ++h) s += sums[h * blocks + threadIdx.x][k];
      const int r = 2 * i + (k >> 1), c = 2 * j + (k & 1);
      if (r < m && c < m) {
        out[r * m + c] = s;
        out[c * m + r] = s;
      }
    }
  }
}

__global__ void __launch_bounds__(1024) muon_thin_iterate_kernel(const __grid_constant__ MuonCall p) {
  __shared__ double A[kMuonThin][kMuonThin + 1], S[kMuonThin][kMuonThin + 1], T[kMuonThin][kMuonThin + 1], W[kMuonThin][kMuonThin + 1];
  const MuonMat& d = muon_table(p.ws)->mat[blockIdx.x];
  const int m = d.m;
  if (m > kMuonThin) return;
  uint8_t* ws = p.ws + d.base;
  const int i = threadIdx.x / m, j = threadIdx.x % m;
  const bool mine = (int)threadIdx.x < m * m;
  const int64_t chunks = thin_chunks(d.n);
  if (mine) {
    const double* g = reinterpret_cast<const double*>(ws + thin_gram_offset(m)) + threadIdx.x;
    double s = 0.0;
    for (int64_t c = 0; c < chunks; ++c) s += g[c * m * m];
    A[i][j] = s;
  }
  __syncthreads();
  double trace = 0.0;
  for (int t = 0; t < m; ++t) trace += A[t][t];
  const bool fine = isfinite(trace);
  const double inv = fine ? 1.0 / (sqrt(trace) + 1e-7) : 0.0;
  __syncthreads();
  if (mine) {
    A[i][j] = fine ? A[i][j] * inv * inv : 0.0;
    T[i][j] = i == j ? inv : 0.0;
  }
  __syncthreads();
  // one product: row i of x times column j of y
  auto dot = [&](const double (*x)[kMuonThin + 1], const double (*y)[kMuonThin + 1]) -> double {
    double s = 0.0, r = 0.0;          // two chains
    int t = 0;
#pragma unroll 4
    for (; t + 1 < m; t += 2) {
      s += x[i][t] * y[t][j];
      r += x[i][t + 1] * y[t + 1][j];
    }
    if (t < m) s += x[i][t] * y[t][j];
    return s + r;
  };
  for (int it = 0; it < p.K; ++it) {
    const float* c = p.coeffs + (p.n_coeffs == 1 ? 0 : 3 * it);
    if (mine) S[i][j] = (double)c[1] * A[i][j] + (double)c[2] * dot(A, A) + (i == j ? (double)c[0] : 0.0);
    __syncthreads();
    double t = 0.0;
    if (mine) {
      t = dot(S, T);
      W[i][j] = dot(S, A);
    }
    __syncthreads();
    if (mine) {
      T[i][j] = t;
      A[i][j] = dot(W, S);
    }
    __syncthreads();
  }
  // T holds 1 / ||U||: beside a norm near FP32's largest values it is stored times 2^64, which keeps
  // it a normal number, and the products T U are taken times 2^-64
  const bool large = inv < 0x1p-100;
  if (mine) reinterpret_cast<float*>(ws)[threadIdx.x] = fine ? (float)(large ? T[i][j] * 0x1p64 : T[i][j]) : 0.0f;
  if (threadIdx.x == 0) {
    *reinterpret_cast<float*>(ws + thin_flag_offset(m)) = !fine ? 0.0f : large ? 0x1p-64f : 1.0f;
    if (!fine) atomicOr(muon_status(p.ws), kStatusNonFinite);
  }
}

// One column of X_K a thread: T U, T's rows read by all threads at once.
__global__ void __launch_bounds__(kThreads) muon_thin_apply_kernel(const __grid_constant__ MuonCall p) {
  __shared__ __align__(16) float T[kMuonThin][kMuonThin];
  const MuonTable& t = *muon_table(p.ws);
  const int mi = owner_of(t.prefix[kUnitsThin], p.count, blockIdx.x);
  const MuonMat& d = t.mat[mi];
  const int64_t c = (int64_t)(blockIdx.x - t.prefix[kUnitsThin][mi]) * kMuonChunk + threadIdx.x;
  const int m = d.m;
  const uint8_t* ws = p.ws + d.base;
  for (int e = threadIdx.x; e < kMuonThin * kMuonThin; e += kThreads) {
    const int i = e / kMuonThin, j = e % kMuonThin;
    T[i][j] = (i < m && j < m) ? reinterpret_cast<const float*>(ws)[i * m + j] : 0.0f;
  }
  const float shift = *reinterpret_cast<const float*>(ws + thin_flag_offset(m));
  const bool fine = shift != 0.0f;
  float u[kMuonThin];
#pragma unroll
  for (int r = 0; r < kMuonThin; r += 8) {
    if (r < m) {
      direction_column8(p, d, r, c, u + r);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[r + i] = 0.0f;
    }
  }
  __syncthreads();
  if (c >= d.n) return;
  const bool blend = p.rate >= 0.0f;
  bool bad = false;
  for (int i0 = 0; i0 < m; i0 += 8) {
    float w[8], s[8];
    if (blend) column8_of(d.w, d.ldw, d.tw, d, i0, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = 0.0f;
#pragma unroll
      for (int j = 0; j < kMuonThin; j += 4) {
        if (j >= m) break;
        const float4 q = *reinterpret_cast<const float4*>(&T[i0 + i][j]);
        s[i] = fmaf(q.x, u[j], s[i]);
        s[i] = fmaf(q.y, u[j + 1], s[i]);
        s[i] = fmaf(q.z, u[j + 2], s[i]);
        s[i] = fmaf(q.w, u[j + 3], s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i >= m) break;
      const float v = fine ? s[i] * shift * d.scale : 0.0f;
      bad |= !isfinite(v);
      const int64_t at = d.tall ? c * d.ldw + i0 + i : (int64_t)(i0 + i) * d.ldw + c;
      put1(d.w, at, d.tw, blend ? fmaf(-p.rate, v, p.keep * w[i]) : v);
    }
  }
  if (bad) atomicOr(muon_status(p.ws), kStatusNonFinite);
}

}  // namespace

cudaError_t launch_muon_thin(const MuonCall& c, int32_t units, cudaStream_t st) {
  muon_thin_gram_kernel<<<(unsigned)units, kThreads, 0, st>>>(c);
  muon_thin_iterate_kernel<<<(unsigned)c.count, kMuonThin * kMuonThin, 0, st>>>(c);
  muon_thin_apply_kernel<<<(unsigned)units, kThreads, 0, st>>>(c);
  return cudaGetLastError();
}

}  // namespace fs4
