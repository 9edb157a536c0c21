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
// Three launches: Gram matrices of 256-column chunks (summed in order: no atomics), one CTA per
// matrix for the iteration, the products T U.
#include <cstdint>

#include "muon_device.cuh"

namespace fs4 {
namespace {

constexpr int kThreads = 256;
static_assert(kMuonChunk == kThreads, "one column a thread");

// U's columns c0 .. c0 + 255 into u[row][column].
__device__ __forceinline__ void load_chunk(const MuonCall& p, const MuonMat& d, int64_t c0, float (*u)[kMuonChunk + 1]) {
  const int count = d.m * kMuonChunk;
  for (int i = threadIdx.x; i < count; i += kThreads) {
    // neighbouring threads read neighbouring elements of G
    const int r = d.tall ? i % d.m : i / kMuonChunk, c = d.tall ? i / d.m : i % kMuonChunk;
    float v = 0.0f;
    if (c0 + c < d.n) v = d.tall ? direction_at(p, d, c0 + c, r) : direction_at(p, d, r, c0 + c);
    u[r][c] = v;
  }
}

__global__ void __launch_bounds__(kThreads) muon_thin_gram_kernel(const __grid_constant__ MuonCall p) {
  __shared__ float u[kMuonThin][kMuonChunk + 1];
  const MuonTable& t = *muon_table(p.ws);
  const int mi = owner_of(t.prefix[kUnitsThin], p.count, blockIdx.x);
  const MuonMat& d = t.mat[mi];
  const int32_t chunk = blockIdx.x - t.prefix[kUnitsThin][mi];
  load_chunk(p, d, (int64_t)chunk * kMuonChunk, u);
  __syncthreads();
  double* out = reinterpret_cast<double*>(p.ws + d.base + thin_gram_offset(d.m)) + (int64_t)chunk * d.m * d.m;
  for (int e = threadIdx.x; e < d.m * d.m; e += kThreads) {
    const int i = e / d.m, j = e % d.m;
    double s = 0.0;
    for (int c = 0; c < kMuonChunk; ++c) s += (double)u[i][c] * (double)u[j][c];
    out[e] = s;
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
    double s = 0.0;
    for (int t = 0; t < m; ++t) s += x[i][t] * y[t][j];
    return s;
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
  if (mine) reinterpret_cast<float*>(ws)[threadIdx.x] = fine ? (float)T[i][j] : 0.0f;
  if (threadIdx.x == 0) {
    *reinterpret_cast<float*>(ws + thin_flag_offset(m)) = fine ? 1.0f : 0.0f;
    if (!fine) atomicOr(muon_status(p.ws), kStatusNonFinite);
  }
}

__global__ void __launch_bounds__(kThreads) muon_thin_apply_kernel(const __grid_constant__ MuonCall p) {
  __shared__ float u[kMuonThin][kMuonChunk + 1];
  __shared__ float T[kMuonThin][kMuonThin];
  const MuonTable& t = *muon_table(p.ws);
  const int mi = owner_of(t.prefix[kUnitsThin], p.count, blockIdx.x);
  const MuonMat& d = t.mat[mi];
  const int64_t c0 = (int64_t)(blockIdx.x - t.prefix[kUnitsThin][mi]) * kMuonChunk;
  const uint8_t* ws = p.ws + d.base;
  const bool fine = *reinterpret_cast<const float*>(ws + thin_flag_offset(d.m)) != 0.0f;
  for (int e = threadIdx.x; e < d.m * d.m; e += kThreads) T[e / d.m][e % d.m] = reinterpret_cast<const float*>(ws)[e];
  load_chunk(p, d, c0, u);
  __syncthreads();
  // X_K of this thread's column, in place of U's
  float x[kMuonThin];
#pragma unroll
  for (int i = 0; i < kMuonThin; ++i) {
    if (i >= d.m) break;
    float s = 0.0f;
    for (int j = 0; j < d.m; ++j) s = fmaf(T[i][j], u[j][threadIdx.x], s);
    x[i] = s;
  }
#pragma unroll
  for (int i = 0; i < kMuonThin; ++i)
    if (i < d.m) u[i][threadIdx.x] = x[i];
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < d.m * kMuonChunk; i += kThreads) {
    const int r = d.tall ? i % d.m : i / kMuonChunk, c = d.tall ? i / d.m : i % kMuonChunk;
    if (c0 + c >= d.n) continue;
    const float v = fine ? u[r][c] * d.scale : 0.0f;
    bad |= !isfinite(v);
    const int64_t at = d.tall ? (c0 + c) * d.ldw + r : r * d.ldw + c0 + c;
    put1(d.w, at, d.tw, p.rate < 0.0f ? v : fmaf(-p.rate, v, p.keep * get1(d.w, at, d.tw)));
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
