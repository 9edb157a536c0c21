// Internal definitions shared by the Muon kernels and their C entry points.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_internal.h"

namespace fs4 {

constexpr int kMuonMaxBatch = 224;      // matrices per call (kernel-parameter table size)
constexpr int64_t kMuonHeader = 256;    // byte 0 of the workspace: the status word
constexpr int kMuonPad = 256;           // working dimensions are padded to multiples of 256
constexpr int64_t kMuonUnit = 16384;    // elements of one partial sum of squares, about

// Matrices with at most this many rows (working orientation) take the thin kernels (muon_thin.cu).
constexpr int kMuonThin = 32;
constexpr int kMuonChunk = 256;         // columns of one unit of the thin kernels

// FP16 operands hold value * 2^k, and a low part holds what the high part lost * 2^11 more:
// X has elements of at most about 1.2 and of 1 / sqrt(n) typically, A and B of a few units.
constexpr float kXScale = 4096.0f, kAScale = 256.0f, kLowScale = 2048.0f;

// One matrix.  The working X is G or, for a tall G, G^T: m x n with m <= n.
struct MuonMat {
  const void* g;
  void* mom;               // momentum, or null (orthogonalise only)
  void* w;                 // weights (updated in place), or the output
  int64_t ldg, ldm, ldw;
  int64_t base;            // its block in the workspace, bytes
  int64_t partial;         // index of its first partial sum
  int32_t m, n, mp, np;
  int32_t tall;
  int32_t parts;           // number of partial sums
  int8_t tg, tm, tw, pad;  // element types
  float scale;             // the update is scale * X_K
};

// Byte offsets inside a matrix's block: X high parts (two, by iteration parity) and low part,
// A high and low, B, then the diagonals of A and B (FP32).  Matrices in the TILED BF16 layout
// of include/fs4.h, FP16 elements.
struct MuonLayout {
  int64_t x[2], xl, a, al, b, da, db, end;
};
__host__ __device__ inline MuonLayout muon_layout(int64_t mp, int64_t np) {
  MuonLayout L;
  const int64_t xn = 2 * mp * np, aa = 2 * mp * mp;
  L.x[0] = 0;
  L.x[1] = xn;
  L.xl = 2 * xn;
  L.a = 3 * xn;
  L.al = L.a + aa;
  L.b = L.al + aa;
  L.da = L.b + aa;
  L.db = L.da + 4 * mp;
  L.end = L.db + 4 * mp;
  return L;
}

// A thin matrix's block: T (m x m FP32), a flag (FP32, 1 if the norm is finite), then one m x m
// FP64 Gram matrix per chunk of columns.
__host__ __device__ inline int64_t thin_flag_offset(int64_t m) { return 4 * m * m; }
__host__ __device__ inline int64_t thin_gram_offset(int64_t m) { return (4 * m * m + 4 + 255) / 256 * 256; }
__host__ __device__ inline int64_t thin_chunks(int64_t n) { return (n + kMuonChunk - 1) / kMuonChunk; }
__host__ __device__ inline int64_t thin_bytes(int64_t m, int64_t n) { return thin_gram_offset(m) + 8 * m * m * thin_chunks(n); }

struct MuonParams {
  int32_t count;
  int32_t slot;            // X's current high part
  int32_t last;            // the last update: write the weights or the output
  int32_t nesterov;
  float a, b, c;           // this iteration's polynomial
  float beta, rest;        // momentum and 1 - momentum
  float keep, rate;        // weights <- keep * weights - rate * scale * X_K; rate < 0: output = scale * X_K
  uint32_t* status;
  double* partials;
  uint8_t* ws;
  int32_t prefix[kMuonMaxBatch + 1];
  MuonMat mat[kMuonMaxBatch];
};
static_assert(sizeof(MuonParams) <= 32000, "kernel parameter block too large");

enum class MuonProduct : int { GramX = 0, GramA = 1, Update = 2 };

cudaError_t launch_muon_moment(const MuonParams& p, cudaStream_t st, int num_sms);
cudaError_t launch_muon_prepare(const MuonParams& p, cudaStream_t st, int num_sms);
// Thin matrices: Gram matrices, the iteration on them (coeffs: K or one triple), the result.
struct MuonCoeffs {
  int32_t K, n;
  float v[3 * FS4_MAX_ITERS];
};
cudaError_t launch_muon_thin(const MuonParams& p, const MuonCoeffs& c, cudaStream_t st);
cudaError_t launch_muon_product(MuonProduct e, const MuonParams& p, cudaStream_t st, int num_sms);

}  // namespace fs4
