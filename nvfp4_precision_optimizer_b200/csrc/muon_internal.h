// Internal definitions shared by the Muon kernels and their C entry points.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "mx_internal.h"

namespace fs4 {

constexpr int kMuonMaxBatch = 224;      // matrices per call
constexpr int kMuonFew = 8;             // calls of at most this many pass a small parameter block
constexpr int kMuonPad = 256;           // working dimensions are padded to multiples of 256
constexpr int64_t kMuonUnit = 4096;     // least elements of one partial sum of squares
constexpr int64_t kMuonParts = 1184;    // about the most partial sums of a matrix (8 CTAs an SM)

// Matrices with at most this many rows (working orientation) take the thin kernels (muon_thin.cu).
constexpr int kMuonThin = 32;
constexpr int kMuonChunk = 256;         // columns of one unit of the thin kernels

// FP16 operands hold value * 2^k: X has elements of at most about 1.2 and of 1 / sqrt(n)
// typically, A and B of a few units.
constexpr float kXScale = 4096.0f, kAScale = 256.0f;

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

// Work units of each kernel and matrix, as prefix sums.
enum MuonUnits { kUnitsMoment = 0, kUnitsThin, kUnitsPrepare, kUnitsGram, kUnitsSquare, kUnitsUpdate, kUnitKinds };

template <int N>
struct MuonTableN {
  int32_t prefix[kUnitKinds][N + 1];
  MuonMat mat[N];
};
// The first kernel of a call gets the table as a parameter and leaves a copy in the workspace for
// the others: a 25 KB parameter block costs each launch about 10 us of host time.
using MuonTable = MuonTableN<kMuonMaxBatch>;

// What every kernel of a call needs.
struct MuonCall {
  uint8_t* ws;
  int32_t count;
  int32_t K, n_coeffs;
  int32_t nesterov;
  float beta, rest;        // momentum and 1 - momentum
  float keep, rate;        // weights <- keep * weights - rate * scale * X_K; rate < 0: output = scale * X_K
  int32_t small;           // the iterate kernel on single CTAs (128 x 64 tiles) instead of pairs
  int32_t split_steps;     // small: 64-element K steps of one part of a split Gram product
  int64_t parts_at, counts_at;   // small: partial tiles and their counts, bytes into the workspace
  int32_t counts;
  int32_t stall;           // test only: the MMA issuers wait on a barrier nothing arrives on
  float coeffs[3 * FS4_MAX_ITERS];
};

// Workspace: [header | counts | table | partial sums | one block per matrix].  Header: the status
// word at byte 0.  Counts: the iterate kernel's finished work, a word per matrix.
constexpr int64_t kMuonHeader = 256, kMuonTableAt = kMuonHeader + 4 * kMuonMaxBatch;
static_assert(kMuonTableAt % 16 == 0, "the table holds pointers");
constexpr int64_t kMuonPartials = (kMuonTableAt + (int64_t)sizeof(MuonTable) + 255) / 256 * 256;
__host__ __device__ inline uint32_t* muon_status(uint8_t* ws) { return reinterpret_cast<uint32_t*>(ws); }
__host__ __device__ inline uint32_t* muon_counts(uint8_t* ws) { return reinterpret_cast<uint32_t*>(ws + kMuonHeader); }
__host__ __device__ inline MuonTable* muon_table(uint8_t* ws) { return reinterpret_cast<MuonTable*>(ws + kMuonTableAt); }
__host__ __device__ inline double* muon_partials(uint8_t* ws) { return reinterpret_cast<double*>(ws + kMuonPartials); }

// Small calls of the iterate kernel: tiles of 128 rows x 64 columns, only those that hold rows and
// columns of the matrix (its rows and the columns of A and B in whole 128s: they are K elements).
constexpr int kMuonSmallUnits = 296;    // most units of a product, two for each of 148 SMs
constexpr int kMuonSmallSteps = 3500;   // most K steps of an update
__host__ __device__ inline int32_t muon_steps(int32_t k) { return (k + 63) / 64; }
__host__ __device__ inline int32_t muon_row_tiles(int32_t m) { return (m + 127) / 128; }
// Tiles of A or B from the diagonal's 256-blocks on.
__host__ __device__ inline int64_t muon_gram_tiles(int32_t m) {
  const int64_t r = muon_row_tiles(m), h = r / 2;
  return 2 * r * r - 4 * (h * (h - 1) + (r & 1 ? h : 0));
}
// Parts of a Gram product with `steps` K steps at `per` a part: adding the parts up costs about
// as much as twelve steps.
__host__ __device__ inline int32_t muon_splits(int32_t steps, int32_t per) {
  return steps < per + 12 ? 1 : (steps + per - 1) / per;
}

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

// A thin matrix's block: T (m x m FP32), the factor of the products T U (FP32, 0 if the norm is not
// finite), then one m x m FP64 Gram matrix per chunk of columns.
__host__ __device__ inline int64_t thin_flag_offset(int64_t m) { return 4 * m * m; }
__host__ __device__ inline int64_t thin_gram_offset(int64_t m) { return (4 * m * m + 4 + 255) / 256 * 256; }
__host__ __device__ inline int64_t thin_chunks(int64_t n) { return (n + kMuonChunk - 1) / kMuonChunk; }
__host__ __device__ inline int64_t thin_bytes(int64_t m, int64_t n) { return thin_gram_offset(m) + 8 * m * m * thin_chunks(n); }

// launchers; the unit counts come from the table's prefix sums
cudaError_t launch_muon_moment(const MuonCall& c, const MuonTable& t, cudaStream_t st);
cudaError_t launch_muon_thin(const MuonCall& c, int32_t units, cudaStream_t st);
cudaError_t launch_muon_prepare(const MuonCall& c, int32_t units, cudaStream_t st, int num_sms);
cudaError_t launch_muon_iterate(const MuonCall& c, int64_t ws_bytes, int32_t units, cudaStream_t st, int num_sms);

}  // namespace fs4
