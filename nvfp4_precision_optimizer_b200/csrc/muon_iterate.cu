// Muon's Newton-Schulz iterations on FP16 operands (sm_100a, tcgen05 kind::f16 on CTA pairs,
// FP32 accumulation in TMEM), all 3K products of all matrices in one persistent launch:
//   Gram    A  = X X^T
//   Square  B  = b A + c A^2
//   Update  X' = a X + B X
// Precision.  X and A are kept as a high and a low FP16 part (22 significand bits); the tensor
// cores read the high parts.  A and B are dominated by their diagonals once X approaches an
// orthogonal matrix, and a X + B X then cancels, so a diagonal rounded to 11 bits would set the
// error of the step.  The diagonals stay in FP32 and out of the operands:
//   A = A0 + D:  A^2 = A0^2 + A0 D + D A0 + D^2,   element ij: (A0^2)_ij + A0_ij (d_i + d_j), d_i^2 on the diagonal
//   B = B0 + E:  a X + B X = (a + e_i) X_ij + (B0 X)_ij
// which the epilogues add from the FP32 diagonals.  The tensor cores multiply B0 by X's high part
// alone, so with X = H + L the update leaves out B0 L.  Where one direction dominates, B L lies in
// that direction and does no harm, but B0 L = B L - E L does not: E L reaches the small singular
// values, which the iterations left raise by a factor a each.  So all but the last two updates
// apply E to H as well (what is left out is then B L):
//   X' = (a + e_i) H_ij + a L_ij + (B0 H)_ij
// and the last two, where nothing small is left to raise and B is nearly diagonal, apply it to H + L.
// Restated in numpy (K = 5, 33 to 1024 rows): Gaussian, decaying and low-rank inputs and up to 1e-5
// of noise beside a few dominant directions 0.1-1.8e-3 from the exact iteration, against up to 4e-2
// with E applied to H + L throughout (and up to 1e-1 with K = 10).  Rounded diagonals give 2.6e-3
// and BF16 operands 1.4-2.4e-2 on Gaussian inputs.  A dominant direction whose elements are all
// equal is the worst case, since equal elements round alike: up to 1.2e-2.
// A and B are symmetric: only 256 x 256 blocks on and above the diagonal are computed and
// stored.  A block below it is read as its mirror image with the operand's M or N index
// fastest, which the tensor core takes directly; so is X as the second operand of the update,
// whose rows are its K index.  Nothing is stored twice.
// Structure.  Large calls: a pair of CTAs computes a 256 x 256 block, 128 rows and 256 TMEM columns each;
// either operand's 256 rows are split over the two, so that a 64-deep stage costs each SM 32 KB
// for 512 cycles of MMAs (a single CTA's 128 x 256 tile would cost 48 KB, more than the 67
// bytes a cycle that L2 delivers to an SM).  Small calls, whose few blocks would leave most SMs
// idle and whose time is the sum of latencies: single CTAs on 128 x 64 tiles, a quarter of the
// epilogue each, only over the rows and columns that the matrices have; a long Gram product is
// split along K, the partial tiles summed in order by the CTA that finishes last.  Two accumulators: a block's epilogue overlaps the
// next block's MMAs.  Both CTAs' copies count on the leader's barrier (tensor maps allow that);
// a relay through the other CTA's threads took 1300 cycles a stage.  The units of all products form one
// sequence, dealt to the CTAs in turn; a unit waits until its matrix's product before is complete (a
// count per matrix in the workspace; the waits are bounded), so the tail of one matrix's product
// overlaps another's, and 3K - 1 launches and their set-up are saved.  Nothing waits for a later
// unit, and all CTAs are resident (a cooperative launch), so some unit can always go on.
// Measured, K = 5: 8192 x 8192 9.2 ms, 1.2 PFLOP/s (83% of the MMA rate at the clock that the power
// cap leaves); seven 2048-wide matrices 2.15 ms; 256 x 256 75 us, 5 us a product: first loads 0.9, MMAs
// 1.3, epilogue 1, the count and the next loads 1.8.
#include <cstdint>
#include <cstddef>
#include <type_traits>

#include "muon_device.cuh"
#include "pair_device.cuh"
#include "pair_host.h"

namespace fs4 {
namespace {

constexpr int kThreads = 320;               // warp 0 producer, warp 1 MMA issuer, warps 2-9 epilogue
constexpr int kTileBytes16 = 16384;         // 128 rows x 64 FP16 elements
constexpr int kGroup = 8;                   // block rows of a raster group: pairs at work share operands in L2

// kPair: 256 x 256 blocks on CTA pairs; else 128 x 64 tiles on single CTAs.
template <bool kPair>
struct Tile {
  static constexpr int kN = kPair ? 256 : 64;              // columns of an accumulator
  static constexpr int kA = 16384, kB = kPair ? 16384 : 8192;   // a stage's operands in one CTA, 64 k
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = kPair ? 6 : 8;
  static constexpr uint32_t kCols = 2 * kN;                // two accumulators
  static constexpr int kWarpCols = kN / 2;                 // columns of one epilogue warp
};

// What the roles need of a matrix, in shared memory.
struct Block {
  int64_t base;
  int32_t m, n;
};
struct Shared {
  uint64_t full[8];            // (pairs: in the leader) the operands of a stage landed
  uint64_t empty[8];           // the MMAs reading the stage finished (both CTAs)
  uint64_t acc_full[2];
  uint64_t acc_empty[2];       // (leader) the accumulator is drained
  uint64_t done;
  uint32_t tmem;
  int32_t abort;
  uint32_t issued[2];          // (leader) stages that each CTA's producer issued
  int32_t arrived;             // CTAs that had finished their part of a split product
  alignas(16) float diag[8][128];   // an epilogue warp's columns of A's diagonal
  int32_t prefix[3][kMuonMaxBatch + 1];   // units of the three products
  Block block[kMuonMaxBatch];
};
template <bool kPair>
constexpr int kSmem = 1024 + Tile<kPair>::kStages * Tile<kPair>::kStage + (int)sizeof(Shared);
static_assert(kSmem<true> <= 232448 && kSmem<false> <= 232448, "over the per-CTA shared-memory limit");
static_assert(offsetof(Shared, diag) % 16 == 0 && Tile<true>::kStage % 1024 == 0 && Tile<false>::kStage % 1024 == 0,
              "read and written 16 bytes at a time");

enum { kGram = 0, kSquare = 1, kUpdate = 2 };

__device__ __forceinline__ int32_t padded(int32_t v) { return (v + kMuonPad - 1) / kMuonPad * kMuonPad; }

// One unit of work: this CTA's rows and columns of an output block, and its range of K.
struct Job {
  int mat;
  int32_t row0, col0;      // first row of this CTA, first column of the accumulator
  int32_t n0;              // first row of the second operand's part in this CTA
  int32_t k0, steps;       // K / 64
  int32_t part, parts;     // of a product split along K
};

// Unit u of a product.  Pairs: within a matrix the blocks go through groups of kGroup block rows,
// column by column, so that the pairs at work read few operand rows and columns.
template <bool kPair, int E>
__device__ __forceinline__ Job make_job(const MuonCall& p, const Shared& sh, int32_t u, uint32_t rank) {
  const int32_t* prefix = sh.prefix[E];
  Job j;
  j.mat = owner_of(prefix, p.count, u);
  const Block& d = sh.block[j.mat];
  int32_t t = u - prefix[j.mat];
  j.k0 = 0;
  j.part = 0;
  j.parts = 1;
  j.steps = muon_steps(E == kGram ? d.n : d.m);
  if constexpr (kPair) {
    const int32_t T = padded(d.m) / 256;
    int32_t I, J;
    if constexpr (E == kUpdate) {
      const int32_t nj = padded(d.n) / 256, g = t / (kGroup * nj), h = min(kGroup, T - kGroup * g);
      t -= g * kGroup * nj;
      J = t / h;
      I = kGroup * g + t % h;
    } else {
      int32_t r0 = 0;
      for (;; r0 += kGroup) {                 // blocks on and above the diagonal
        const int32_t h = min(kGroup, T - r0), tri = h * (h + 1) / 2, size = tri + h * (T - r0 - h);
        if (t >= size) { t -= size; continue; }
        if (t >= tri) {
          J = r0 + h + (t - tri) / h;
          I = r0 + (t - tri) % h;
        } else {
          int32_t c = 0;
          while (t > c) t -= ++c;
          J = r0 + c;
          I = r0 + t;
        }
        break;
      }
    }
    j.row0 = 256 * I + 128 * (int32_t)rank;
    j.col0 = 256 * J;
    j.n0 = 256 * J + 128 * (int32_t)rank;
  } else {
    if (E == kGram) {
      j.parts = muon_splits(j.steps, p.split_steps);
      j.part = t % j.parts;
      t /= j.parts;
      if (j.parts > 1) {
        j.k0 = j.part * p.split_steps;
        j.steps = min(p.split_steps, j.steps - j.k0);
      }
    }
    const int32_t rows = muon_row_tiles(d.m);
    int32_t i = 0, c = 0;
    if constexpr (E == kUpdate) {
      i = t % rows;
      c = t / rows;
    } else {                                  // 64-column tiles from the 256-block on the diagonal on
      for (;; ++i) {
        const int32_t size = 2 * rows - 4 * (i >> 1);
        if (t < size) break;
        t -= size;
      }
      c = 4 * (i >> 1) + t;
    }
    j.row0 = 128 * i;
    j.col0 = j.n0 = 64 * c;
  }
  return j;
}

// Row `at` of a symmetric operand is stored from the 256-block on the diagonal on: the first k
// step there.  Steps before it are read as the mirror image.
__device__ __forceinline__ int32_t first_row_step(int32_t at) { return (at >> 8) * 4; }

struct Maps {
  CUtensorMap rows128, rows64;     // the workspace as 128-byte rows, copied 128 or 64 at a time
};

// The units of product number ph (0 .. 3K - 1) that this CTA or pair takes: dealt on from where the
// product before ended.
template <bool kPair>
struct Deal {
  int32_t next = kPair ? blockIdx.x >> 1 : blockIdx.x;
  __device__ __forceinline__ int32_t step() const { return kPair ? gridDim.x >> 1 : gridDim.x; }
  // after a product of `total` units
  __device__ __forceinline__ void skip(int32_t total) {
    next = (next - total) % step();
    if (next < 0) next += step();
  }
};

// What a matrix's count must have reached before its units of product (it, E) start: every epilogue
// warp adds one when its part of a unit is stored.
template <bool kPair, int E>
__device__ __forceinline__ uint32_t units_before(const Shared& sh, int mat, int it) {
  const int32_t g = sh.prefix[kGram][mat + 1] - sh.prefix[kGram][mat], q = sh.prefix[kSquare][mat + 1] - sh.prefix[kSquare][mat],
                x = sh.prefix[kUpdate][mat + 1] - sh.prefix[kUpdate][mat];
  return (uint32_t)(it * (g + q + x) + (E > kGram ? g : 0) + (E > kSquare ? q : 0)) * (kPair ? 16u : 8u);
}

// Where a CTA's copies go and are counted.
struct Target {
  const Maps* maps;
  const uint8_t* ws;
  uint64_t* bar;         // single CTAs
  uint32_t cluster_bar;  // pairs: the leader's
};
template <bool kPair, int kRows>
__device__ __forceinline__ void copy_rows(const Target& t, uint32_t dst, int64_t src) {
  if constexpr (kPair) tma_rows_pair(dst, kRows == 128 ? &t.maps->rows128 : &t.maps->rows64, (int32_t)(src >> 7), t.cluster_bar);
  else bulk_g2s_addr(dst, t.ws + src, 128 * kRows, t.bar);
}
// One operand of a job: kRows (64 or 128) of its rows of M or N, 64 k at a time.  Addresses advance
// by constants; the producer's thread has little time for more.
template <bool kPair, int kRows>
struct Source {
  int64_t rows, columns;     // k step 0, read by rows (a tile, or half of one, per step) ...
  int64_t pitch;             // ... or, mirrored, by columns: 128 stored rows are `pitch` apart
  int32_t turn;              // k steps below this are read by columns

  // rows at.. of a matrix with cp padded columns at src
  __device__ __forceinline__ Source(int64_t src, int32_t cp, int32_t at, int32_t turn_) : turn(turn_) {
    pitch = (int64_t)(cp >> 6) * kTileBytes16;
    rows = src + (at >> 7) * pitch + (at & 127) * 128;
    columns = src + (int64_t)(at >> 6) * kTileBytes16;
  }
  __device__ __forceinline__ void copy(const Target& t, uint32_t dst, int32_t k) const {
    if (k < turn) {
      // 64 stored rows, halves of neighbouring tiles
      const int64_t from = columns + (k >> 1) * pitch + (k & 1) * (kTileBytes16 / 2);
#pragma unroll
      for (int i = 0; i < kRows / 64; ++i) copy_rows<kPair, 64>(t, dst + i * (kTileBytes16 / 2), from + i * kTileBytes16);
    } else {
      copy_rows<kPair, kRows>(t, dst, rows + (int64_t)k * kTileBytes16);
    }
  }
};

// ------------------------------------------------------------------ epilogue
// Chunks 2 i and 2 i + 1 of a row lie in one 32-byte piece, in the order of the row's bit 0.
__device__ __forceinline__ Pair ordered(const Pair& r, bool swap) {
  Pair o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.w[i] = swap ? r.w[4 + i] : r.w[i];
    o.w[4 + i] = swap ? r.w[i] : r.w[4 + i];
  }
  return o;
}
__device__ __forceinline__ uint4 quad(const Pair& p, int i) { return make_uint4(p.w[4 * i], p.w[4 * i + 1], p.w[4 * i + 2], p.w[4 * i + 3]); }

// 32 results (columns col .. col + 31 of working row `row`) into the weights or the output.
// Returns whether a result is not finite.
template <typename T>
__device__ __forceinline__ bool write_result(const MuonCall& p, const MuonMat& d, int32_t row, int32_t col, float* y, int lane) {
  bool bad = false;
  constexpr int kPer = 32 / (int)sizeof(T);                  // elements of 32 bytes
  const bool blend = p.rate >= 0.0f;
  auto result = [&](float x, float w) -> float {
    const float u = x * d.scale;
    bad |= !isfinite(u);
    return blend ? fmaf(-p.rate, u, p.keep * w) : u;
  };
  T* w = static_cast<T*>(d.w);
  // in each case the old weights' loads are in flight together
  if (!d.tall && col + 32 <= d.n && ((reinterpret_cast<uintptr_t>(w) | (uintptr_t)(d.ldw * (int64_t)sizeof(T))) & 31) == 0) {
    if (row >= d.m) return false;
    T* at = w + row * d.ldw + col;
#pragma unroll
    for (int q = 0; q < 32 / kPer; q += 2) {
      Pair r[2]{};
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (blend) r[b] = load_pair(at + (q + b) * kPer);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        T* e = reinterpret_cast<T*>(r[b].w);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
        put_as(e + i, result(y[(q + b) * kPer + i], blend ? to_f32(e[i]) : 0.0f));
        }
        store_pair(at + (q + b) * kPer, r[b]);
      }
    }
    return bad;
  }
  // Neighbouring lanes hold neighbouring elements of a tall matrix's rows.  Rows that do not start
  // on 32 bytes: the warp's 32 x 32 values change places first.
  uint32_t* v = reinterpret_cast<uint32_t*>(y);
  if (!d.tall) turn32(v, lane);
  const int32_t r0 = d.tall ? row : row - lane, c0 = d.tall ? col : col + lane;      // of value 0
  if (r0 >= d.m || c0 >= d.n) return false;
  const int32_t count = min(32, d.tall ? d.n - c0 : d.m - r0);
  T* at = w + (d.tall ? (int64_t)c0 * d.ldw + r0 : (int64_t)r0 * d.ldw + c0);
#pragma unroll
  for (int h = 0; h < 32; h += 8) {
    float old[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) old[i] = (blend && h + i < count) ? to_f32(at[(h + i) * d.ldw]) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (h + i < count) put_as(at + (h + i) * d.ldw, result(y[h + i], old[i]));
  }
  return bad;
}

// Input of 32 columns: A or X, high and low parts.
struct Input {
  Pair h[2], l[2];
};

// What one epilogue warp (rows 32 quad .. + 31 of this CTA's 128, kWarpCols columns) reads and
// writes of a block.
template <bool kPair, int E>
struct Place {
  const uint8_t* in_hi;
  const uint8_t* in_lo;
  uint8_t* out_hi;
  uint8_t* out_lo;
  float* da;             // diagonals of A and B
  float* db;
  int32_t row, col0;     // this lane's row, the warp's first column
  int x6;
  bool swap, diagonal;

  __device__ __forceinline__ Place(const MuonCall& p, const Shared& sh, const Job& j, int it, int quad_, int half, int lane) {
    const Block& d = sh.block[j.mat];
    const int32_t mp = padded(d.m), np = padded(d.n), cp = E == kUpdate ? np : mp;
    const MuonLayout L = muon_layout(mp, np);
    uint8_t* ws = p.ws + d.base;
    const bool odd = (it & 1) != 0;
    row = j.row0 + 32 * quad_ + lane;
    col0 = j.col0 + Tile<kPair>::kWarpCols * half;
    const int64_t tile = ((int64_t)(row >> 7) * (cp >> 6) + (col0 >> 6)) * kTileBytes16 + (row & 127) * 128;
    in_hi = ws + (E == kUpdate ? (odd ? L.x[1] : L.x[0]) : L.a) + tile;
    in_lo = ws + (E == kUpdate ? L.xl : L.al) + tile;
    out_hi = ws + (E == kUpdate ? (odd ? L.x[0] : L.x[1]) : E == kSquare ? L.b : L.a) + tile;
    out_lo = ws + (E == kUpdate ? L.xl : L.al) + tile;
    da = reinterpret_cast<float*>(ws + L.da);
    db = reinterpret_cast<float*>(ws + L.db);
    swap = (row & 1) != 0;
    x6 = row & 6;
    diagonal = E != kUpdate;
  }
  // 32-byte piece i (0, 1) of the 32 columns from c (a multiple of 32) on
  __device__ __forceinline__ int piece(int c, int i) const {
    const int in = (col0 & 32) + c;
    return (in >> 6) * kTileBytes16 + 16 * ((((in & 32) >> 3) + 2 * i) ^ x6);
  }
  __device__ __forceinline__ void load(Input& in, int c) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      in.h[i] = load_pair(in_hi + piece(c, i));
      in.l[i] = load_pair(in_lo + piece(c, i));
    }
  }
};

// Before the accumulator is ready: the first of the warp's input and the diagonal entries.
struct Ahead {
  Input in[2];
  float own;             // d_i (Square) or a + e_i (Update)
  float own_low;         // Update: what multiplies X's low part, a or a + e_i
};
template <bool kPair, int E, bool kLast>
__device__ __forceinline__ void look_ahead(const MuonCall& p, const Place<kPair, E>& w, Ahead& a, float* diag, int it, int lane) {
  if constexpr (E == kGram) return;
  w.load(a.in[0], 0);
  if constexpr (kPair && !kLast) w.load(a.in[1], 32);
  if constexpr (E == kSquare) {
    a.own = __ldcg(w.da + w.row);
    __syncwarp();
    if constexpr (kPair) reinterpret_cast<float4*>(diag)[lane] = __ldcg(reinterpret_cast<const float4*>(w.da + w.col0) + lane);
    else diag[lane] = __ldcg(w.da + w.col0 + lane);
    __syncwarp();
  } else {
    const float pa = p.coeffs[p.n_coeffs == 1 ? 0 : 3 * it];
    a.own = pa + __ldcg(w.db + w.row);
    a.own_low = it >= p.K - 2 ? a.own : pa;
  }
}

// kLast: the last update, which writes the weights or the output (an instance of its own, so that
// its registers do not crowd the others).
template <bool kPair, int E, bool kLast>
__device__ __forceinline__ void epilogue(const MuonCall& p, const Place<kPair, E>& w, Ahead& a, const float* diag, const MuonMat* m, int it,
                                         uint32_t taddr, int lane, const float* summed) {
  const float* poly = p.coeffs + (p.n_coeffs == 1 ? 0 : 3 * it);
  const float pb = poly[1], pc = poly[2];
  bool bad = false;
  // (rolled: a block's epilogue runs once per product, and its instructions come from L2)
#pragma unroll 1
  for (int c = 0; c < Tile<kPair>::kWarpCols; c += 32) {
    float v[32];
    if (!kPair && E == kGram && summed) {      // a product split along K: the partial sums' sum
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = summed[i];
    } else {
      tmem_ld32(taddr + c, v);
    }
    const int32_t col = w.col0 + c;
    // the 32 x 32 part on the diagonal (whole warps: rows and columns are multiples of 32)
    const bool on = w.diagonal && (w.row & ~31) == col;
    if constexpr (E == kGram) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= kAScale / (kXScale * kXScale);
      if (on) {
        float e = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          e = lane == i ? v[i] : e;
          v[i] = lane == i ? 0.0f : v[i];
        }
        w.da[w.row] = e * (1.0f / kAScale);
      }
    } else {
      const Input in = a.in[0];
      if constexpr (kPair && !kLast) {
        a.in[0] = a.in[1];
        if (c < 64) w.load(a.in[1], c + 64);       // the input two steps on
      } else if constexpr (kPair) {
        if (c < 96) w.load(a.in[0], c + 32);       // (registers: one step on)
      }
      float e = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float* y = v + 8 * q;
        const uint4 hi = quad(ordered(in.h[q >> 1], w.swap), q & 1), lo = quad(ordered(in.l[q >> 1], w.swap), q & 1);
        if constexpr (E == kSquare) {
          float x[8];
          join8(hi, lo, x);
          const float4 d0 = reinterpret_cast<const float4*>(diag + c)[2 * q], d1 = reinterpret_cast<const float4*>(diag + c)[2 * q + 1];
          const float dc[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
          if (on) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (lane == 8 * q + i) e = y[i];
          }
          // kAScale times b A0 + c (A0^2 + A0 (d_i + d_j))
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], fmaf(pc, a.own + dc[i], pb), y[i] * (pc / kAScale));
        } else {
          // kXScale times (a + e_i) H + (a or a + e_i) L + B0 H
          const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
          const float own_low = kLast ? a.own : a.own_low;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = fmaf(a.own, half_lo(h[i]), fmaf(own_low, half_lo(l[i]), y[2 * i] * (1.0f / kAScale)));
            y[2 * i + 1] = fmaf(a.own, half_hi(h[i]), fmaf(own_low, half_hi(l[i]), y[2 * i + 1] * (1.0f / kAScale)));
          }
        }
      }
      if (E == kSquare && on) {
        w.db[w.row] = fmaf(a.own, fmaf(pc, a.own, pb), e * (pc / (kAScale * kAScale)));
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (lane == i) v[i] = 0.0f;
      }
    }
    if constexpr (kLast) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kXScale;
      if (m->tw == kTypeF32) bad |= write_result<float>(p, *m, w.row, col, v, lane);
      else if (m->tw == kTypeBf16) bad |= write_result<__nv_bfloat16>(p, *m, w.row, col, v, lane);
      else bad |= write_result<__half>(p, *m, w.row, col, v, lane);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 h0, h1, l0, l1;
        split8(v + 16 * i, h0, l0);
        split8(v + 16 * i + 8, h1, l1);
        store_pair(w.out_hi + w.piece(c, i), ordered(Pair{{h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w}}, w.swap));
        if constexpr (E != kSquare)
          store_pair(w.out_lo + w.piece(c, i), ordered(Pair{{l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w}}, w.swap));
      }
    }
  }
  if (kLast && bad) atomicOr(muon_status(p.ws), kStatusNonFinite);
}

// ------------------------------------------------------------------ counts in the workspace
__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ bool wait_count(const uint32_t* count, uint32_t target, uint32_t* status, volatile int* abort) {
  if (load_acquire(count) >= target) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (*abort) return false;
    if (load_acquire(count) >= target) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      *abort = 1;
      return false;
    }
  }
}
// Generic writes before, asynchronous (TMA) reads after, or the other way round.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ------------------------------------------------------------------ roles, one product each
template <bool kPair>
struct Ring {
  uint32_t s = 0, ph = 0, issued = 0;
  __device__ __forceinline__ void next() {
    ++issued;
    if (++s == (uint32_t)Tile<kPair>::kStages) { s = 0; ph ^= 1u; }
  }
};

template <bool kPair, int E>
__device__ __forceinline__ bool produce(const MuonCall& p, const Maps& maps, Shared& sh, Ring<kPair>& ring, Deal<kPair>& deal, int it, uint32_t base,
                                        uint32_t rank, volatile int* abort) {
  using T = Tile<kPair>;
  const int32_t total = sh.prefix[E][p.count];
  const uint32_t leader_full = kPair ? cluster_map(smem_addr(&sh.full[0]), 0) : 0u;
  int seen = -1;       // the last matrix found ready for this product
  for (int32_t u = deal.next; u < total; u += deal.step()) {
    const Job j = make_job<kPair, E>(p, sh, u, rank);
    const Block& d = sh.block[j.mat];
    const int32_t mp = padded(d.m), np = padded(d.n);
    const MuonLayout L = muon_layout(mp, np);
    const int64_t x = d.base + ((it & 1) ? L.x[1] : L.x[0]);
    const int64_t sym = d.base + (E == kSquare ? L.a : L.b);
    if (j.mat != seen && (E != kGram || it > 0)) {
      if (!wait_count(muon_counts(p.ws) + j.mat, units_before<kPair, E>(sh, j.mat, it), muon_status(p.ws), abort)) return false;
      fence_async();
      seen = j.mat;
    }
    // symmetric operands are read as their mirror image below the diagonal's 256-blocks; X as
    // the update's second operand always by columns
    const Source<kPair, 128> first(E == kGram ? x : sym, E == kGram ? np : mp, j.row0, E == kGram ? 0 : first_row_step(j.row0));
    const Source<kPair, T::kB / 128> second(E == kSquare ? sym : x, E == kSquare ? mp : np, j.n0,
                                            E == kGram ? 0 : E == kSquare ? first_row_step(j.n0) : 0x7FFFFFFF);
    for (int32_t k = j.k0; k < j.k0 + j.steps; ++k) {
      if (!mbar_wait(&sh.empty[ring.s], ring.ph ^ 1u, muon_status(p.ws), abort)) return false;
      const uint32_t a = base + ring.s * T::kStage;
      Target t{&maps, p.ws, &sh.full[ring.s], 0u};
      if constexpr (kPair) t.cluster_bar = leader_full + 8 * ring.s;
      if (rank == 0) mbar_arrive_expect_tx(&sh.full[ring.s], (kPair ? 2 : 1) * T::kStage);
      first.copy(t, a, k);
      second.copy(t, a + T::kA, k);
      ring.next();
    }
  }
  deal.skip(total);
  return true;
}

template <bool kPair, int E>
__device__ __forceinline__ bool multiply(const MuonCall& p, Shared& sh, Ring<kPair>& ring, Deal<kPair>& deal, uint32_t& tl, uint32_t base, uint32_t tmem,
                                         volatile int* abort) {
  using T = Tile<kPair>;
  const uint64_t ra0 = sdesc_sw128(base), rb0 = sdesc_sw128(base + T::kA);
  const uint64_t ca0 = sdesc_sw128_mn(base, kTileBytes16 / 2), cb0 = sdesc_sw128_mn(base + T::kA, kTileBytes16 / 2);
  constexpr uint64_t kStep = T::kStage >> 4;
  const int32_t total = sh.prefix[E][p.count];
  for (int32_t u = deal.next; u < total; u += deal.step(), ++tl) {
    const Job j = make_job<kPair, E>(p, sh, u, 0);
    const uint32_t acc = tmem + (uint32_t)T::kN * (tl & 1u);
    if (!mbar_wait_cluster(&sh.acc_empty[tl & 1u], ((tl >> 1) & 1u) ^ 1u, muon_status(p.ws), abort)) return false;
    tc_fence_after();
    const int32_t a_turn = E == kGram ? 0 : first_row_step(j.row0);
    const int32_t b_turn = E == kGram ? 0 : E == kSquare ? first_row_step(j.n0) : 0x7FFFFFFF;
    for (int32_t i = 0; i < j.steps; ++i) {
      const int32_t k = j.k0 + i;
      const bool landed = kPair ? mbar_wait_cluster(&sh.full[ring.s], ring.ph, muon_status(p.ws), abort)
                                : mbar_wait(&sh.full[ring.s], ring.ph, muon_status(p.ws), abort);
      if (!landed) return false;
      tc_fence_after();
      const bool am = k < a_turn, bm = k < b_turn;
      // (constant steps and instruction descriptors: every value computed here is an issue slot more)
      auto issue = [&](auto am_c, auto bm_c) {
        constexpr int kAm = decltype(am_c)::value, kBm = decltype(bm_c)::value;
        // 16 k: 32 bytes along a row, or 16 rows of 128 bytes
        const uint64_t da = (kAm ? ca0 : ra0) + ring.s * kStep, db = (kBm ? cb0 : rb0) + ring.s * kStep;
        constexpr uint64_t ia = kAm ? 128 : 2, ib = kBm ? 128 : 2;
        constexpr uint32_t idesc = idesc_f16(kPair ? 256 : 128, T::kN, kAm, kBm);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t acc_on = h != 0 ? 1u : (i != 0 ? 1u : 0u);
          if constexpr (kPair) tc_mma_f16_pair(acc, da + h * ia, db + h * ib, idesc, acc_on);
          else tc_mma_bf16(acc, da + h * ia, db + h * ib, idesc, acc_on);   // kind::f16: the type is in idesc
        }
      };
      using No = std::integral_constant<int, 0>;
      using Yes = std::integral_constant<int, 1>;
      if constexpr (E == kGram) {
        issue(No{}, No{});
      } else if constexpr (E == kUpdate) {
        if (am) issue(Yes{}, Yes{});
        else issue(No{}, Yes{});
      } else {
        if (am && bm) issue(Yes{}, Yes{});
        else if (am) issue(Yes{}, No{});
        else if (bm) issue(No{}, Yes{});
        else issue(No{}, No{});
      }
      if constexpr (kPair) tc_commit_pair(&sh.empty[ring.s]);
      else tc_commit(&sh.empty[ring.s]);
      ring.next();
    }
    if constexpr (kPair) tc_commit_pair(&sh.acc_full[tl & 1u]);
    else tc_commit(&sh.acc_full[tl & 1u]);
  }
  deal.skip(total);
  return true;
}

// The small variant's eight epilogue warps: true if it is true in all of them.
__device__ __forceinline__ bool vote(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// A split product's unit: leave this part's sums in the workspace; the CTA that finishes a tile's
// last part adds all parts up, in their order, into `v` and returns true.
__device__ __forceinline__ bool sum_parts(const MuonCall& p, Shared& sh, const Job& j, int32_t u, uint32_t taddr, int quad_, int half,
                                          int lane, float* v) {
  tmem_ld32(taddr, v);
  // [unit][row][column]: 128 bytes a lane
  const int64_t at = ((int64_t)(32 * quad_ + lane) * 64 + 32 * half) * 4;
  uint8_t* parts = p.ws + p.parts_at;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    Pair r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[8 * q + i]);
    store_pair(parts + (int64_t)u * (128 * 64 * 4) + at + 32 * q, r);
  }
  const int32_t first = u - j.part;
  uint32_t* arrived = reinterpret_cast<uint32_t*>(p.ws + p.counts_at) + first;
  named_bar(2, 256);
  if (threadIdx.x == 64) {
    __threadfence();
    const uint32_t before = atomicAdd(arrived, 1u);
    __threadfence();
    sh.arrived = (int32_t)before;
    if (before == (uint32_t)j.parts - 1) *arrived = 0u;     // for the next iteration
  }
  named_bar(2, 256);
  if (sh.arrived != j.parts - 1) return false;
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  for (int s = 0; s < j.parts; ++s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const Pair r = load_pair(parts + (int64_t)(first + s) * (128 * 64 * 4) + at + 32 * q);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * q + i] += __uint_as_float(r.w[i]);
    }
  }
  return true;
}

template <bool kPair, int E, bool kLast>
__device__ __forceinline__ bool finish(const MuonCall& p, Shared& sh, Deal<kPair>& deal, uint32_t& tl, int it, uint32_t tmem, uint32_t rank, int quad_,
                                       int half, int lane, volatile int* abort, bool alive) {
  using T = Tile<kPair>;
  const int32_t total = sh.prefix[E][p.count];
  int seen = -1;
  bool ok = kPair || alive;
  for (int32_t u = deal.next; u < total; u += deal.step(), ++tl) {
    const Job j = make_job<kPair, E>(p, sh, u, rank);
    const uint32_t b = tl & 1u;
    const Place<kPair, E> w(p, sh, j, it, quad_, half, lane);
    float* diag = sh.diag[4 * half + quad_];
    // other CTAs' results are read below: see them
    if (ok && j.mat != seen && (E != kGram || it > 0)) {
      if (lane == 0) ok = wait_count(muon_counts(p.ws) + j.mat, units_before<kPair, E>(sh, j.mat, it), muon_status(p.ws), abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      __syncwarp();      // orders the lanes' loads behind lane 0's acquire (a vote orders nothing)
      seen = j.mat;
    }
    if (kPair && !ok) return false;
    Ahead a;
    look_ahead<kPair, E, kLast>(p, w, a, diag, it, lane);
    if (ok && lane == 0) ok = mbar_wait(&sh.acc_full[b], (tl >> 1) & 1u, muon_status(p.ws), abort);
    ok = __all_sync(0xFFFFFFFFu, ok);
    // The small variant's warps meet in split units: all of them work there or none. A vote, not
    // the flag, which another warp may raise between two warps' reads; and a warp whose wait ran
    // out stays, without work, so that it is there for the votes that follow.
    if (!kPair && E == kGram && j.parts > 1) ok = vote(ok);
    if (!ok) {
      if (kPair) return false;
      continue;
    }
    __syncwarp();
    tc_fence_after();
    const uint32_t taddr = tmem + (uint32_t)T::kN * b + ((uint32_t)(32 * quad_) << 16) + (uint32_t)(T::kWarpCols * half);
    const MuonMat* m = &muon_table(p.ws)->mat[j.mat];
    if (!kPair && E == kGram && j.parts > 1) {
      float v[32];
      if (sum_parts(p, sh, j, u, taddr, quad_, half, lane, v)) epilogue<kPair, E, kLast>(p, w, a, diag, m, it, taddr, lane, v);
    } else {
      epilogue<kPair, E, kLast>(p, w, a, diag, m, it, taddr, lane, nullptr);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (rank == 0) mbar_arrive(&sh.acc_empty[b]);
      else mbar_arrive_remote(cluster_map(smem_addr(&sh.acc_empty[b]), 0));
      // this warp's results (__syncwarp orders the lanes' before the release); a producer that
      // sees the count fences its TMA copies behind it
      asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(muon_counts(p.ws) + j.mat), "r"(1u) : "memory");
    }
  }
  deal.skip(total);
  return ok;
}

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1) muon_iterate_kernel(const __grid_constant__ MuonCall p, const __grid_constant__ Maps maps) {
  using T = Tile<kPair>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + T::kStages * T::kStage);
  volatile int* abort = &sh.abort;
  uint32_t* status = muon_status(p.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPair ? cluster_rank() : 0u;
  const MuonTable& t = *muon_table(p.ws);
  for (int i = threadIdx.x; i <= p.count; i += kThreads) {
    sh.prefix[kGram][i] = t.prefix[kUnitsGram][i];
    sh.prefix[kSquare][i] = t.prefix[kUnitsSquare][i];
    sh.prefix[kUpdate][i] = t.prefix[kUnitsUpdate][i];
    if (i < p.count) sh.block[i] = Block{t.mat[i].base, t.mat[i].m, t.mat[i].n};
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], kPair ? 16 : 8);
    }
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    fence_mbar_init();
    if constexpr (kPair) {
      tma_prefetch_map(&maps.rows128);
      tma_prefetch_map(&maps.rows64);
    }
  }
  if (warp == 1) {
    if constexpr (kPair) tmem_alloc_pair(&sh.tmem, T::kCols);
    else tmem_alloc(&sh.tmem, T::kCols);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) {
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tmem = sh.tmem, base = smem_addr(smem);

  if (warp == 0) {
    if (lane == 0) {
      Ring<kPair> ring;
      Deal<kPair> deal;
      bool ok = true;
      for (int ph = 0; ph < 3 * p.K && ok; ++ph) {
        const int it = ph / 3, e = ph - 3 * it;
        ok = e == kGram ? produce<kPair, kGram>(p, maps, sh, ring, deal, it, base, rank, abort)
             : e == kSquare ? produce<kPair, kSquare>(p, maps, sh, ring, deal, it, base, rank, abort)
                            : produce<kPair, kUpdate>(p, maps, sh, ring, deal, it, base, rank, abort);
      }
      // every copy lands before the CTA or the pair may exit (a pair's count on the leader's barriers)
      if (rank == 0) await_own(sh.full, T::kStages, ring.issued, status);
      if constexpr (kPair) tell_issued(&sh.issued[rank], ring.issued);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      Ring<kPair> ring;
      Deal<kPair> deal;
      uint32_t tl = 0;
      bool ok = !p.stall || mbar_wait(&sh.done, 0, status, abort);     // (test only: a wait that runs out)
      for (int ph = 0; ph < 3 * p.K && ok; ++ph) {
        const int e = ph % 3;
        ok = e == kGram ? multiply<kPair, kGram>(p, sh, ring, deal, tl, base, tmem, abort)
             : e == kSquare ? multiply<kPair, kSquare>(p, sh, ring, deal, tl, base, tmem, abort)
                            : multiply<kPair, kUpdate>(p, sh, ring, deal, tl, base, tmem, abort);
      }
      if constexpr (kPair) tc_commit_pair(&sh.done);
      else tc_commit(&sh.done);
      volatile int never = 0;
      mbar_wait(&sh.done, 0, status, &never);
    }
  } else {
    const int quad_ = warp & 3, half = (warp - 2) >> 2;
    Deal<kPair> deal;
    uint32_t tl = 0;
    bool ok = true;
    for (int ph = 0; ph < 3 * p.K && (ok || !kPair); ++ph) {
      const int it = ph / 3, e = ph - 3 * it;
      ok = e == kGram ? finish<kPair, kGram, false>(p, sh, deal, tl, it, tmem, rank, quad_, half, lane, abort, ok)
           : e == kSquare ? finish<kPair, kSquare, false>(p, sh, deal, tl, it, tmem, rank, quad_, half, lane, abort, ok)
           : it < p.K - 1 ? finish<kPair, kUpdate, false>(p, sh, deal, tl, it, tmem, rank, quad_, half, lane, abort, ok)
                          : finish<kPair, kUpdate, true>(p, sh, deal, tl, it, tmem, rank, quad_, half, lane, abort, ok);
    }
  }
  __syncwarp();
  // (pairs) the leader's MMAs read the other CTA's memory: neither leaves before both are done
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) {
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  if constexpr (kPair) {
    if (rank == 0 && threadIdx.x == 0) await_issued(sh.full, T::kStages, T::kStage, sh.issued[0], sh.issued[1], status);
  }
  if (warp == 1) {
    if constexpr (kPair) tmem_dealloc_pair(tmem, T::kCols);
    else tmem_dealloc(tmem, T::kCols);
  }
  if constexpr (kPair) {
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
}

}  // namespace

cudaError_t launch_muon_iterate(const MuonCall& c, int64_t ws_bytes, int32_t units, cudaStream_t st, int num_sms) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  Maps maps{};
  cudaError_t e;
  if (c.small) {
    static PairSlots set;       // devices whose shared-memory limit is raised
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set.pairs[dev] == 0) {
      if ((e = cudaFuncSetAttribute(muon_iterate_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<false>)) != cudaSuccess)
        return e;
      set.pairs[dev] = 1;
    }
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(units < num_sms ? units : num_sms));
    cfg.dynamicSmemBytes = kSmem<false>;
    return cudaLaunchKernelEx(&cfg, muon_iterate_kernel<false>, c, maps);
  }
  static PairSlots slots;
  int pairs = 0;
  if ((e = pair_slots(slots, muon_iterate_kernel<true>, kThreads, kSmem<true>, &pairs)) != cudaSuccess) return e;
  if ((e = make_row_map(&maps.rows128, c.ws, ws_bytes / 128 * 128, 128)) != cudaSuccess) return e;
  if ((e = make_row_map(&maps.rows64, c.ws, ws_bytes / 128 * 128, 64)) != cudaSuccess) return e;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
  cfg.dynamicSmemBytes = kSmem<true>;
  return cudaLaunchKernelEx(&cfg, muon_iterate_kernel<true>, c, maps);
}

}  // namespace fs4
