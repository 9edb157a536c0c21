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
// which the epilogues add from the FP32 diagonals.  Measured on Gaussian and low-rank inputs
// (numpy, 256^2 to 768 x 2048): 0.4-1.3e-3 from the exact iteration after five steps, against
// 2.6e-3 with rounded diagonals and 1.4-2.4e-2 with BF16 operands.
// A and B are symmetric: only 256 x 256 blocks on and above the diagonal are computed and
// stored.  A block below it is read as its mirror image with the operand's M or N index
// fastest, which the tensor core takes directly; so is X as the second operand of the update,
// whose rows are its K index.  Nothing is stored twice.
// Structure.  A pair of CTAs computes a 256 x 256 block, 128 rows and 256 TMEM columns each;
// either operand's 256 rows are split over the two, so that a 64-deep stage costs each SM 32 KB
// for 512 cycles of MMAs (a single CTA's 128 x 256 tile would cost 48 KB, more than the 67
// bytes a cycle that L2 delivers to an SM).  Two accumulators: a block's epilogue overlaps the
// next block's MMAs.  Both CTAs' copies count on the leader's barrier (tensor maps allow that);
// a relay through the other CTA's threads took 1300 cycles a stage.  Between products the
// launch's CTAs meet at a counter in the workspace (a cooperative launch: all are resident; the
// wait is bounded), which saves 3K - 1 launches and their set-up.
#include <cstdint>
#include <cstddef>
#include <type_traits>

#include "muon_device.cuh"
#include "pair_device.cuh"
#include "pair_host.h"

namespace fs4 {
namespace {

constexpr int kThreads = 320;               // warp 0 producer, warp 1 MMA issuer, warps 2-9 epilogue
constexpr int kStages = 6;
constexpr int kOperand = 16384;             // bytes of one operand's half in a stage: 128 rows x 64 k
constexpr int kStage = 2 * kOperand;
constexpr uint32_t kCols = 512;             // two 256-column accumulators
constexpr int kGroup = 8;                   // block rows of a raster group: pairs at work share operands in L2

// What the roles need of a matrix, in shared memory.
struct Block {
  int64_t base;
  int32_t mp, np;
};
struct Shared {
  uint64_t full[kStages];      // leader: both CTAs' operands of a stage landed
  uint64_t empty[kStages];     // the MMAs reading the stage finished (both CTAs)
  uint64_t acc_full[2];
  uint64_t acc_empty[2];       // leader: both CTAs drained the accumulator
  uint64_t go;                 // the producer saw every CTA finish the product before
  uint64_t done;
  uint32_t tmem;
  int32_t abort;
  alignas(16) float diag[8][128];   // an epilogue warp's columns of A's diagonal
  int32_t prefix[2][kMuonMaxBatch + 1];   // units of the Gram products and of the update
  Block block[kMuonMaxBatch];
};
constexpr int kSmem = 1024 + kStages * kStage + (int)sizeof(Shared);
static_assert(kSmem <= 232448, "over the per-CTA shared-memory limit");
static_assert(offsetof(Shared, diag) % 16 == 0 && kStages * kStage % 1024 == 0, "read and written 16 bytes at a time");

enum { kGram = 0, kSquare = 1, kUpdate = 2 };

// One 256 x 256 output block.
struct Job {
  int mat;
  int32_t I, J;        // block row and column
  int32_t steps;       // K / 64
};

// Unit u of a product.  Within a matrix the blocks go through groups of kGroup block rows,
// column by column, so that the pairs at work read few operand rows and columns.
template <int E>
__device__ __forceinline__ Job make_job(const Shared& sh, int count, int32_t u) {
  const int32_t* prefix = sh.prefix[E == kUpdate ? 1 : 0];
  Job j;
  j.mat = owner_of(prefix, count, u);
  const Block& d = sh.block[j.mat];
  int32_t t = u - prefix[j.mat];
  const int32_t T = d.mp / 256;
  if constexpr (E == kUpdate) {
    const int32_t nj = d.np / 256, g = t / (kGroup * nj), h = min(kGroup, T - kGroup * g);
    t -= g * kGroup * nj;
    j.J = t / h;
    j.I = kGroup * g + t % h;
    j.steps = d.mp / 64;
  } else {
    int32_t r0 = 0;
    for (;; r0 += kGroup) {                 // blocks on and above the diagonal
      const int32_t h = min(kGroup, T - r0), tri = h * (h + 1) / 2, size = tri + h * (T - r0 - h);
      if (t >= size) { t -= size; continue; }
      if (t >= tri) {
        j.J = r0 + h + (t - tri) / h;
        j.I = r0 + (t - tri) % h;
      } else {
        int32_t c = 0;
        while (t > c) t -= ++c;
        j.J = r0 + c;
        j.I = r0 + t;
      }
      break;
    }
    j.steps = (E == kGram ? d.np : d.mp) / 64;
  }
  return j;
}

// Whether block row `blk` of a symmetric operand at k step `k` is read as its mirror image.
__device__ __forceinline__ bool mirrored(int32_t blk, int32_t k) { return (k >> 2) < blk; }

struct Maps {
  CUtensorMap rows128, rows64;     // the workspace as 128-byte rows, copied 128 or 64 at a time
};

// 128 rows of M or N from row0 on, 64 k: one tile.
__device__ __forceinline__ void load_rows(const Maps& m, uint32_t dst, int64_t src, int32_t cp, int32_t row0, int32_t k, uint32_t bar) {
  tma_rows_pair(dst, &m.rows128, (int32_t)((src >> 7) + ((int64_t)(row0 >> 7) * (cp >> 6) + k) * 128), bar);
}
// 64 stored rows from 64 k on, 128 columns from col0 on: halves of two neighbouring tiles.
__device__ __forceinline__ void load_columns(const Maps& m, uint32_t dst, int64_t src, int32_t cp, int32_t col0, int32_t k, uint32_t bar) {
  const int32_t row = (int32_t)((src >> 7) + ((int64_t)(k >> 1) * (cp >> 6) + (col0 >> 6)) * 128 + (k & 1) * 64);
  tma_rows_pair(dst, &m.rows64, row, bar);
  tma_rows_pair(dst + kOperand / 2, &m.rows64, row + 128, bar);
}

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
template <typename T>
__device__ __forceinline__ void write_result(const MuonCall& p, const MuonMat& d, int32_t row, int32_t col, const float* y, bool& bad) {
  if (row >= d.m) return;
  constexpr int kPer = 32 / (int)sizeof(T);                  // elements of 32 bytes
  const bool blend = p.rate >= 0.0f;
  auto result = [&](float x, float w) -> float {
    const float u = x * d.scale;
    bad |= !isfinite(u);
    return blend ? fmaf(-p.rate, u, p.keep * w) : u;
  };
  T* w = static_cast<T*>(d.w);
  if (!d.tall && col + 32 <= d.n && ((reinterpret_cast<uintptr_t>(w) | (uintptr_t)(d.ldw * (int64_t)sizeof(T))) & 31) == 0) {
    T* at = w + row * d.ldw + col;
#pragma unroll
    for (int q = 0; q < 32 / kPer; ++q) {
      Pair r{};
      if (blend) r = load_pair(at + q * kPer);
      T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if constexpr (sizeof(T) == 4) e[i] = result(y[q * kPer + i], e[i]);
        else if constexpr (std::is_same<T, __half>::value) e[i] = __float2half_rn(result(y[q * kPer + i], __half2float(e[i])));
        else e[i] = __float2bfloat16_rn(result(y[q * kPer + i], __bfloat162float(e[i])));
      }
      store_pair(at + q * kPer, r);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (col + i >= d.n) break;
    const int64_t at = d.tall ? (int64_t)(col + i) * d.ldw + row : row * d.ldw + col + i;
    put_as(w + at, result(y[i], blend ? get_as(w + at) : 0.0f));
  }
}

// Input of 32 columns: A or X, high and low parts.
struct Input {
  Pair h[2], l[2];
};

// What one epilogue warp (rows 32 quad .. + 31 of this CTA's 128, columns 128 half .. + 127) reads
// and writes of a block.
template <int E>
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

  __device__ __forceinline__ Place(const MuonCall& p, const Shared& sh, const Job& j, int it, uint32_t rank, int quad_, int half,
                                   int lane) {
    const Block& d = sh.block[j.mat];
    const MuonLayout L = muon_layout(d.mp, d.np);
    uint8_t* ws = p.ws + d.base;
    const int32_t cp = E == kUpdate ? d.np : d.mp;
    const bool odd = (it & 1) != 0;
    row = 256 * j.I + 128 * (int32_t)rank + 32 * quad_ + lane;
    col0 = 256 * j.J + 128 * half;
    const int64_t tile = ((int64_t)(row >> 7) * (cp >> 6) + (col0 >> 6)) * kOperand + (row & 127) * 128;
    in_hi = ws + (E == kUpdate ? (odd ? L.x[1] : L.x[0]) : L.a) + tile;
    in_lo = ws + (E == kUpdate ? L.xl : L.al) + tile;
    out_hi = ws + (E == kUpdate ? (odd ? L.x[0] : L.x[1]) : E == kSquare ? L.b : L.a) + tile;
    out_lo = ws + (E == kUpdate ? L.xl : L.al) + tile;
    da = reinterpret_cast<float*>(ws + L.da);
    db = reinterpret_cast<float*>(ws + L.db);
    swap = (row & 1) != 0;
    x6 = row & 6;
    diagonal = E != kUpdate && j.I == j.J;
  }
  // 32-byte piece i (0, 1) of the 32 columns from c (0, 32, 64, 96) on
  __device__ __forceinline__ int piece(int c, int i) const { return (c >> 6) * kOperand + 16 * ((((c & 32) >> 3) + 2 * i) ^ x6); }
  __device__ __forceinline__ void load(Input& in, int c) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      in.h[i] = load_pair(in_hi + piece(c, i));
      in.l[i] = load_pair(in_lo + piece(c, i));
    }
  }
};

// Before the accumulator is ready: half of the warp's input and the diagonal entries.
struct Ahead {
  Input in[2];
  float own;             // d_i (Square) or a + e_i (Update)
};
template <int E>
__device__ __forceinline__ void look_ahead(const MuonCall& p, const Place<E>& w, Ahead& a, float* diag, int it, int lane) {
  if constexpr (E == kGram) return;
  w.load(a.in[0], 0);
  w.load(a.in[1], 32);
  if constexpr (E == kSquare) {
    a.own = __ldcg(w.da + w.row);
    const float4 c = __ldcg(reinterpret_cast<const float4*>(w.da + w.col0) + lane);
    __syncwarp();
    reinterpret_cast<float4*>(diag)[lane] = c;
    __syncwarp();
  } else {
    a.own = p.coeffs[p.n_coeffs == 1 ? 0 : 3 * it] + __ldcg(w.db + w.row);
  }
}

template <int E>
__device__ __forceinline__ void epilogue(const MuonCall& p, const Place<E>& w, Ahead& a, const float* diag, const MuonMat* m, int it,
                                         uint32_t taddr, int lane) {
  const bool last = E == kUpdate && it == p.K - 1;
  const float* poly = p.coeffs + (p.n_coeffs == 1 ? 0 : 3 * it);
  const float pb = poly[1], pc = poly[2];
  bool bad = false;
  // (rolled: a block's epilogue runs once per product, and its instructions come from L2)
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float v[32];
    tmem_ld32(taddr + c, v);
    const int32_t col = w.col0 + c;
    // the 32 x 32 part on the diagonal (whole warps: rows and columns are multiples of 32)
    const bool on = w.diagonal && (w.row & ~31) == col;
    if constexpr (E == kGram) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= kAScale / (kXScale * kXScale);
      if (on) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (lane == i) {
            w.da[w.row] = v[i] * (1.0f / kAScale);
            v[i] = 0.0f;
          }
      }
    } else {
      const Input in = a.in[0];
      a.in[0] = a.in[1];
      if (c < 64) w.load(a.in[1], c + 64);       // the input two steps on
      float e = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float* y = v + 8 * q;
        float x[8];
        join8(quad(ordered(in.h[q >> 1], w.swap), q & 1), quad(ordered(in.l[q >> 1], w.swap), q & 1), x);
        if constexpr (E == kSquare) {
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
          // kXScale times (a + e_i) X + B0 X
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = fmaf(a.own, x[i], y[i] * (1.0f / kAScale));
        }
      }
      if (E == kSquare && on) {
        w.db[w.row] = fmaf(a.own, fmaf(pc, a.own, pb), e * (pc / (kAScale * kAScale)));
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (lane == i) v[i] = 0.0f;
      }
    }
    if (last) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= 1.0f / kXScale;
      if (m->tw == kTypeF32) write_result<float>(p, *m, w.row, col, v, bad);
      else if (m->tw == kTypeBf16) write_result<__nv_bfloat16>(p, *m, w.row, col, v, bad);
      else write_result<__half>(p, *m, w.row, col, v, bad);
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
  if (bad) atomicOr(muon_status(p.ws), kStatusNonFinite);
}

// ------------------------------------------------------------------ the launch's barrier
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
struct Ring {
  uint32_t s = 0, ph = 0, issued = 0;
  __device__ __forceinline__ void next() {
    ++issued;
    if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
  }
};

template <int E>
__device__ __forceinline__ bool produce(const MuonCall& p, const Maps& maps, Shared& sh, Ring& ring, int it, uint32_t base,
                                        uint32_t rank, volatile int* abort) {
  const int32_t total = sh.prefix[E == kUpdate ? 1 : 0][p.count];
  for (int32_t u = blockIdx.x >> 1; u < total; u += gridDim.x >> 1) {
    const Job j = make_job<E>(sh, p.count, u);
    const Block& d = sh.block[j.mat];
    const MuonLayout L = muon_layout(d.mp, d.np);
    const int64_t x = d.base + ((it & 1) ? L.x[1] : L.x[0]);
    const int64_t sym = d.base + (E == kSquare ? L.a : L.b);
    const int32_t rowI = 256 * j.I + 128 * (int32_t)rank, rowJ = 256 * j.J + 128 * (int32_t)rank;
    for (int32_t k = 0; k < j.steps; ++k) {
      if (!mbar_wait(&sh.empty[ring.s], ring.ph ^ 1u, muon_status(p.ws), abort)) return false;
      const uint32_t a = base + ring.s * kStage, b = a + kOperand;
      const uint32_t bar = cluster_map(smem_addr(&sh.full[ring.s]), 0);
      if (rank == 0) mbar_arrive_expect_tx(&sh.full[ring.s], 2 * kStage);
      if constexpr (E == kGram) {
        load_rows(maps, a, x, d.np, rowI, k, bar);
        load_rows(maps, b, x, d.np, rowJ, k, bar);
      } else {
        if (mirrored(j.I, k)) load_columns(maps, a, sym, d.mp, rowI, k, bar);
        else load_rows(maps, a, sym, d.mp, rowI, k, bar);
        if constexpr (E == kUpdate) load_columns(maps, b, x, d.np, rowJ, k, bar);
        else if (mirrored(j.J, k)) load_columns(maps, b, sym, d.mp, rowJ, k, bar);
        else load_rows(maps, b, sym, d.mp, rowJ, k, bar);
      }
      ring.next();
    }
  }
  return true;
}

template <int E>
__device__ __forceinline__ bool multiply(const MuonCall& p, Shared& sh, Ring& ring, uint32_t& tl, uint32_t base, uint32_t tmem,
                                         volatile int* abort) {
  const uint64_t ra0 = sdesc_sw128(base), rb0 = sdesc_sw128(base + kOperand);
  const uint64_t ca0 = sdesc_sw128_mn(base, kOperand / 2), cb0 = sdesc_sw128_mn(base + kOperand, kOperand / 2);
  constexpr uint64_t kStep = kStage >> 4;
  const int32_t total = sh.prefix[E == kUpdate ? 1 : 0][p.count];
  for (int32_t u = blockIdx.x >> 1; u < total; u += gridDim.x >> 1, ++tl) {
    const Job j = make_job<E>(sh, p.count, u);
    const uint32_t acc = tmem + 256u * (tl & 1u);
    if (!mbar_wait_cluster(&sh.acc_empty[tl & 1u], ((tl >> 1) & 1u) ^ 1u, muon_status(p.ws), abort)) return false;
    tc_fence_after();
    for (int32_t k = 0; k < j.steps; ++k) {
      if (!mbar_wait_cluster(&sh.full[ring.s], ring.ph, muon_status(p.ws), abort)) return false;
      tc_fence_after();
      const bool am = E != kGram && mirrored(j.I, k);
      const bool bm = E == kUpdate || (E == kSquare && mirrored(j.J, k));
      // 16 k: 32 bytes along a row, or 16 rows of 128 bytes
      const uint64_t da = (am ? ca0 : ra0) + ring.s * kStep, db = (bm ? cb0 : rb0) + ring.s * kStep;
      const uint64_t ia = am ? 128 : 2, ib = bm ? 128 : 2;
      const uint32_t idesc = idesc_f16(256, 256, am, bm);
#pragma unroll
      for (int h = 0; h < 4; ++h) tc_mma_f16_pair(acc, da + h * ia, db + h * ib, idesc, (k | h) != 0 ? 1u : 0u);
      tc_commit_pair(&sh.empty[ring.s]);
      ring.next();
    }
    tc_commit_pair(&sh.acc_full[tl & 1u]);
  }
  return true;
}

template <int E>
__device__ __forceinline__ bool finish(const MuonCall& p, Shared& sh, uint32_t& tl, int it, uint32_t tmem, uint32_t rank, int quad_,
                                       int half, int lane, volatile int* abort) {
  const int32_t total = sh.prefix[E == kUpdate ? 1 : 0][p.count];
  for (int32_t u = blockIdx.x >> 1; u < total; u += gridDim.x >> 1, ++tl) {
    const Job j = make_job<E>(sh, p.count, u);
    const uint32_t b = tl & 1u;
    const Place<E> w(p, sh, j, it, rank, quad_, half, lane);
    float* diag = sh.diag[4 * half + quad_];
    Ahead a;
    look_ahead<E>(p, w, a, diag, it, lane);
    const int got = lane == 0 ? (mbar_wait(&sh.acc_full[b], (tl >> 1) & 1u, muon_status(p.ws), abort) ? 1 : 0) : 0;
    if (__shfl_sync(0xFFFFFFFFu, got, 0) == 0) return false;
    __syncwarp();
    tc_fence_after();
    epilogue<E>(p, w, a, diag, &muon_table(p.ws)->mat[j.mat], it,
                tmem + 256u * b + ((uint32_t)(32 * quad_) << 16) + (uint32_t)(128 * half), lane);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (rank == 0) mbar_arrive(&sh.acc_empty[b]);
      else mbar_arrive_remote(cluster_map(smem_addr(&sh.acc_empty[b]), 0));
    }
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) muon_iterate_kernel(const __grid_constant__ MuonCall p, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + kStages * kStage);
  volatile int* abort = &sh.abort;
  uint32_t* status = muon_status(p.ws);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const MuonTable& t = *muon_table(p.ws);
  for (int i = threadIdx.x; i <= p.count; i += kThreads) {
    sh.prefix[0][i] = t.prefix[kUnitsGram][i];
    sh.prefix[1][i] = t.prefix[kUnitsUpdate][i];
    if (i < p.count) sh.block[i] = Block{t.mat[i].base, t.mat[i].mp, t.mat[i].np};
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.acc_full[b], 1);
      mbar_init(&sh.acc_empty[b], 16);
    }
    mbar_init(&sh.go, 1);
    mbar_init(&sh.done, 1);
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&maps.rows128);
    tma_prefetch_map(&maps.rows64);
  }
  if (warp == 1) tmem_alloc_pair(&sh.tmem, kCols);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, base = smem_addr(smem);
  const uint32_t* count = muon_barrier(p.ws);

  if (warp == 0) {
    if (lane == 0) {
      Ring ring;
      bool ok = true;
      for (int ph = 0; ph < 3 * p.K && ok; ++ph) {
        if (ph > 0) {
          ok = wait_count(count, (uint32_t)ph * gridDim.x, status, abort);
          mbar_arrive(&sh.go);
          if (!ok) break;
          fence_async();
        }
        const int it = ph / 3, e = ph - 3 * it;
        ok = e == kGram ? produce<kGram>(p, maps, sh, ring, it, base, rank, abort)
             : e == kSquare ? produce<kSquare>(p, maps, sh, ring, it, base, rank, abort)
                            : produce<kUpdate>(p, maps, sh, ring, it, base, rank, abort);
      }
      // every copy lands before the pair may exit (they count on the leader's barriers)
      if (rank == 0) {
        for (uint32_t i = ring.issued > (uint32_t)kStages ? ring.issued - kStages : 0u; i < ring.issued; ++i) {
          volatile int never = 0;
          mbar_wait(&sh.full[i % kStages], (i / kStages) & 1u, status, &never);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      Ring ring;
      uint32_t tl = 0;
      bool ok = true;
      for (int ph = 0; ph < 3 * p.K && ok; ++ph) {
        const int e = ph % 3;
        ok = e == kGram ? multiply<kGram>(p, sh, ring, tl, base, tmem, abort)
             : e == kSquare ? multiply<kSquare>(p, sh, ring, tl, base, tmem, abort)
                            : multiply<kUpdate>(p, sh, ring, tl, base, tmem, abort);
      }
      tc_commit_pair(&sh.done);
      volatile int never = 0;
      mbar_wait(&sh.done, 0, status, &never);
    }
  } else {
    const int quad_ = warp & 3, half = (warp - 2) >> 2;
    uint32_t tl = 0;
    bool ok = true;
    for (int ph = 0; ph < 3 * p.K; ++ph) {
      const int it = ph / 3, e = ph - 3 * it;
      if (ph > 0 && ok) {                 // other CTAs' results are read below
        const int got = lane == 0 ? (mbar_wait(&sh.go, (uint32_t)(ph - 1) & 1u, status, abort) ? 1 : 0) : 0;
        ok = __shfl_sync(0xFFFFFFFFu, got, 0) != 0;
        __syncwarp();
      }
      if (ok)
        ok = e == kGram ? finish<kGram>(p, sh, tl, it, tmem, rank, quad_, half, lane, abort)
             : e == kSquare ? finish<kSquare>(p, sh, tl, it, tmem, rank, quad_, half, lane, abort)
                            : finish<kUpdate>(p, sh, tl, it, tmem, rank, quad_, half, lane, abort);
      // every thread's results before the count (the barrier orders them before the release);
      // a producer that sees the count fences its TMA copies behind it
      named_bar(1, 256);
      if (threadIdx.x == 64) {
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(muon_barrier(p.ws)), "r"(1u) : "memory");
      }
    }
  }
  __syncwarp();
  // the leader's MMAs read the other CTA's memory: neither leaves before both are done
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kCols);
  __syncthreads();
  cluster_arrive();
  cluster_wait();
}

}  // namespace

cudaError_t launch_muon_iterate(const MuonCall& c, int64_t ws_bytes, int32_t gram_units, int32_t update_units, cudaStream_t st) {
  static PairSlots slots;
  int pairs = 0;
  cudaError_t e = pair_slots(slots, muon_iterate_kernel, kThreads, kSmem, &pairs);
  if (e != cudaSuccess) return e;
  Maps maps;
  if ((e = make_row_map(&maps.rows128, c.ws, ws_bytes / 128 * 128, 128)) != cudaSuccess) return e;
  if ((e = make_row_map(&maps.rows64, c.ws, ws_bytes / 128 * 128, 64)) != cudaSuccess) return e;
  const int32_t units = gram_units > update_units ? gram_units : update_units;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeCooperative;
  at[1].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, muon_iterate_kernel, c, maps);
}

}  // namespace fs4
