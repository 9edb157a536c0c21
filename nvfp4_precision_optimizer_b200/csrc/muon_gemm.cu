// The three products of a Muon Newton-Schulz iteration on FP16 operands (sm_100a, tcgen05
// kind::f16 on CTA pairs, FP32 accumulation in TMEM):
//   GramX   A  = X X^T
//   GramA   B  = b A + c A^2
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
#include <cstdint>

#include "muon_device.cuh"
#include "pair_device.cuh"

namespace fs4 {
namespace {

constexpr int kThreads = 320;               // warp 0 producer, warp 1 MMA issuer, warps 2-9 epilogue
constexpr int kStages = 6;
constexpr int kOperand = 16384;             // bytes of one operand's half in a stage: 128 rows x 64 k
constexpr int kStage = 2 * kOperand;
constexpr int kSmem = 1024 + kStages * kStage + 256;
constexpr uint32_t kCols = 512;             // two 256-column accumulators
static_assert(kSmem <= 232448, "over the per-CTA shared-memory limit");

// One 256 x 256 output block.
struct Job {
  int mat;
  int32_t I, J;        // block row and column
  int32_t steps;       // K / 64
};

template <MuonProduct E>
__device__ __forceinline__ Job make_job(const MuonParams& p, int32_t u) {
  Job j;
  j.mat = owner_of(p.prefix, p.count, u);
  const MuonMat& d = p.mat[j.mat];
  int32_t t = u - p.prefix[j.mat];
  if constexpr (E == MuonProduct::Update) {
    const int32_t nj = d.np / 256;
    j.I = t / nj;
    j.J = t - j.I * nj;
    j.steps = d.mp / 64;
  } else {
    const int32_t T = d.mp / 256;
    j.I = 0;
    while (t >= T - j.I) { t -= T - j.I; ++j.I; }
    j.J = j.I + t;
    j.steps = (E == MuonProduct::GramX ? d.np : d.mp) / 64;
  }
  return j;
}

// This CTA's half (128 rows of M or N from block row `blk`) of a symmetric operand's k step:
// the stored block, or the mirror of the one above the diagonal.  Both are 16 KB.
__device__ __forceinline__ bool mirrored(int32_t blk, int32_t k) { return (k >> 2) < blk; }

__device__ __forceinline__ void load_rows(uint32_t dst, const uint8_t* src, int64_t cp, int64_t row0, int32_t k, uint64_t* bar) {
  bulk_g2s_addr(dst, src + ((row0 >> 7) * (cp >> 6) + k) * (int64_t)kOperand, kOperand, bar);
}
// 64 stored rows from 64 k on, 128 columns from col0 on: two 64-column pieces.
__device__ __forceinline__ void load_columns(uint32_t dst, const uint8_t* src, int64_t cp, int64_t col0, int32_t k, uint64_t* bar) {
  const uint8_t* s = src + ((int64_t)(k >> 1) * (cp >> 6) + (col0 >> 6)) * kOperand + (k & 1) * (kOperand / 2);
  bulk_g2s_addr(dst, s, kOperand / 2, bar);
  bulk_g2s_addr(dst + kOperand / 2, s + kOperand, kOperand / 2, bar);
}

__device__ __forceinline__ uint32_t two_halves(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// v[8] = (high + low / 2^11) of one 16-byte chunk each.
__device__ __forceinline__ void join8(uint4 hi, uint4 lo, float* v) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = fmaf(half_lo(l[i]), 1.0f / kLowScale, half_lo(h[i]));
    v[2 * i + 1] = fmaf(half_hi(l[i]), 1.0f / kLowScale, half_hi(h[i]));
  }
}
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = two_halves(v[2 * i], v[2 * i + 1]);
    l[i] = two_halves((v[2 * i] - half_lo(h[i])) * kLowScale, (v[2 * i + 1] - half_hi(h[i])) * kLowScale);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// One epilogue warp: rows 32 quad .. + 31 of this CTA's 128, columns 128 half .. + 127.
template <MuonProduct E>
__device__ __forceinline__ void epilogue(const MuonParams& p, const Job& j, uint32_t acc, uint32_t rank, int quad, int half,
                                         int lane) {
  const MuonMat& d = p.mat[j.mat];
  const MuonLayout L = muon_layout(d.mp, d.np);
  uint8_t* ws = p.ws + d.base;
  const int64_t row = 256ll * j.I + 128 * rank + 32 * quad + lane;     // this lane's row
  const int64_t col0 = 256ll * j.J + 128 * half;
  const int64_t cp = E == MuonProduct::Update ? d.np : d.mp;
  const uint32_t taddr = acc + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * half);
  const uint8_t* in_hi = ws + (E == MuonProduct::Update ? (p.slot ? L.x[1] : L.x[0]) : L.a);
  const uint8_t* in_lo = ws + (E == MuonProduct::Update ? L.xl : L.al);
  uint8_t* out_hi = ws + (E == MuonProduct::Update ? (p.slot ? L.x[0] : L.x[1]) : E == MuonProduct::GramA ? L.b : L.a);
  uint8_t* out_lo = ws + (E == MuonProduct::Update ? L.xl : L.al);
  const float* da = reinterpret_cast<const float*>(ws + L.da);
  float d_row = 0.0f, e_row = 0.0f;
  if constexpr (E == MuonProduct::GramA) d_row = da[row];
  if constexpr (E == MuonProduct::Update) e_row = p.a + reinterpret_cast<const float*>(ws + L.db)[row];
  const bool diagonal = E != MuonProduct::Update && j.I == j.J;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float v[32];
    tmem_ld32(taddr + c, v);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t col = col0 + c + 8 * q;
      const int64_t off = tiled_chunk_offset_bf16(row, col, cp);
      float x[8], y[8];
      if constexpr (E != MuonProduct::GramX)
        join8(*reinterpret_cast<const uint4*>(in_hi + off), *reinterpret_cast<const uint4*>(in_lo + off), x);
      if constexpr (E == MuonProduct::GramX) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[8 * q + i] * (kAScale / (kXScale * kXScale));
        if (diagonal && row >= col && row < col + 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (row == col + i) {
              reinterpret_cast<float*>(ws + L.da)[row] = y[i] * (1.0f / kAScale);
              y[i] = 0.0f;
            }
        }
      } else if constexpr (E == MuonProduct::GramA) {
        const float4 d0 = *reinterpret_cast<const float4*>(da + col), d1 = *reinterpret_cast<const float4*>(da + col + 4);
        const float dc[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        // kAScale times b A0 + c (A0^2 + A0 (d_i + d_j))
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], fmaf(p.c, d_row + dc[i], p.b), v[8 * q + i] * (p.c / kAScale));
        if (diagonal && row >= col && row < col + 8) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (row == col + i) {
              reinterpret_cast<float*>(ws + L.db)[row] =
                  fmaf(d_row, fmaf(p.c, d_row, p.b), v[8 * q + i] * (p.c / (kAScale * kAScale)));
              y[i] = 0.0f;
            }
        }
      } else {
        // kXScale times (a + e_i) X + B0 X
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(e_row, x[i], v[8 * q + i] * (1.0f / kAScale));
      }
      if (E == MuonProduct::Update && p.last) {
        if (row < d.m) {
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (col + i >= d.n) continue;
            const float u = y[i] * (1.0f / kXScale) * d.scale;
            bad |= !isfinite(u);
            const int64_t at = d.tall ? (col + i) * d.ldw + row : row * d.ldw + col + i;
            put1(d.w, at, d.tw, p.rate < 0.0f ? u : fmaf(-p.rate, u, p.keep * get1(d.w, at, d.tw)));
          }
          if (bad) atomicOr(p.status, kStatusNonFinite);
        }
      } else {
        uint4 hi, lo;
        split8(y, hi, lo);
        *reinterpret_cast<uint4*>(out_hi + off) = hi;
        if constexpr (E != MuonProduct::GramA) *reinterpret_cast<uint4*>(out_lo + off) = lo;
      }
    }
  }
}

template <MuonProduct E>
__global__ void __launch_bounds__(kThreads, 1) muon_product_kernel(const __grid_constant__ MuonParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStage);   // this CTA's halves landed
  uint64_t* peer = full + kStages;             // leader: the other CTA's halves landed
  uint64_t* empty = peer + kStages;            // the MMAs reading the stage finished (both CTAs)
  uint64_t* acc_full = empty + kStages;        // [2]
  uint64_t* acc_empty = acc_full + 2;          // [2] leader: both CTAs drained the accumulator
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int32_t total = p.prefix[p.count];

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&peer[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 16);
    }
    mbar_init(done, 1);
    *abort_flag = (__ldcg(p.status) & kStatusTimeout) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kCols);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t base = smem_addr(smem);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int32_t u = first; u < total && ok; u += step) {
        const Job j = make_job<E>(p, u);
        const MuonMat& d = p.mat[j.mat];
        const MuonLayout L = muon_layout(d.mp, d.np);
        const uint8_t* ws = p.ws + d.base;
        const uint8_t* x = ws + (p.slot ? L.x[1] : L.x[0]);
        const int64_t rowI = 256ll * j.I + 128 * rank, rowJ = 256ll * j.J + 128 * rank;
        for (int32_t k = 0; k < j.steps; ++k) {
          if (!mbar_wait(&empty[s], ph ^ 1u, p.status, abort_flag)) { ok = false; break; }
          const uint32_t a = base + s * kStage, b = a + kOperand;
          mbar_arrive_expect_tx(&full[s], kStage);
          if constexpr (E == MuonProduct::GramX) {
            load_rows(a, x, d.np, rowI, k, &full[s]);
            load_rows(b, x, d.np, rowJ, k, &full[s]);
          } else {
            const uint8_t* sym = ws + (E == MuonProduct::GramA ? L.a : L.b);
            if (mirrored(j.I, k)) load_columns(a, sym, d.mp, rowI, k, &full[s]);
            else load_rows(a, sym, d.mp, rowI, k, &full[s]);
            if constexpr (E == MuonProduct::Update) load_columns(b, x, d.np, rowJ, k, &full[s]);
            else if (mirrored(j.J, k)) load_columns(b, sym, d.mp, rowJ, k, &full[s]);
            else load_rows(b, sym, d.mp, rowJ, k, &full[s]);
          }
          ++issued;
          if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
        }
      }
      // every issued copy lands before the CTA may exit
      for (uint32_t i = issued > (uint32_t)kStages ? issued - kStages : 0u; i < issued; ++i) {
        volatile int never = 0;
        mbar_wait(&full[i % kStages], (i / kStages) & 1u, p.status, &never);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank != 0) {
      // tell the leader when this CTA's halves of a stage have landed
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int32_t u = first; u < total && ok; u += step) {
        const Job j = make_job<E>(p, u);
        for (int32_t k = 0; k < j.steps; ++k) {
          if (!mbar_wait(&full[s], ph, p.status, abort_flag)) { ok = false; break; }
          mbar_arrive_cluster(cluster_map(smem_addr(&peer[s]), 0));
          if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
        }
      }
    } else if (lane == 0) {
      uint32_t s = 0, ph = 0, tl = 0;
      bool ok = true;
      const uint64_t ra0 = sdesc_sw128(base), rb0 = sdesc_sw128(base + kOperand);
      const uint64_t ca0 = sdesc_sw128_mn(base, kOperand / 2), cb0 = sdesc_sw128_mn(base + kOperand, kOperand / 2);
      constexpr uint64_t kStep = kStage >> 4;
      for (int32_t u = first; u < total && ok; u += step, ++tl) {
        const Job j = make_job<E>(p, u);
        const uint32_t acc = tmem + 256u * (tl & 1u);
        if (!mbar_wait_cluster(&acc_empty[tl & 1u], ((tl >> 1) & 1u) ^ 1u, p.status, abort_flag)) break;
        tc_fence_after();
        for (int32_t k = 0; k < j.steps; ++k) {
          if (!mbar_wait(&full[s], ph, p.status, abort_flag) || !mbar_wait_cluster(&peer[s], ph, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const bool am = E != MuonProduct::GramX && mirrored(j.I, k);
          const bool bm = E == MuonProduct::Update || (E == MuonProduct::GramA && mirrored(j.J, k));
          // 16 k: 32 bytes along a row, or 16 rows of 128 bytes
          const uint64_t da = (am ? ca0 : ra0) + s * kStep, db = (bm ? cb0 : rb0) + s * kStep;
          const uint64_t ia = am ? 128 : 2, ib = bm ? 128 : 2;
          const uint32_t idesc = idesc_f16(256, 256, am, bm);
#pragma unroll
          for (int h = 0; h < 4; ++h) tc_mma_f16_pair(acc, da + h * ia, db + h * ib, idesc, (k | h) != 0 ? 1u : 0u);
          tc_commit_pair(&empty[s]);
          if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(&acc_full[tl & 1u]);
      }
      tc_commit_pair(done);
      volatile int never = 0;
      mbar_wait(done, 0, p.status, &never);
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint32_t tl = 0;
    for (int32_t u = first; u < total; u += step, ++tl) {
      const Job j = make_job<E>(p, u);
      const uint32_t b = tl & 1u;
      const bool ok = __shfl_sync(0xFFFFFFFFu, lane == 0 ? (mbar_wait(&acc_full[b], (tl >> 1) & 1u, p.status, abort_flag) ? 1 : 0) : 0, 0) != 0;
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      epilogue<E>(p, j, tmem + 256u * b, rank, quad, half, lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(smem_addr(&acc_empty[b]), 0));
    }
  }
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

template <MuonProduct E>
cudaError_t launch_product(const MuonParams& p, cudaStream_t st, int num_sms) {
  // CTA pairs that are resident at once, by device (a pair needs two SMs of one cluster)
  static int pairs[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.gridDim = dim3((unsigned)(num_sms & ~1));
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (pairs[dev] == 0) {
    if ((e = cudaFuncSetAttribute(muon_product_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, muon_product_kernel<E>, &cfg)) != cudaSuccess) return e;
    pairs[dev] = n > 0 ? n : 1;
  }
  const int total = p.prefix[p.count];
  cfg.gridDim = dim3((unsigned)(2 * (total < pairs[dev] ? total : pairs[dev])));
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, muon_product_kernel<E>, p);
}

}  // namespace

cudaError_t launch_muon_product(MuonProduct e, const MuonParams& p, cudaStream_t st, int num_sms) {
  switch (e) {
    case MuonProduct::GramX: return launch_product<MuonProduct::GramX>(p, st, num_sms);
    case MuonProduct::GramA: return launch_product<MuonProduct::GramA>(p, st, num_sms);
    default: return launch_product<MuonProduct::Update>(p, st, num_sms);
  }
}

}  // namespace fs4
