// Large MXFP4 products (sm_100a): persistent CTA pairs, tcgen05.mma cta_group::2 kind::mxf4.
//
// A pair computes a 256 x 256 tile of D, 128 rows each; A's and B's 256 rows are split over the
// two CTAs' shared memory.  A stage of 256 K-elements costs an SM 35 KB (codes 32, scales 3) for
// four MMAs of 128 cycles, 70 bytes a cycle, about what L2 delivers to an SM; a single CTA's
// 128 x 256 tile would need 51 KB.  Scales go from shared memory to TMEM with tcgen05.cp, six
// atoms a stage (A's two, B's two bands of two), issued by a thread of their own: a copy takes
// about 52 cycles to issue and an MMA 66, and together they would exceed the stage's 512.
// TMEM holds one 256-column accumulator and the scales of every stage, so the epilogue drains
// the accumulator into registers first and hands it back before it converts and stores.
// Measured: 8192 x 8192 x 4096 to BF16 104 us, 5.3 PFLOP/s; 8192 x 16384 x 8192 375 us, 5.9 PFLOP/s,
// tensor pipe 78% active (a single CTA's 128 x 128 tiles: 822 us for the first).
#include <cstdint>

#include "mx_internal.h"
#include "pair_device.cuh"
#include "pair_host.h"

namespace fs4 {
namespace {

constexpr int kThreads = 384;         // warp 0 producer, 1 MMA issuer, 2 scale copier, 3 idle, 4-11 epilogue
constexpr int kStages = 6;
constexpr int kCodes = kTileBytes;    // 128 rows x 256 elements
constexpr int kSf = 2 * kAtomBytes;   // their scales
constexpr int kStage = 2 * kCodes + 3 * kSf;
constexpr uint32_t kAccCols = 256, kSfCols = 24;
constexpr uint32_t kCols = 512;
static_assert(kAccCols + kStages * kSfCols <= kCols, "accumulator and scales over the TMEM columns");
static_assert(kStage % 1024 == 0, "stages must keep 1024-byte alignment");
constexpr int kGroup = 8;             // tile rows of a raster group: pairs at work share operands in L2

struct Shared {
  uint64_t full[kStages];     // leader: both CTAs' operands landed
  uint64_t scales[kStages];   // leader: the stage's scales are in TMEM
  uint64_t empty[kStages];    // the MMAs reading the stage finished (both CTAs)
  uint64_t acc_full;
  uint64_t acc_empty;         // leader: both CTAs drained the accumulator
  uint64_t done[2];
  uint32_t tmem;
  int32_t abort;
  uint32_t issued[2];         // leader: stages that each CTA's producer issued
};
constexpr int kSmem = 1024 + kStages * kStage + (int)sizeof(Shared);
static_assert(kSmem <= 232448, "over the per-CTA shared-memory limit");

struct PairArgs {
  CUtensorMap a_codes, a_scales, b_codes, b_scales;
  int32_t M, N;
  int32_t kt;                 // 256-element K tiles
  int32_t tiles_m, tiles_n;
  void* d;
  int64_t ldd;
  int32_t accumulate;
  int32_t after_quantize;
  uint32_t* status;
  int32_t stall;              // see MxGemmArgs
};

__device__ __forceinline__ void tile_of(const PairArgs& a, int32_t u, int32_t& I, int32_t& J) {
  const int32_t g = u / (kGroup * a.tiles_n), h = min(kGroup, a.tiles_m - kGroup * g);
  u -= g * kGroup * a.tiles_n;
  J = u / h;
  I = kGroup * g + u % h;
}

// 32 columns of one row of D; a warp's rows follow one another.
template <typename T>
__device__ __forceinline__ void store_row(const PairArgs& a, int32_t row, int32_t col, int lane, uint32_t* acc) {
  if (col >= a.N) return;
  constexpr int kPer = 32 / (int)sizeof(T);
  T* d = static_cast<T*>(a.d);
  if (col + 32 <= a.N && ((reinterpret_cast<uintptr_t>(d) | (uintptr_t)(a.ldd * (int64_t)sizeof(T))) & 31) == 0) {
    if (row >= a.M) return;
    T* at = d + row * a.ldd + col;
#pragma unroll
    for (int q = 0; q < 32 / kPer; q += 2) {
      Pair r[2]{};
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (a.accumulate) r[b] = load_pair(at + (q + b) * kPer);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        T* e = reinterpret_cast<T*>(r[b].w);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
        const float v = __uint_as_float(acc[(q + b) * kPer + i]);
        put_as(e + i, a.accumulate ? v + to_f32(e[i]) : v);
        }
        store_pair(at + (q + b) * kPer, r[b]);
      }
    }
    return;
  }
  // rows that do not start on 32 bytes: the warp's values change places, then a row at a time (4096 x
  // 4094 x 2048 to BF16: 153 us with a lane a row)
  turn32(acc, lane);
  const int32_t r0 = row - lane;
  if (col + lane >= a.N) return;
  T* at = d + (int64_t)r0 * a.ldd + col + lane;
#pragma unroll
  for (int h = 0; h < 32; h += 8) {
    float old[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) old[i] = (a.accumulate && r0 + h + i < a.M) ? to_f32(at[(h + i) * a.ldd]) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + h + i < a.M) put_as(at + (h + i) * a.ldd, __uint_as_float(acc[h + i]) + old[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) mxfp4_pair_kernel(const __grid_constant__ PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared& sh = *reinterpret_cast<Shared*>(smem + kStages * kStage);
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t first = blockIdx.x >> 1, step = gridDim.x >> 1, total = a.tiles_m * a.tiles_n;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.scales[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    mbar_init(&sh.acc_full, 1);
    mbar_init(&sh.acc_empty, 16);
    mbar_init(&sh.done[0], 1);
    mbar_init(&sh.done[1], 1);
    sh.abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&a.a_codes);
    tma_prefetch_map(&a.b_codes);
    tma_prefetch_map(&a.a_scales);
    tma_prefetch_map(&a.b_scales);
  }
  if (warp == 1) tmem_alloc_pair(&sh.tmem, kCols);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = sh.tmem, base = smem_addr(smem);

  if (warp == 0 && lane == 0) {
    uint32_t s = 0, ph = 0, issued = 0;
    bool ok = true;
    wait_for_quantize(a.after_quantize);
    for (int32_t u = first; u < total && ok; u += step) {
      int32_t I, J;
      tile_of(a, u, I, J);
      // rows of 128 bytes: a codes tile is 128 of them, the scales of a tile 8
      int32_t ra = (2 * I + (int32_t)rank) * a.kt, rb = (2 * J + (int32_t)rank) * a.kt, rb0 = 2 * J * a.kt;
      for (int32_t k = 0; k < a.kt; ++k, ++ra, ++rb, ++rb0) {
        if (!mbar_wait(&sh.empty[s], ph ^ 1u, a.status, abort)) { ok = false; break; }
        const uint32_t st = base + s * kStage, sf = st + 2 * kCodes;
        const uint32_t bar = cluster_map(smem_addr(&sh.full[s]), 0);
        if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * kStage);
        tma_rows_pair(sf, &a.a_scales, 8 * ra, bar);
        tma_rows_pair(sf + kSf, &a.b_scales, 8 * rb0, bar);
        tma_rows_pair(sf + 2 * kSf, &a.b_scales, 8 * (rb0 + a.kt), bar);
        tma_rows_pair(st, &a.a_codes, 128 * ra, bar);
        tma_rows_pair(st + kCodes, &a.b_codes, 128 * rb, bar);
        ++issued;
        if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
      }
    }
    // every copy lands before the pair may exit (they count on the leader's barriers)
    if (rank == 0) await_own(sh.full, kStages, issued, a.status);
    tell_issued(&sh.issued[rank], issued);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    uint32_t s = 0, ph = 0, tl = 0;
    bool ok = !a.stall || mbar_wait(&sh.done[0], 0, a.status, abort);     // (test only: a wait that runs out)
    const uint64_t da0 = sdesc_sw128(base), db0 = sdesc_sw128(base + kCodes);
    constexpr uint64_t kStep = kStage >> 4;
    for (int32_t u = first; u < total && ok; u += step, ++tl) {
      if (!mbar_wait_cluster(&sh.acc_empty, (tl & 1u) ^ 1u, a.status, abort)) break;
      tc_fence_after();
      for (int32_t k = 0; k < a.kt; ++k) {
        if (!mbar_wait(&sh.scales[s], ph, a.status, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sf = tmem + kAccCols + kSfCols * s;
        const uint64_t da = da0 + s * kStep, db = db0 + s * kStep;
#pragma unroll
        for (int h = 0; h < 4; ++h)
          tc_mma_mxf4_pair(tmem, da + 2 * h, db + 2 * h, idesc_mxf4(256, 256, h & 1), sf + 4 * (h >> 1), sf + 8 + 8 * (h >> 1),
                           (k | h) != 0 ? 1u : 0u);
        tc_commit_pair(&sh.empty[s]);
        if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
      }
      if (!ok) break;
      tc_commit_pair(&sh.acc_full);
    }
    tc_commit_own(&sh.done[0]);
    volatile int never = 0;
    mbar_wait(&sh.done[0], 0, a.status, &never);
  } else if (warp == 2 && lane == 0 && rank == 0) {
    // A stage's TMEM columns are free once its shared memory was refilled: the MMAs that read
    // both had completed.  Column order: A k-halves 0, 1; then for each half B's two bands.
    uint32_t s = 0, ph = 0;
    bool ok = true;
    const uint64_t ds0 = sdesc_sf_atom(base + 2 * kCodes);
    for (int32_t u = first; u < total && ok; u += step) {
      for (int32_t k = 0; k < a.kt; ++k) {
        if (!mbar_wait_cluster(&sh.full[s], ph, a.status, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sf = tmem + kAccCols + kSfCols * s;
        const uint64_t ds = ds0 + (uint64_t)s * (kStage >> 4);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          const uint32_t col = i < 2 ? 4 * i : 8 + 8 * (i & 1) + 4 * ((i - 2) >> 1);
          tc_copy_sf_pair(sf + col, ds + (uint64_t)(i * (kAtomBytes >> 4)));
        }
        tc_commit_own(&sh.scales[s]);
        if (++s == (uint32_t)kStages) { s = 0; ph ^= 1u; }
      }
    }
    tc_commit_own(&sh.done[1]);
    volatile int never = 0;
    mbar_wait(&sh.done[1], 0, a.status, &never);
  } else if (warp >= 4) {
    const int quad = warp & 3, half = (warp - 4) >> 2;
    uint32_t tl = 0;
    for (int32_t u = first; u < total; u += step, ++tl) {
      int32_t I, J;
      tile_of(a, u, I, J);
      const int got = lane == 0 ? (mbar_wait(&sh.acc_full, tl & 1u, a.status, abort) ? 1 : 0) : 0;
      if (__shfl_sync(0xFFFFFFFFu, got, 0) == 0) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t taddr = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * half);
      uint32_t acc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_async(taddr + 32 * c, acc[c]);
      tmem_wait_ld32(acc[0]);
      tmem_ld_order(acc[1]);
      tmem_ld_order(acc[2]);
      tmem_ld_order(acc[3]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(&sh.acc_empty);
        else mbar_arrive_remote(cluster_map(smem_addr(&sh.acc_empty), 0));
      }
      const int32_t row = 256 * I + 128 * (int32_t)rank + 32 * quad + lane, col = 256 * J + 128 * half;
#pragma unroll
      for (int c = 0; c < 4; ++c) store_row<T>(a, row, col + 32 * c, lane, acc[c]);
    }
  }
  __syncwarp();
  // the leader's MMAs and copies read the other CTA's memory: neither leaves before both are done
  tc_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  if (rank == 0 && threadIdx.x == 0) await_issued(sh.full, kStages, kStage, sh.issued[0], sh.issued[1], a.status);
  if (warp == 1) tmem_dealloc_pair(tmem, kCols);
  __syncthreads();
  cluster_arrive();
  cluster_wait();
}

template <typename T>
cudaError_t launch_pair(const PairArgs& a, cudaStream_t st) {
  static PairSlots slots;
  int pairs = 0;
  cudaError_t e = pair_slots(slots, mxfp4_pair_kernel<T>, kThreads, kSmem, &pairs);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = a.after_quantize ? 2 : 1;
  cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, mxfp4_pair_kernel<T>, a);
}

}  // namespace

cudaError_t launch_mxfp4_pair(const MxGemmArgs& g, cudaStream_t st) {
  PairArgs a;
  const int64_t kt = (g.K + 255) / 256, bands_a = (g.M + 127) / 128, bands_b = (g.N + 127) / 128;
  cudaError_t e;
  if ((e = make_row_map(&a.a_codes, g.a_codes, bands_a * kt * kCodes, 128)) != cudaSuccess) return e;
  if ((e = make_row_map(&a.a_scales, g.a_scales, bands_a * kt * kSf, 8)) != cudaSuccess) return e;
  if ((e = make_row_map(&a.b_codes, g.b_codes, bands_b * kt * kCodes, 128)) != cudaSuccess) return e;
  if ((e = make_row_map(&a.b_scales, g.b_scales, bands_b * kt * kSf, 8)) != cudaSuccess) return e;
  a.M = (int32_t)g.M;
  a.N = (int32_t)g.N;
  a.kt = (int32_t)kt;
  a.tiles_m = (int32_t)((g.M + 255) / 256);
  a.tiles_n = (int32_t)((g.N + 255) / 256);
  a.d = g.d;
  a.ldd = g.ldd;
  a.accumulate = g.accumulate;
  a.after_quantize = g.after_quantize;
  a.status = g.status;
  a.stall = g.stall;
  switch (g.dtype) {
    case kTypeF32: return launch_pair<float>(a, st);
    case kTypeBf16: return launch_pair<__nv_bfloat16>(a, st);
    default: return launch_pair<__half>(a, st);
  }
}

}  // namespace fs4
