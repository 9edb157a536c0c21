// MXFP4 products D = deq(A) deq(B)^T (+ D) on the 5th-generation tensor cores (sm_100a):
// tcgen05.mma kind::mxf4, E2M1 operands with one UE8M0 scale per 32 elements of K, FP32
// accumulation in TMEM, operands in the TILED layout of include/fs4.h.
#include <cstdint>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace fs4 {
namespace {

// One 128 x TN tile of D^(T) per CTA, K split over the CTAs of a cluster.  The operand on the
// tensor core's 128-row side is P, the one on its TN-row side Q; with few rows of A (decoding)
// P = B, so that the weights fill the tensor core and the tokens are its narrow side.
struct TileArgs {
  const uint8_t* p_codes;
  const uint8_t* p_scales;
  const uint8_t* q_codes;
  const uint8_t* q_scales;
  int32_t P, Q;        // rows of the operands
  int32_t kt;          // 256-element K tiles
  int32_t splits;      // CTAs along K = cluster size
  int32_t q_tiles;
  void* d;
  int64_t ldp, ldq;    // strides of D along P and Q (elements)
  int32_t dtype;
  int32_t accumulate;
  uint32_t* status;
};

constexpr int kTileThreads = 192;    // warp 0 producer, warp 1 MMA issuer, warps 2-5 epilogue
constexpr int kPartPitch = 129;      // floats between a partial tile's Q rows: conflict-free both ways

template <int TN>
struct TileCfg {
  static constexpr int kP = kTileBytes;                    // P codes of one stage: 128 rows x 128 bytes
  static constexpr int kQ = TN * 128;                      // Q codes
  static constexpr int kSf = 2 * kAtomBytes;               // scales of 128 rows x 256 elements
  static constexpr int kStage = kP + ((kQ + 1023) / 1024) * 1024 + 2 * kSf;
  static constexpr int kStages = TN <= 32 ? 5 : 4;
  static constexpr uint32_t kAcc = TN < 32 ? 32 : TN;      // TMEM columns of the accumulator
  static constexpr int kPart = (int)kAcc * kPartPitch * 4;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSmem = 1024 + (kRing > kPart ? kRing : kPart) + 256;
  static constexpr uint32_t kCols = kAcc + kStages * 16 <= 128 ? 128 : 256;
  static_assert(kAcc + kStages * 16 <= kCols, "scale-factor ring over the TMEM columns");
  static_assert(kStage % 1024 == 0, "stages must keep 1024-byte alignment");
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ void store_rounded(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_rounded(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_rounded(__half* p, float v) { *p = __float2half_rn(v); }

// Sum the cluster's partial tiles (rank order, so the result does not depend on timing) and
// write rows [q_lo, q_hi) of this tile.
template <int TN, typename T>
__device__ __forceinline__ void tile_store(const TileArgs& a, const float* part, int64_t p0, int64_t q0, int q_lo, int q_hi) {
  const uint32_t base = smem_addr(part);
  T* d = static_cast<T*>(a.d);
  const int rows = q_hi - q_lo;
  for (int i = threadIdx.x; i < rows * 128; i += kTileThreads) {
    // neighbouring threads take neighbouring elements of D
    int p, q;
    if (a.ldp == 1) { p = i & 127; q = q_lo + (i >> 7); }
    else { q = q_lo + i % rows; p = i / rows; }
    if (p0 + p >= a.P || q0 + q >= a.Q) continue;
    const uint32_t off = (uint32_t)(q * kPartPitch + p) * 4u;
    float v = 0.0f;
    if (a.splits == 1) {
      v = part[q * kPartPitch + p];
    } else {
      for (int s = 0; s < a.splits; ++s) v += cluster_load(cluster_map(base + off, (uint32_t)s));
    }
    T* dst = d + (p0 + p) * a.ldp + (q0 + q) * a.ldq;
    if (a.accumulate) v += to_float(*dst);
    store_rounded(dst, v);
  }
}

template <int TN>
__global__ void __launch_bounds__(kTileThreads) mxfp4_tile_kernel(const __grid_constant__ TileArgs a) {
  using C = TileCfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (C::kRing > C::kPart ? C::kRing : C::kPart));
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits;
  const int tile = blockIdx.x / a.splits;
  const int64_t p0 = (int64_t)(tile / a.q_tiles) * 128, q0 = (int64_t)(tile % a.q_tiles) * TN;
  const int k0 = (int)((int64_t)a.kt * split / a.splits), k1 = (int)((int64_t)a.kt * (split + 1) / a.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t base = smem_addr(smem);
  // rows of Q present in its 128-row band from q0 on (the TILED layout pads rows to 128)
  constexpr uint32_t kTx = C::kP + C::kQ + 2 * C::kSf;

  if (warp == 0 && lane == 0) {
    const int64_t band = (int64_t)a.kt * kTileBytes, sband = (int64_t)a.kt * C::kSf;
    const uint8_t* pc = a.p_codes + (p0 >> 7) * band + (int64_t)k0 * kTileBytes;
    const uint8_t* ps = a.p_scales + (p0 >> 7) * sband + (int64_t)k0 * C::kSf;
    const uint8_t* qc = a.q_codes + (q0 >> 7) * band + (int64_t)k0 * kTileBytes + (q0 & 127) * 128;
    const uint8_t* qs = a.q_scales + (q0 >> 7) * sband + (int64_t)k0 * C::kSf;
    uint32_t s = 0, ph = 0;
    int k = k0;
    for (; k < k1; ++k) {
      if (!mbar_wait(&empty[s], ph ^ 1u, a.status, abort_flag)) break;
      const uint32_t st = base + s * C::kStage;
      mbar_arrive_expect_tx(&full[s], kTx);
      bulk_g2s_addr(st + C::kStage - 2 * C::kSf, ps, C::kSf, &full[s]);
      bulk_g2s_addr(st + C::kStage - C::kSf, qs, C::kSf, &full[s]);
      bulk_g2s_addr(st, pc, C::kP, &full[s]);
      bulk_g2s_addr(st + C::kP, qc, C::kQ, &full[s]);
      pc += kTileBytes; qc += kTileBytes;
      ps += C::kSf; qs += C::kSf;
      if (++s == (uint32_t)C::kStages) { s = 0; ph ^= 1u; }
    }
    // every issued copy lands before the shared memory is reused or given up
    const int issued = k - k0;
    for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i) {
      volatile int never = 0;
      mbar_wait(&full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u, a.status, &never);
    }
  } else if (warp == 1 && lane == 0) {
    uint32_t s = 0, ph = 0;
    const uint64_t dp0 = sdesc_sw128(base), dq0 = sdesc_sw128(base + C::kP);
    const uint64_t ds0 = sdesc_sf_atom(base + C::kStage - 2 * C::kSf);
    constexpr uint64_t kStep = C::kStage >> 4;
    // Q rows from q0 on start at this 32-row group of their scale atom
    const uint32_t qcol = TN < 32 ? 0u : (uint32_t)((q0 & 127) >> 5);   // (a 16-row tile is the only one)
    for (int k = k0; k < k1; ++k) {
      if (!mbar_wait(&full[s], ph, a.status, abort_flag)) break;
      tc_fence_after();
      // each stage has scale columns of its own: P's two atoms, then Q's two
      const uint32_t sf = tmem + C::kAcc + 16 * s;
      const uint64_t ds = ds0 + s * kStep;
#pragma unroll
      for (int i = 0; i < 4; ++i) tc_copy_sf(sf + 4 * i, ds + (uint64_t)(i * (kAtomBytes >> 4)));
#pragma unroll
      for (int h = 0; h < 4; ++h)
        tc_mma_mxf4(tmem, dp0 + s * kStep + 2 * h, dq0 + s * kStep + 2 * h, idesc_mxf4(128, TN, h & 1), sf + 4 * (h >> 1),
                    sf + 8 + 4 * (h >> 1) + qcol, (k > k0 || h > 0) ? 1u : 0u);
      tc_commit(&empty[s]);
      if (++s == (uint32_t)C::kStages) { s = 0; ph ^= 1u; }
    }
    tc_commit(done);
    volatile int never = 0;
    mbar_wait(done, 0, a.status, &never);
  }
  __syncwarp();
  // The MMAs have completed (warp 1 waited) and every copy has landed (warp 0 waited): the
  // stages' memory becomes the partial tile.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int quad = warp & 3;
    const int p = 32 * quad + lane;
#pragma unroll
    for (int c = 0; c < (int)C::kAcc; c += 32) {
      float v[32];
      tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) part[(c + i) * kPartPitch + p] = v[i];
    }
    tc_fence_before();
  }
  if (a.splits > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  const int q_lo = TN * split / a.splits, q_hi = TN * (split + 1) / a.splits;
  if (a.dtype == kTypeF32) tile_store<TN, float>(a, part, p0, q0, q_lo, q_hi);
  else if (a.dtype == kTypeBf16) tile_store<TN, __nv_bfloat16>(a, part, p0, q0, q_lo, q_hi);
  else tile_store<TN, __half>(a, part, p0, q0, q_lo, q_hi);
  if (a.splits > 1) {      // no CTA leaves while another reads its partial tile
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kCols);
}

template <int TN>
cudaError_t launch_tile(const TileArgs& a, int64_t tiles, cudaStream_t st) {
  using C = TileCfg<TN>;
  cudaError_t e = cudaFuncSetAttribute(mxfp4_tile_kernel<TN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * a.splits));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mxfp4_tile_kernel<TN>, a);
}

}  // namespace

cudaError_t launch_mxfp4_gemm(const MxGemmArgs& g, cudaStream_t st, int num_sms) {
  if (((g.M + 255) / 256) * ((g.N + 255) / 256) >= 40) return launch_mxfp4_pair(g, st);
  TileArgs a{};
  // the narrow side: A's rows when they are at most 64 and no more than B's
  const bool swap = g.M <= 64 && g.M <= g.N;
  a.p_codes = swap ? g.b_codes : g.a_codes; a.p_scales = swap ? g.b_scales : g.a_scales;
  a.q_codes = swap ? g.a_codes : g.b_codes; a.q_scales = swap ? g.a_scales : g.b_scales;
  a.P = (int32_t)(swap ? g.N : g.M);
  a.Q = (int32_t)(swap ? g.M : g.N);
  a.ldp = swap ? 1 : g.ldd;
  a.ldq = swap ? g.ldd : 1;
  a.kt = (int32_t)((g.K + 255) / 256);
  a.d = g.d; a.dtype = g.dtype; a.accumulate = g.accumulate; a.status = g.status;
  const int tn = a.Q <= 16 ? 16 : a.Q <= 32 ? 32 : a.Q <= 64 ? 64 : 128;
  a.q_tiles = (a.Q + tn - 1) / tn;
  const int64_t tiles = (int64_t)((a.P + 127) / 128) * a.q_tiles;
  a.splits = 1;
  while (a.splits < 8 && 2 * a.splits <= a.kt && tiles * a.splits * 2 <= num_sms) a.splits *= 2;
  switch (tn) {
    case 16: return launch_tile<16>(a, tiles, st);
    case 32: return launch_tile<32>(a, tiles, st);
    case 64: return launch_tile<64>(a, tiles, st);
    default: return launch_tile<128>(a, tiles, st);
  }
}

}  // namespace fs4
