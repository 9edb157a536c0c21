// MXFP4 products D = deq(A) deq(B)^T (+ D) on the 5th-generation tensor cores (sm_100a):
// tcgen05.mma kind::mxf4, E2M1 operands with one UE8M0 scale per 32 elements of K, FP32
// accumulation in TMEM, operands in the TILED layout of include/fs4.h.
#include <cstdint>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace fs4 {
namespace {

// Few rows or small products are bound by latency and by the weights' bytes: 1 x 28672 x 8192 reads
// them at 5.1 TB/s (24.8 us), 1 x 8192 x 8192 takes 11.5 us of which about 5.6 do not depend on the
// size, 250 x 512 x 640 takes 8 us.  Splitting K over a cluster fills the device where tiles are few;
// its CTAs add their partial tiles up through shared memory, in rank order.
//
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
  int64_t ldd;
  int32_t swapped;     // P is D's columns (else its rows)
  int32_t dtype;
  int32_t accumulate;
  uint32_t* status;
  int32_t after_quantize;   // starts while the quantisation of A still runs
  // fused quantisation of Q: its rows as the caller has them
  const void* x;
  int64_t ldx;
  int32_t x_dtype, K;
  int32_t ceil_rule;
  int32_t stall;       // see MxGemmArgs
  int32_t vec;         // x's rows start on 16-byte boundaries
};

constexpr int kTileThreads = 192;    // warp 0 producer, warp 1 MMA issuer, warps 2-5 epilogue

template <int TN, bool kFused>
struct TileCfg {
  static constexpr int kP = kTileBytes;                    // P codes of one stage: 128 rows x 128 bytes
  static constexpr int kQ = TN * 128;                      // Q codes of 256 elements
  static constexpr int kSf = 2 * kAtomBytes;               // scales of 128 rows x 256 elements
  static constexpr int kQAll = kQ + kSf;                   // fused: Q of one K tile, kept for the whole call
  static constexpr int kStage = kFused ? kP + kSf : kP + kQ + 2 * kSf;
  static constexpr int kStages = TN <= 32 ? 5 : 4;
  static constexpr uint32_t kAcc = TN < 32 ? 32 : TN;      // TMEM columns of the accumulator
  // a partial tile has D's orientation, rows 4 floats apart in banks: 128 columns or kAcc
  static constexpr int kWide = 128 + 4, kNarrow = (int)kAcc + 4;
  static constexpr int kPart = 4 * ((int)kAcc * kWide > 128 * kNarrow ? (int)kAcc * kWide : 128 * kNarrow);
  static constexpr int kRing = kStages * kStage;
  static constexpr int kMain = ((kRing > kPart ? kRing : kPart) + 1023) / 1024 * 1024;
  static constexpr int kSmem = 1024 + kMain + 256;
  static constexpr uint32_t kCols = kAcc + kStages * 16 <= 128 ? 128 : 256;
  static_assert(kAcc + kStages * 16 <= kCols, "scale-factor ring over the TMEM columns");
  static_assert(kStage % 1024 == 0 && kQAll % 1024 == 0, "stages must keep 1024-byte alignment");
};

// Eight elements of x from (r, c) on; absent ones are 0.
__device__ __forceinline__ void load_x8(const TileArgs& a, int64_t r, int64_t c, float* v) {
  const int64_t at = r * a.ldx + c;
  if (a.vec && c + 8 <= a.K) {
    if (a.x_dtype == kTypeF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + at);
      const float4 s = __ldg(p), t = __ldg(p + 1);
      v[0] = s.x; v[1] = s.y; v[2] = s.z; v[3] = s.w; v[4] = t.x; v[5] = t.y; v[6] = t.z; v[7] = t.w;
      return;
    }
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = a.x_dtype == kTypeBf16 ? __uint_as_float(u[i] << 16) : half_lo(u[i]);
      v[2 * i + 1] = a.x_dtype == kTypeBf16 ? __uint_as_float(u[i] & 0xFFFF0000u) : half_hi(u[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.0f;
    if (c + i >= a.K) continue;
    if (a.x_dtype == kTypeF32) v[i] = static_cast<const float*>(a.x)[at + i];
    else if (a.x_dtype == kTypeBf16) v[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.x)[at + i]);
    else v[i] = __half2float(static_cast<const __half*>(a.x)[at + i]);
  }
}

// Quantise Q's rows (nearest, as mxfp4_quantize_kernel does) for K tiles k0 .. k1 - 1 into their
// shared-memory image: one warp 256 elements of a row, four lanes a block.  The rest of the
// TN rows is zero.  128 threads, thread index t.
template <int TN>
__device__ __forceinline__ void quantize_q(const TileArgs& a, uint8_t* q, int k0, int k1, int t) {
  using C = TileCfg<TN, true>;
  const int lane = t & 31, warp = t >> 5;
  for (int i = t; i < (k1 - k0) * (C::kQAll / 16); i += 128) reinterpret_cast<uint4*>(q)[i] = make_uint4(0u, 0u, 0u, 0u);
  named_bar(1, 128);
  // kBatch tasks of a warp at once, their loads issued first
  constexpr int kBatch = 4;
  const int tasks = a.Q * (k1 - k0);
  for (int t0 = warp; t0 < tasks; t0 += 4 * kBatch) {
    float v[kBatch][8];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int task = t0 + 4 * i;
      if (task < tasks) load_x8(a, task % a.Q, 256ll * (k0 + task / a.Q) + 8 * lane, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int task = t0 + 4 * i, r = task % a.Q;
      if (task >= tasks) break;
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[i][e]) & 0x7FFFFFFFu);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t byte = mx_scale_byte(m, a.ceil_rule != 0);
      uint32_t w = 0u;
      if (byte != 255u) {
        const float s = mx_inverse_scale(byte);
        w = pack8_e2m1(v[i][0] * s, v[i][1] * s, v[i][2] * s, v[i][3] * s, v[i][4] * s, v[i][5] * s, v[i][6] * s, v[i][7] * s);
      }
      uint8_t* tile = q + task / a.Q * C::kQAll;
      const int b = lane >> 2;              // 32-element block of the 256
      *reinterpret_cast<uint32_t*>(tile + 128 * r + 16 * (b ^ (r & 7)) + 4 * (lane & 3)) = w;
      if ((lane & 3) == 0) tile[C::kQ + kAtomBytes * (b >> 2) + 16 * r + (b & 3)] = (uint8_t)byte;
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");     // the tensor core reads what was stored
}

// Sum the cluster's partial tiles (rank order, so the result does not depend on timing) and
// write rows [lo, hi) of the tile's kC columns at D[r0.., c0..]: four columns a thread and load.
template <int kC, typename T>
__device__ __forceinline__ void tile_store(const TileArgs& a, const float* part, int64_t r0, int64_t c0, int rows, int cols, int lo,
                                           int hi) {
  constexpr int kPitch = kC + 4;
  T* d = static_cast<T*>(a.d);
  const uint32_t base = smem_addr(part);
  const int total = (hi - lo) * (kC / 4);
  for (int i = threadIdx.x; i < total; i += kTileThreads) {
    const int r = lo + i / (kC / 4), c = 4 * (i % (kC / 4));
    const uint32_t off = (uint32_t)(r * kPitch + c) * 4u;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.splits == 1) {
      v = *reinterpret_cast<const float4*>(reinterpret_cast<const uint8_t*>(part) + off);
    } else {
      float4 x[8];           // all CTAs' loads at once: one takes about 600 ns
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < a.splits) x[s] = cluster_load4(cluster_map(base, (uint32_t)s) + off);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s < a.splits) { v.x += x[s].x; v.y += x[s].y; v.z += x[s].z; v.w += x[s].w; }
    }
    if (r >= rows) continue;
    T* at = d + (r0 + r) * a.ldd + c0 + c;
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (c + 4 <= cols && (reinterpret_cast<uintptr_t>(at) & (4 * sizeof(T) - 1)) == 0) {
      struct alignas(4 * sizeof(T)) Four { T t[4]; } o;
      if (a.accumulate) o = *reinterpret_cast<const Four*>(at);
#pragma unroll
      for (int k = 0; k < 4; ++k) put_as(&o.t[k], a.accumulate ? e[k] + to_f32(o.t[k]) : e[k]);
      *reinterpret_cast<Four*>(at) = o;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < cols) put_as(at + k, a.accumulate ? e[k] + to_f32(at[k]) : e[k]);
    }
  }
}

template <int TN, typename T>
__device__ __forceinline__ void tile_finish(const TileArgs& a, const float* part, int64_t p0, int64_t q0, int split) {
  constexpr int kAcc = TN < 32 ? 32 : TN;
  const int p_n = (int)(a.P - p0 < 128 ? a.P - p0 : 128), q_n = (int)(a.Q - q0 < TN ? a.Q - q0 : TN);
  if (a.swapped) tile_store<128, T>(a, part, q0, p0, q_n, p_n, TN * split / a.splits, TN * (split + 1) / a.splits);
  else tile_store<kAcc, T>(a, part, p0, q0, p_n, q_n, 128 * split / a.splits, 128 * (split + 1) / a.splits);
}

template <int TN, bool kFused>
__global__ void __launch_bounds__(kTileThreads) mxfp4_tile_kernel(const __grid_constant__ TileArgs a) {
  using C = TileCfg<TN, kFused>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_all = smem + C::kMain;      // fused: Q's K tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(q_all + (kFused ? (a.kt + a.splits - 1) / a.splits * C::kQAll : 0));
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint64_t* ready = done + 1;            // fused: Q is quantised
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ready + 1);
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
    mbar_init(ready, 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t base = smem_addr(smem);
  constexpr uint32_t kTx = kFused ? C::kP + C::kSf : C::kP + C::kQ + 2 * C::kSf;

  if (warp == 0 && lane == 0) {
    const int64_t band = (int64_t)a.kt * kTileBytes, sband = (int64_t)a.kt * C::kSf;
    const uint8_t* pc = a.p_codes + (p0 >> 7) * band + (int64_t)k0 * kTileBytes;
    const uint8_t* ps = a.p_scales + (p0 >> 7) * sband + (int64_t)k0 * C::kSf;
    const uint8_t* qc = a.q_codes + (q0 >> 7) * band + (int64_t)k0 * kTileBytes;
    const uint8_t* qs = a.q_scales + (q0 >> 7) * sband + (int64_t)k0 * C::kSf;
    uint32_t s = 0, ph = 0;
    int k = k0;
    // A may still be being quantised: the ring's first stages get the other operand before the wait
    auto load_p = [&](uint32_t st, uint32_t s) {
      bulk_g2s_addr(st + C::kP, ps, C::kSf, &full[s]);
      bulk_g2s_addr(st, pc, C::kP, &full[s]);
      pc += kTileBytes;
      ps += C::kSf;
    };
    auto load_q = [&](uint32_t st, uint32_t s) {
      bulk_g2s_addr(st + C::kP + C::kSf, qs, C::kSf, &full[s]);
      bulk_g2s_addr(st + C::kP + 2 * C::kSf, qc, C::kQ, &full[s]);
      qc += kTileBytes;
      qs += C::kSf;
    };
    const bool split = !kFused && a.after_quantize;
    const int head = split ? (k1 - k0 < C::kStages ? k1 - k0 : C::kStages) : 0;
    if constexpr (!kFused) {
      for (int i = 0; i < head; ++i) {
        mbar_arrive_expect_tx(&full[i], kTx);
        if (a.swapped) load_p(base + i * C::kStage, i);
        else load_q(base + i * C::kStage, i);
      }
      wait_for_quantize(a.after_quantize);
    }
    for (; k < k1; ++k) {
      const bool begun = k - k0 < head;
      if (!begun) {
        if (!mbar_wait(&empty[s], ph ^ 1u, a.status, abort_flag)) break;
        mbar_arrive_expect_tx(&full[s], kTx);
      }
      const uint32_t st = base + s * C::kStage;
      if (!begun || !a.swapped) load_p(st, s);
      if constexpr (!kFused) {
        if (!begun || a.swapped) load_q(st, s);
      }
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
    constexpr uint64_t kStep = C::kStage >> 4;
    const uint64_t dp0 = sdesc_sw128(base), dps0 = sdesc_sf_atom(base + C::kP);
    uint64_t dq = sdesc_sw128(kFused ? smem_addr(q_all) : base + C::kP + 2 * C::kSf);
    uint64_t dqs = sdesc_sf_atom(kFused ? smem_addr(q_all) + C::kQ : base + C::kP + C::kSf);
    const uint64_t dq0 = dq, dqs0 = dqs;
    // test only: a wait that runs out
    bool ok = !a.stall || mbar_wait(done, 0, a.status, abort_flag);
    if (kFused && ok) ok = mbar_wait(ready, 0, a.status, abort_flag);
    for (int k = k0; ok && k < k1; ++k) {
      if (!mbar_wait(&full[s], ph, a.status, abort_flag)) break;
      tc_fence_after();
      // each stage has scale columns of its own: P's two atoms, then Q's two
      const uint32_t sf = tmem + C::kAcc + 16 * s;
      const uint64_t dp = dp0 + s * kStep, dps = dps0 + s * kStep;
      if constexpr (!kFused) {
        dq = dq0 + s * kStep;
        dqs = dqs0 + s * kStep;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tc_copy_sf(sf + 4 * i, dps + (uint64_t)(i * (kAtomBytes >> 4)));
        tc_copy_sf(sf + 8 + 4 * i, dqs + (uint64_t)(i * (kAtomBytes >> 4)));
      }
#pragma unroll
      for (int h = 0; h < 4; ++h)
        tc_mma_mxf4(tmem, dp + 2 * h, dq + 2 * h, idesc_mxf4(128, TN, h & 1), sf + 4 * (h >> 1),
                    sf + 8 + 4 * (h >> 1), (k > k0 || h > 0) ? 1u : 0u);
      tc_commit(&empty[s]);
      if constexpr (kFused) {
        dq += C::kQAll >> 4;
        dqs += C::kQAll >> 4;
      }
      if (++s == (uint32_t)C::kStages) { s = 0; ph ^= 1u; }
    }
    tc_commit(done);
    volatile int never = 0;
    mbar_wait(done, 0, a.status, &never);
  } else if (warp >= 2) {
    if constexpr (kFused) {
      quantize_q<TN>(a, q_all, k0, k1, threadIdx.x - 64);
      mbar_arrive(ready);
    }
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
      if (a.swapped) {
#pragma unroll
        for (int i = 0; i < 32; ++i) part[(c + i) * C::kWide + p] = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(part + p * C::kNarrow + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    tc_fence_before();
  }
  if (a.splits > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (a.dtype == kTypeF32) tile_finish<TN, float>(a, part, p0, q0, split);
  else if (a.dtype == kTypeBf16) tile_finish<TN, __nv_bfloat16>(a, part, p0, q0, split);
  else tile_finish<TN, __half>(a, part, p0, q0, split);
  if (a.splits > 1) {      // no CTA leaves while another reads its partial tile
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kCols);
}

template <int TN, bool kFused>
cudaError_t launch_tile(const TileArgs& a, int64_t tiles, cudaStream_t st) {
  using C = TileCfg<TN, kFused>;
  const int per = (a.kt + a.splits - 1) / a.splits;
  const int smem = C::kSmem + (kFused ? per * C::kQAll : 0);
  static unsigned long long set = 0ull;      // devices whose limit is raised; a benign race
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(set >> dev & 1)) {
    e = cudaFuncSetAttribute(mxfp4_tile_kernel<TN, kFused>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem + (kFused ? 16 * C::kQAll : 0));
    if (e != cudaSuccess) return e;
    if (dev < 64) set |= 1ull << dev;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * a.splits));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.after_quantize ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, mxfp4_tile_kernel<TN, kFused>, a);
}

// CTAs along K (the cluster size), for a device that holds `slots` CTAs at once: the fewest that
// give the least time in waves of kt / splits steps.
int splits_of(int64_t tiles, int kt, int64_t slots) {
  int best = 1;
  int64_t cost = INT64_MAX;
  for (int s = 1; s <= 8 && s <= kt; ++s) {
    // a wave's fixed part (set-up, first loads, reduction) weighs about four steps
    const int64_t c = (tiles * s + slots - 1) / slots * ((kt + s - 1) / s + 4);
    if (c < cost) { cost = c; best = s; }
  }
  return best;
}

}  // namespace

cudaError_t launch_mxfp4_gemm(const MxGemmArgs& g, cudaStream_t st, int num_sms) {
  // CTA pairs from the point on where 256 x 256 tiles keep enough of them busy; with a long K and few
  // tiles, splitting K does more.  Both sides (us, tile kernel and pairs): 256 x 8192 x 8192 (32 tiles)
  // 21.0 and 17.8, 768 x 2048 x 2048 (24) 10.7 and 9.8, 1024 x 1024 x 512 (16) 9.2 and 7.8, 1024 x 1024
  // x 16384 (16) 22.7 and 27.1, 128 x 8192 x 8192 (32, half empty) 15.2 and 17.4.
  const int64_t tiles256 = ((g.M + 255) / 256) * ((g.N + 255) / 256);
  if (g.M > 128 && g.N > 128 && tiles256 >= (g.K <= 2048 ? 16 : 24)) return launch_mxfp4_pair(g, st);
  TileArgs a{};
  // the narrow side: A's rows when they are at most 64 and no more than B's
  const bool swap = g.M <= 64 && g.M <= g.N;
  a.p_codes = swap ? g.b_codes : g.a_codes; a.p_scales = swap ? g.b_scales : g.a_scales;
  a.q_codes = swap ? g.a_codes : g.b_codes; a.q_scales = swap ? g.a_scales : g.b_scales;
  a.P = (int32_t)(swap ? g.N : g.M);
  a.Q = (int32_t)(swap ? g.M : g.N);
  a.swapped = swap;
  a.ldd = g.ldd;
  a.kt = (int32_t)((g.K + 255) / 256);
  a.d = g.d; a.dtype = g.dtype; a.accumulate = g.accumulate; a.status = g.status;
  a.after_quantize = g.after_quantize;
  a.stall = g.stall;
  // (tiles of fewer than 128 rows of Q are alone, so every tile starts a 128-row band)
  const int tn = a.Q <= 16 ? 16 : a.Q <= 32 ? 32 : a.Q <= 64 ? 64 : 128;
  a.q_tiles = (a.Q + tn - 1) / tn;
  const int64_t tiles = (int64_t)((a.P + 127) / 128) * a.q_tiles;
  // two CTAs of the narrow tiles fit an SM
  a.splits = splits_of(tiles, a.kt, tn <= 32 ? 2 * num_sms : num_sms);
  switch (tn) {
    case 16: return launch_tile<16, false>(a, tiles, st);
    case 32: return launch_tile<32, false>(a, tiles, st);
    case 64: return launch_tile<64, false>(a, tiles, st);
    default: return launch_tile<128, false>(a, tiles, st);
  }
}

bool mxfp4_linear_fused(const MxLinearArgs& g, cudaStream_t st, int num_sms, cudaError_t* error) {
  if (g.M > 16) return false;
  TileArgs a{};
  a.p_codes = g.w_codes; a.p_scales = g.w_scales;
  a.P = (int32_t)g.N;
  a.Q = (int32_t)g.M;
  a.swapped = 1;
  a.ldd = g.ldd;
  a.kt = (int32_t)((g.K + 255) / 256);
  a.d = g.d; a.dtype = g.d_dtype; a.accumulate = g.accumulate; a.status = g.status;
  a.x = g.x; a.ldx = g.ldx; a.x_dtype = g.x_dtype; a.K = (int32_t)g.K; a.ceil_rule = g.ceil_rule;
  a.stall = g.stall;
  a.vec = reinterpret_cast<uintptr_t>(g.x) % 16 == 0 && (g.M == 1 || g.ldx * type_bytes(g.x_dtype) % 16 == 0);
  a.q_tiles = 1;
  const int64_t tiles = (g.N + 127) / 128;
  a.splits = splits_of(tiles, a.kt, 2 * num_sms);
  const int per = (a.kt + a.splits - 1) / a.splits;
  // One batch of loads a warp (16 row pieces of 256 elements a CTA) takes less than the launch
  // that it saves, two take more: 8192 x 8192 with 1 row 12.3 us against 15.7, with 8 rows 19.5
  // against 16.4.
  if (g.M * per > 16) return false;
  *error = launch_tile<16, true>(a, tiles, st);
  return true;
}

}  // namespace fs4
