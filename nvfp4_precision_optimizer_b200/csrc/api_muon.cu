// C entry points of the Muon step (declared in include/fs4.h): argument checks, workspace plan
// and the launch sequence.
#include <cfloat>
#include <cmath>
#include <cstring>

#include "fs4_device.cuh"
#include "muon_internal.h"

using namespace fs4;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool known_type(int32_t t) { return t == FS4_F32 || t == FS4_BF16 || t == FS4_F16; }
inline int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

bool shape_ok(int64_t m, int64_t n) { return m >= 1 && n >= 1 && m <= FS4_MAX_DIM && n <= FS4_MAX_DIM; }

int64_t parts_of(int64_t m, int64_t n) {
  const int64_t unit = m * n / kMuonParts > kMuonUnit ? m * n / kMuonParts : kMuonUnit;
  const int64_t rows = (unit + n - 1) / n;      // rows of one partial sum
  return (m + rows - 1) / rows;
}

// The FP16 operands hold X up to 16 and B = b A + c A^2 up to 255.  X_0 has norm 1, so A's
// eigenvalues s lie in [0, 1] at first, and near it wherever an iteration converges: the bound on B
// is that of b s + c s^2 there, its largest value at 1 or at the vertex.  The steep first triples of
// published schedules, as (8.2, -22.5, 15.9), are of that kind, although b alone is large.
bool coeffs_ok(const float* t) {
  const double a = t[0], b = t[1], c = t[2];
  if (!(std::fabs(a) <= 16.0) || !std::isfinite(b) || !std::isfinite(c)) return false;
  double most = std::fabs(b + c);
  const double s = c != 0.0 ? -b / (2.0 * c) : 0.0;
  if (s > 0.0 && s < 1.0) most = std::fmax(most, std::fabs(s * (b + c * s)));
  return most <= 255.0;
}

struct Plan {
  int64_t bytes = 0;           // of the workspace
  bool small = false;          // see MuonCall
  int32_t split_steps = 1;
  int64_t parts_at = 0, counts_at = 0, counts = 0;
};

// The plan depends on the sizes only.  Small calls are those whose products fit kMuonSmallUnits
// tiles of the small kind and whose updates take at most kMuonSmallSteps K steps in all.  Both sides
// (us for K = 5, small tiles and pairs): 256 x 8192 183 and 320, 1024 x 1024 160 and 196, 512 x 4096
// (2048 steps) 221 and 244, 768 x 3000 (3384) 243 and 249, 1024 x 2048 (4096) 239 and 225, 1536 x
// 1536 (6912) 305 and 240.
Plan plan(int32_t count, const int64_t* rows, const int64_t* cols, MuonTable* t) {
  Plan pl;
  int64_t parts = 0, updates = 0, grams = 0, steps = 0;
  auto sides = [&](int32_t i, int32_t& m, int32_t& n) {
    m = (int32_t)(rows[i] < cols[i] ? rows[i] : cols[i]);
    n = (int32_t)(rows[i] < cols[i] ? cols[i] : rows[i]);
  };
  int32_t m, n;
  for (int32_t i = 0; i < count; ++i) {
    if (t) {
      t->mat[i].partial = parts;
      t->mat[i].parts = (int32_t)parts_of(rows[i], cols[i]);
    }
    parts += parts_of(rows[i], cols[i]);
    sides(i, m, n);
    if (m <= kMuonThin) continue;
    updates += (int64_t)muon_row_tiles(m) * muon_steps(n);
    steps += (int64_t)muon_row_tiles(m) * muon_steps(n) * muon_steps(m);
    grams += muon_gram_tiles(m);
  }
  pl.small = updates > 0 && updates <= kMuonSmallUnits && grams <= kMuonSmallUnits && steps <= kMuonSmallSteps;
  int64_t off = up(kMuonPartials + 8 * parts, 1024);
  if (pl.small) {
    // the shortest parts, of 8 steps at least, that keep the Gram products' units in bounds
    for (pl.split_steps = 8;; pl.split_steps += 4) {
      grams = 0;
      for (int32_t i = 0; i < count; ++i) {
        sides(i, m, n);
        if (m > kMuonThin) grams += muon_gram_tiles(m) * muon_splits(muon_steps(n), pl.split_steps);
      }
      if (grams <= kMuonSmallUnits) break;
    }
    pl.counts = grams;
    pl.counts_at = off;
    pl.parts_at = up(off + 4 * grams, 1024);
    off = pl.parts_at + grams * (128 * 64 * 4);
  }
  for (int32_t i = 0; i < count; ++i) {
    sides(i, m, n);
    if (t) t->mat[i].base = off;
    off = up(off + (m <= kMuonThin ? thin_bytes(m, n) : muon_layout(up(m, kMuonPad), up(n, kMuonPad)).end), 1024);
  }
  pl.bytes = off;
  return pl;
}

// Work units of a matrix in each kernel.  Thin matrices need no norm (their Gram matrix has
// it), so no pass of their own without a momentum.
int64_t units_of(const MuonMat& m, int kind, const Plan& pl) {
  const bool thin = m.m <= kMuonThin;
  const int64_t T = m.mp / 256;
  switch (kind) {
    case kUnitsMoment: return !thin || m.mom ? m.parts : 0;
    case kUnitsThin: return thin ? thin_chunks(m.n) : 0;
    case kUnitsPrepare: return thin ? 0 : (int64_t)(m.mp / 128) * (m.np / 64);
    case kUnitsGram:
      if (pl.small && !thin) return muon_gram_tiles(m.m) * muon_splits(muon_steps(m.n), pl.split_steps);
      [[fallthrough]];
    case kUnitsSquare: return thin ? 0 : pl.small ? muon_gram_tiles(m.m) : T * (T + 1) / 2;
    default: return thin ? 0 : pl.small ? (int64_t)muon_row_tiles(m.m) * muon_steps(m.n) : T * (m.np / 256);
  }
}

thread_local MuonTable t_table;   // 25 KB: too large for every caller's stack

fs4_status run(int32_t count, const fs4_muon_desc* descs, bool step, int32_t K, const float* coeffs, int32_t n_coeffs, double lr,
               double beta, double weight_decay, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (!descs || !coeffs) return FS4_ERR_INVALID_ARG;
  if (count < 1 || count > kMuonMaxBatch || K < 1 || K > FS4_MAX_ITERS) return FS4_ERR_SHAPE;
  if (n_coeffs != 1 && n_coeffs != K) return FS4_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(step ? FS4_MUON_NESTEROV | FS4_TEST_STALL : 0u)) return FS4_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n_coeffs; ++i)
    if (!coeffs_ok(coeffs + 3 * i)) return FS4_ERR_INVALID_ARG;
  // the kernels take the rate and the decay factor in FP32, where 0 times infinity would be NaN
  if (step && (!(lr >= 0.0 && lr <= FLT_MAX) || !(beta >= 0.0 && beta < 1.0) || !(std::fabs(1.0 - lr * weight_decay) <= FLT_MAX)))
    return FS4_ERR_INVALID_ARG;
  MuonTable& t = t_table;
  static thread_local int64_t rows[kMuonMaxBatch], cols[kMuonMaxBatch];
  static thread_local Span out[2 * kMuonMaxBatch], in[kMuonMaxBatch];
  int32_t outs = 0;
  for (int32_t i = 0; i < count; ++i) {
    const fs4_muon_desc& d = descs[i];
    if (!d.w || !d.g || (step ? !d.m : d.m != nullptr)) return FS4_ERR_INVALID_ARG;
    if (!shape_ok(d.rows, d.cols)) return FS4_ERR_SHAPE;
    if (!known_type(d.w_dtype) || !known_type(d.g_dtype) || (step && !known_type(d.m_dtype)) || !std::isfinite(d.scale))
      return FS4_ERR_INVALID_ARG;
    if (d.ld_w < d.cols || d.ld_g < d.cols || (step && d.ld_m < d.cols)) return FS4_ERR_INVALID_ARG;
    const int64_t most = INT64_MAX / 4 / d.rows;
    if (d.ld_w > most || d.ld_g > most || (step && d.ld_m > most)) return FS4_ERR_INVALID_ARG;
    if (!aligned(d.w, type_bytes(d.w_dtype)) || !aligned(d.g, type_bytes(d.g_dtype)) || (step && !aligned(d.m, type_bytes(d.m_dtype))))
      return FS4_ERR_INVALID_ARG;
    MuonMat& m = t.mat[i];
    m.g = d.g; m.mom = step ? d.m : nullptr; m.w = d.w;
    m.ldg = d.ld_g; m.ldm = d.ld_m; m.ldw = d.ld_w;
    m.tg = (int8_t)d.g_dtype; m.tm = (int8_t)(step ? d.m_dtype : 0); m.tw = (int8_t)d.w_dtype;
    m.scale = d.scale;
    m.tall = d.rows > d.cols;
    m.m = (int32_t)(m.tall ? d.cols : d.rows);
    m.n = (int32_t)(m.tall ? d.rows : d.cols);
    m.mp = (int32_t)up(m.m, kMuonPad);
    m.np = (int32_t)up(m.n, kMuonPad);
    rows[i] = d.rows;
    cols[i] = d.cols;
    in[i] = matrix_at(d.g, d.rows, d.cols, d.ld_g, d.g_dtype);
    out[outs++] = matrix_at(d.w, d.rows, d.cols, d.ld_w, d.w_dtype);
    if (step) out[outs++] = matrix_at(d.m, d.rows, d.cols, d.ld_m, d.m_dtype);
  }
  const Plan pl = plan(count, rows, cols, &t);
  const int64_t need = pl.bytes;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < (size_t)need) return FS4_ERR_WORKSPACE;
  const Span ws = bytes_at(workspace, need);
  for (int32_t i = 0; i < outs; ++i) {
    if (meet(out[i], ws)) return FS4_ERR_ALIAS;
    for (int32_t k = 0; k < count; ++k)
      if (meet(out[i], in[k])) return FS4_ERR_ALIAS;
    for (int32_t k = i + 1; k < outs; ++k)
      if (meet(out[i], out[k])) return FS4_ERR_ALIAS;
  }
  for (int32_t k = 0; k < count; ++k)
    if (meet(in[k], ws)) return FS4_ERR_ALIAS;
  int sms = 0;
  const fs4_status ds = current_device(&sms);
  if (ds != FS4_OK) return ds;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int kind = 0; kind < kUnitKinds; ++kind) {
    int64_t acc = 0;
    t.prefix[kind][0] = 0;
    for (int32_t i = 0; i < count; ++i) {
      acc += units_of(t.mat[i], kind, pl);
      if (acc > 0x7FFFFFFF) return FS4_ERR_SHAPE;
      t.prefix[kind][i + 1] = (int32_t)acc;
    }
  }
  MuonCall c{};
  c.ws = static_cast<uint8_t*>(workspace);
  c.count = count;
  c.K = K;
  c.n_coeffs = n_coeffs;
  c.nesterov = (flags & FS4_MUON_NESTEROV) ? 1 : 0;
  c.beta = (float)beta;
  c.rest = (float)(1.0 - beta);
  c.rate = step ? (float)lr : -1.0f;
  c.keep = step ? (float)(1.0 - lr * weight_decay) : 0.0f;
  c.small = pl.small ? 1 : 0;
  c.split_steps = pl.split_steps;
  c.parts_at = pl.parts_at;
  c.counts_at = pl.counts_at;
  c.counts = (int32_t)pl.counts;
  c.stall = (flags & FS4_TEST_STALL) ? 1 : 0;
  std::memcpy(c.coeffs, coeffs, sizeof(float) * 3 * n_coeffs);
  if (launch_muon_moment(c, t, st) != cudaSuccess) return FS4_ERR_CUDA;
  if (t.prefix[kUnitsThin][count] && launch_muon_thin(c, t.prefix[kUnitsThin][count], st) != cudaSuccess) return FS4_ERR_CUDA;
  if (t.prefix[kUnitsPrepare][count]) {
    if (launch_muon_prepare(c, t.prefix[kUnitsPrepare][count], st, sms) != cudaSuccess) return FS4_ERR_CUDA;
    int32_t units = 0;
    for (int kind : {kUnitsGram, kUnitsSquare, kUnitsUpdate})
      if (t.prefix[kind][count] > units) units = t.prefix[kind][count];
    if (launch_muon_iterate(c, need, units, st, sms) != cudaSuccess) return FS4_ERR_CUDA;
  }
  return FS4_OK;
}

}  // namespace

extern "C" {

size_t fs4_muon_workspace_size(int32_t count, const int64_t* rows, const int64_t* cols) {
  if (count < 1 || count > kMuonMaxBatch || !rows || !cols) return 0;
  for (int32_t i = 0; i < count; ++i)
    if (!shape_ok(rows[i], cols[i])) return 0;
  return (size_t)plan(count, rows, cols, nullptr).bytes;
}

fs4_status fs4_muon_orthogonalize(int32_t count, const fs4_muon_desc* descs, int32_t K, const float* coeffs, int32_t n_coeffs,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return run(count, descs, false, K, coeffs, n_coeffs, 0.0, 0.0, 0.0, 0u, workspace, workspace_bytes, stream);
}

fs4_status fs4_muon_step(int32_t count, const fs4_muon_desc* descs, int32_t K, const float* coeffs, int32_t n_coeffs, double lr,
                         double beta, double weight_decay, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
  return run(count, descs, true, K, coeffs, n_coeffs, lr, beta, weight_decay, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
