// tg_train_api.cu -- the C ABI of the training operators (include/tg.h): argument checks and
// launches of layer norm and of activation checkpoints in 8 bits.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/tg.h"
#include "tg_api_common.h"
#include "tg_internal.h"
#include "tg_tile_scheduler.cuh"
#include "tg_wgrad_config.h"

using namespace tg::abi;

namespace {

bool known_dtype(int d) { return d == TG_F16 || d == TG_BF16 || d == TG_F32; }
uint64_t elem_bytes(int d) { return d == TG_F32 ? 4 : 2; }
uint64_t kept_blocks(int64_t cols) { return (static_cast<uint64_t>(cols) + 31) / 32; }

bool off_by(const void* p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// bytes from the first to the last element of a [rows, cols] matrix with row stride ld
uint64_t span(int64_t rows, int64_t cols, int64_t ld, uint64_t elem) {
  return rows == 0 ? 0 : ((static_cast<uint64_t>(rows) - 1) * ld + cols) * elem;
}

int check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
    return fail(TG_ERR_ARG, "sizes must be in [0, 2^31): rows=%lld cols=%lld", (long long)rows,
                (long long)cols);
  return TG_OK;
}

int check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > kMaxDim)
    return fail(TG_ERR_ARG, "%s=%lld must be at least the row's %lld values and below 2^31", name,
                (long long)ld, (long long)cols);
  return TG_OK;
}

// A required device array of ``elem``-byte elements.
int check_array(const void* p, uint64_t elem, const char* name) {
  if (!p) return fail(TG_ERR_ARG, "null pointer: %s", name);
  if (off_by(p, elem))
    return fail(TG_ERR_ALIGN, "%s must be %llu-byte aligned", name, (unsigned long long)elem);
  return check_device_ptr(p, name);
}

// The array ``p`` if the caller gave it.
int check_optional(const void* p, uint64_t elem, const char* name) {
  return p ? check_array(p, elem, name) : TG_OK;
}

// A device array: ``bytes`` from its first element to past its last.  pitch != 0: a matrix whose
// rows are ``row`` bytes, ``pitch`` bytes apart.
struct Region {
  const void* p;
  uint64_t bytes;
  const char* name;
  uint64_t row = 0, pitch = 0;
};

Region matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, uint64_t elem,
              const char* name) {
  return {p, span(rows, cols, ld, elem), name, cols * elem, ld * elem};
}

// Whether two arrays share no byte.  Matrices of one pitch may lie in each other's gaps, as column
// slices of one buffer do: their rows then take separate parts of every ``pitch`` bytes.  Anything
// else is told apart by where it begins and ends.
bool apart(const Region& a, const Region& b) {
  if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return true;
  if (a.pitch == 0 || a.pitch != b.pitch) return false;
  const uint64_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  // how far into a's rows b's begin
  const uint64_t at = b0 >= a0 ? (b0 - a0) % a.pitch : a.pitch - 1 - (a0 - b0 - 1) % a.pitch;
  return at >= a.row && at + b.row <= a.pitch;
}

// No output may overlap an input or another output (regions [0, outs) are the outputs).
int check_apart(const Region* r, int outs, int n) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (r[i].p && r[j].p && !apart(r[i], r[j]))
        return fail(TG_ERR_ARG, "%s overlaps %s", r[i].name, r[j].name);
  return TG_OK;
}

int check_params(int dtype, int param_dtype) {
  if (!known_dtype(dtype)) return fail(TG_ERR_ARG, "unknown dtype %d", dtype);
  if (param_dtype != TG_F32 && param_dtype != dtype)
    return fail(TG_ERR_ARG, "param_dtype %d must be TG_F32 or the values' type %d", param_dtype,
                dtype);
  return TG_OK;
}

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// How the weight gradient [cols, outs] over ``tokens`` tokens is cut into units.
struct WgradPlan {
  uint32_t halves;      // N-halves of 256 columns in a tile of dW
  uint32_t m_tiles, n_tiles, k_blocks, splits, blocks_per_split, split_from, units, pairs;
  uint64_t workspace;   // bytes of partial sums (0: one split)
  double us;            // what the plan is expected to take
};

// Microseconds on GB300 that the choice of a plan goes by: a k-block of a whole tile and of its
// half-width unit; what a unit's epilogue keeps the MMAs waiting (two accumulators overlap it); the
// join, and bytes of partial sums a microsecond, written and read.
constexpr double kWgBlockUs[2] = {0.40, 0.56}, kWgHalfBlockUs[2] = {0.33, 0.40};
constexpr double kWgDrainUs[2] = {0.2, 2.0}, kWgJoinUs = 2.5;
constexpr double kWgWriteBytes = 5e6, kWgReadBytes = 4e6;
constexpr uint64_t kWgMinBlocks = 8;   // k-blocks of a unit, when the tokens are split

// The plan with tiles of ``halves`` N-halves and the tokens in about ``splits`` ranges.
WgradPlan wgrad_plan_of(int64_t tokens, int64_t cols, int64_t outs, uint64_t pairs,
                        uint32_t halves, uint64_t splits) {
  WgradPlan w;
  w.halves = halves;
  w.m_tiles = static_cast<uint32_t>(ceil_div(cols, tg::kPairBM));
  w.n_tiles = static_cast<uint32_t>(ceil_div(outs, halves * tg::kBN));
  w.k_blocks = static_cast<uint32_t>(ceil_div(tokens, tg::kWgBK));
  const uint32_t tiles = w.m_tiles * w.n_tiles;
  w.blocks_per_split = static_cast<uint32_t>(ceil_div(w.k_blocks, splits));
  w.splits = w.k_blocks ? static_cast<uint32_t>(ceil_div(w.k_blocks, w.blocks_per_split)) : 1;
  w.workspace = 0;
  w.split_from = w.units = tiles;
  if (w.splits == 1)
    tg::PersistentTileScheduler::tail_split(tiles, static_cast<uint32_t>(pairs), w.split_from,
                                            w.units);
  const uint64_t all = static_cast<uint64_t>(w.units) * w.splits;
  w.pairs = static_cast<uint32_t>(all < pairs ? all : pairs);
  const uint32_t h = halves - 1;
  const double whole = static_cast<double>(ceil_div(w.split_from * uint64_t(w.splits), pairs));
  w.us = whole * (w.blocks_per_split * kWgBlockUs[h] + kWgDrainUs[h]);
  if (w.units > w.split_from) w.us += w.k_blocks * kWgHalfBlockUs[h];
  if (w.splits > 1) {
    w.workspace = static_cast<uint64_t>(w.splits) * w.m_tiles * tg::kPairBM * outs * 4;
    const double sums = static_cast<double>(w.splits) * cols * outs * 4.0;
    w.us += sums / kWgWriteBytes + kWgJoinUs + sums / kWgReadBytes;
  }
  return w;
}

// Tiles of two N-halves halve the bytes that have to be widened for each multiplication, and have
// eight MMAs a k-block where one half has four and is bound by shared memory; tiles of one make
// smaller units, which fill the pairs when there are few.  Fewer tiles than pairs: the tokens may
// also be split, so that every pair has a unit, at the price of partial sums in fp32.  The least
// expected time decides.  Measured (bf16, us back to back; one half / two halves, splits in
// brackets): 8192^3 760 / 558, 1024 x 4096 x 4096 36 / 30, 32768 x 1000
// x 512 36.5 [9] / 36.6 [19], 65536 x 512 x 512 38.6 [19] / 44.8 [38]; two halves, whole / split:
// 2048^3 19.4 / 26.3 [2], 16384 x 2048 x 1024 - / 53 [4].
WgradPlan wgrad_plan(int64_t tokens, int64_t cols, int64_t outs, int max_pairs) {
  const uint64_t pairs = static_cast<uint64_t>(max_pairs);
  WgradPlan best = wgrad_plan_of(tokens, cols, outs, pairs, 1, 1);
  for (uint32_t halves = 1; halves <= (outs > tg::kBN ? 2u : 1u); ++halves) {
    const WgradPlan whole = wgrad_plan_of(tokens, cols, outs, pairs, halves, 1);
    if (whole.us < best.us) best = whole;
    uint64_t splits = pairs / (uint64_t(whole.m_tiles) * whole.n_tiles);
    if (splits > whole.k_blocks / kWgMinBlocks) splits = whole.k_blocks / kWgMinBlocks;
    if (splits < 2) continue;
    const WgradPlan cut = wgrad_plan_of(tokens, cols, outs, pairs, halves, splits);
    if (cut.us < best.us) best = cut;
  }
  return best;
}

int check_wgrad_sizes(int64_t tokens, int64_t cols, int64_t outs) {
  if (int rc = check_sizes(tokens, cols)) return rc;
  if (outs < 0 || outs > kMaxDim)
    return fail(TG_ERR_ARG, "outs=%lld must be in [0, 2^31)", (long long)outs);
  if (outs % 8 != 0)
    return fail(TG_ERR_ALIGN, "outs=%lld must be a multiple of 8 (16-byte rows)", (long long)outs);
  if (ceil_div(cols, 128) * ceil_div(outs, 256) > static_cast<uint64_t>(kMaxDim))
    return fail(TG_ERR_ARG, "too many output tiles");
  return TG_OK;
}

#define TG_TRY(call)                 \
  do {                               \
    const int rc_ = (call);          \
    if (rc_ != TG_OK) return rc_;    \
  } while (0)

int wgrad_impl(const void* q, const void* sc, const void* dy, void* dw, int64_t tokens, int64_t cols,
               int64_t outs, int64_t ld_dy, int64_t ld_dw, int dtype, void* ws, int64_t ws_bytes,
               void* stream, bool debug, uint64_t watchdog_ns, int64_t inject) {
  if (dtype != TG_F16 && dtype != TG_BF16) return fail(TG_ERR_ARG, "unknown dtype %d", dtype);
  TG_TRY(check_wgrad_sizes(tokens, cols, outs));
  TG_TRY(check_ld(ld_dy, outs, "ld_dy"));
  TG_TRY(check_ld(ld_dw, outs, "ld_dw"));
  if (ws_bytes < 0) return fail(TG_ERR_ARG, "negative workspace size");
  if (cols == 0 || outs == 0) return TG_OK;
  if (ld_dy % 8 != 0 || ld_dw % 8 != 0)
    return fail(TG_ERR_ALIGN, "ld_dy=%lld and ld_dw=%lld must be multiples of 8 (16-byte rows)",
                (long long)ld_dy, (long long)ld_dw);
  TG_TRY(check_array(dw, 16, "dW"));
  const uint64_t kb = kept_blocks(cols);
  if (tokens > 0) {
    TG_TRY(check_array(q, 16, "q"));
    TG_TRY(check_array(sc, 1, "s"));
    TG_TRY(check_array(dy, 16, "dY"));
  }
  int sms = 0, max_pairs = 0;
  TG_TRY(wgrad_ready(&sms, &max_pairs));
  const WgradPlan w = wgrad_plan(tokens, cols, outs, max_pairs);
  if (w.workspace > 0) {
    if (!ws || static_cast<uint64_t>(ws_bytes) < w.workspace)
      return fail(TG_ERR_ARG, "workspace of %lld bytes; the split sums need %llu",
                  (long long)(ws ? ws_bytes : 0), (unsigned long long)w.workspace);
    TG_TRY(check_array(ws, 256, "workspace"));
  }
  const Region r[] = {matrix(dw, cols, outs, ld_dw, 2, "dW"),
                      {w.workspace ? ws : nullptr, w.workspace, "workspace"},
                      {q, tokens * kb * 32, "q"},
                      {sc, tokens * kb, "s"},
                      matrix(dy, tokens, outs, ld_dy, 2, "dY")};
  TG_TRY(check_apart(r, 2, 5));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tokens == 0) {
    e = cudaMemset2DAsync(dw, ld_dw * 2, 0, outs * 2, cols, st);
    return e == cudaSuccess ? TG_OK : fail_cuda("zero fill of dW", e);
  }
  const CUtensorMapDataType t16 =
      dtype == TG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  tg::WgradLaunch l;
  TG_TRY(encode_tiled(&l.tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q, kb * 32, tokens, tg::kBM,
                      tg::kWgBK, "q", false));
  TG_TRY(encode_tiled(&l.tmB, t16, 2, dy, outs, tokens, tg::kBChunkCols, tg::kWgBK, "dY", true,
                      ld_dy * 2));
  if (w.splits > 1)
    TG_TRY(encode_tiled(&l.tmC, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ws, outs,
                        static_cast<uint64_t>(w.splits) * w.m_tiles * tg::kPairBM, 32, 32,
                        "workspace"));
  else
    TG_TRY(encode_tiled(&l.tmC, t16, 2, dw, outs, cols, tg::kEpiN, 32, "dW", true, ld_dw * 2));
  l.tma_scales = kb % 16 == 0 && !off_by(sc, 16) ? 1u : 0u;
  l.tmS = l.tmQ;
  if (l.tma_scales)
    TG_TRY(encode_tiled(&l.tmS, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, sc, kb, tokens,
                        tg::kWgScalePitch, tg::kWgBK, "s", false));
  l.scales = sc;
  l.dw = dw;
  l.partials = static_cast<float*>(ws);
  l.cols = static_cast<uint32_t>(cols);
  l.outs = static_cast<uint32_t>(outs);
  l.tokens = static_cast<uint32_t>(tokens);
  l.scale_cols = static_cast<uint32_t>(kb);
  l.ld_dw = ld_dw;
  l.m_blocks = w.m_tiles;
  l.n_blocks = w.n_tiles;
  l.k_blocks = w.k_blocks;
  // Whole columns of tiles in turn: a wave reads few columns of dY and all of x, which is half of
  // dY's size a value and stays in the L2.  Measured (us, bf16, whole columns / groups of 8 in row
  // order): 8192^3 566 / 580, 32768 x 8192 x 4096 1138 / 1191, 16384 x 2048 x 16384 623 / 648,
  // 4000 x 2048 x 7000 84.6 / 84.6, 16384 x 16384 x 2048 591 / 586.
  l.group = w.m_tiles < 255u ? w.m_tiles : 255u;
  l.column_major = 1;
  l.split_from = w.split_from;
  l.total_units = w.units;
  l.splits = w.splits;
  l.blocks_per_split = w.blocks_per_split;
  l.halves = w.halves;
  l.grid = 2 * w.pairs;
  l.watchdog_ns = watchdog_ns ? watchdog_ns : default_watchdog_ns(w.k_blocks);
  l.inject_skip_phase = inject;
  l.sms = sms;
  if (debug && (e = tg::clear_watchdog_status(st)) != cudaSuccess)
    return fail_cuda("clearing the watchdog word", e);
  if ((e = tg::launch_wgrad(dtype, debug, l, st)) != cudaSuccess)
    return fail_cuda("weight gradient launch", e);
  if (debug) {
    unsigned int word = 0;
    if ((e = tg::read_and_clear_watchdog_status(&word, st)) != cudaSuccess)
      return fail_cuda("weight gradient execution", e);
    if (word)
      return fail(TG_ERR_TIMEOUT, "watchdog: a wait gave up (roles 0x%x: 1 producer or conversion, "
                  "2 MMA, 4 epilogue, 8 shutdown)", word);
  }
  return TG_OK;
}

}  // namespace

extern "C" {

int tg_layernorm_fwd(const void* x_dev, const void* gamma_dev, const void* beta_dev, void* y_dev,
                     float* mean_dev, float* rstd_dev, void* yq_dev, void* ys_dev, int64_t rows,
                     int64_t cols, int64_t ld_x, int64_t ld_y, int dtype, int param_dtype,
                     float eps, void* stream) {
  TG_TRY(check_params(dtype, param_dtype));
  TG_TRY(check_sizes(rows, cols));
  TG_TRY(check_ld(ld_x, cols, "ld_x"));
  TG_TRY(check_ld(ld_y, cols, "ld_y"));
  if (!(eps >= 0.0f)) return fail(TG_ERR_ARG, "eps must not be negative");
  if ((yq_dev == nullptr) != (ys_dev == nullptr))
    return fail(TG_ERR_ARG, "a checkpoint of y needs both yq and ys");
  if (rows == 0) return TG_OK;
  const uint64_t e = elem_bytes(dtype), pe = elem_bytes(param_dtype), kb = kept_blocks(cols);
  const uint64_t stat = 4 * static_cast<uint64_t>(rows), param = pe * cols;
  if (cols == 0) {   // the mean of no values: 0 / 0
    for (float* out : {mean_dev, rstd_dev}) {
      if (!out) continue;
      TG_TRY(check_array(out, 4, out == mean_dev ? "mean" : "rstd"));
      const cudaError_t err =   // every byte 255: NaN
          cudaMemsetAsync(out, 0xFF, stat, static_cast<cudaStream_t>(stream));
      if (err != cudaSuccess) return fail_cuda("filling the statistics", err);
    }
    return TG_OK;
  }
  TG_TRY(check_array(x_dev, e, "x"));
  TG_TRY(check_array(y_dev, e, "y"));
  TG_TRY(check_optional(gamma_dev, pe, "gamma"));
  TG_TRY(check_optional(beta_dev, pe, "beta"));
  TG_TRY(check_optional(mean_dev, 4, "mean"));
  TG_TRY(check_optional(rstd_dev, 4, "rstd"));
  TG_TRY(check_optional(yq_dev, 16, "yq"));
  TG_TRY(check_optional(ys_dev, 1, "ys"));
  const Region r[] = {matrix(y_dev, rows, cols, ld_y, e, "y"),
                      {mean_dev, stat, "mean"},
                      {rstd_dev, stat, "rstd"},
                      {yq_dev, rows * kb * 32, "yq"},
                      {ys_dev, rows * kb, "ys"},
                      matrix(x_dev, rows, cols, ld_x, e, "x"),
                      {gamma_dev, param, "gamma"},
                      {beta_dev, param, "beta"}};
  TG_TRY(check_apart(r, 5, 8));
  int sms = 0;
  TG_TRY(device_ready(&sms, nullptr));
  tg::NormLaunch l;
  l.sms = sms;
  l.x = x_dev;
  l.gamma = gamma_dev;
  l.beta = beta_dev;
  l.y = y_dev;
  l.mean = mean_dev;
  l.rstd = rstd_dev;
  l.q = yq_dev;
  l.s = ys_dev;
  l.rows = rows;
  l.cols = cols;
  l.ld_x = ld_x;
  l.ld_y = ld_y;
  l.dtype = dtype;
  l.param_dtype = param_dtype;
  l.eps = eps;
  const cudaError_t err = tg::launch_norm_fwd(l, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TG_OK : fail_cuda("layer norm launch", err);
}

int64_t tg_layernorm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  TG_TRY(check_sizes(rows, cols));
  if (rows == 0 || cols == 0) return 0;
  int sms = 0;
  TG_TRY(device_ready(&sms, nullptr));
  return tg::norm_bwd_workspace(rows, cols, sms);
}

int tg_layernorm_bwd(const void* dy_dev, const void* x_dev, const void* xq_dev, const void* xs_dev,
                     const void* gamma_dev, const float* mean_dev, const float* rstd_dev,
                     void* dx_dev, void* dgamma_dev, void* dbeta_dev, int64_t rows, int64_t cols,
                     int64_t ld_dy, int64_t ld_x, int64_t ld_dx, int dtype, int param_dtype,
                     void* workspace_dev, int64_t workspace_bytes, void* stream) {
  TG_TRY(check_params(dtype, param_dtype));
  TG_TRY(check_sizes(rows, cols));
  TG_TRY(check_ld(ld_dy, cols, "ld_dy"));
  TG_TRY(check_ld(ld_dx, cols, "ld_dx"));
  if (x_dev) TG_TRY(check_ld(ld_x, cols, "ld_x"));
  if ((xq_dev == nullptr) != (xs_dev == nullptr))
    return fail(TG_ERR_ARG, "a checkpoint of x is both xq and xs");
  if (x_dev && xq_dev) return fail(TG_ERR_ARG, "give x or its checkpoint, not both");
  if (workspace_bytes < 0) return fail(TG_ERR_ARG, "negative workspace size");
  if (cols == 0) return TG_OK;
  const uint64_t e = elem_bytes(dtype), pe = elem_bytes(param_dtype), kb = kept_blocks(cols);
  if (rows > 0) {
    TG_TRY(check_array(dy_dev, e, "dy"));
    if (xq_dev) {
      TG_TRY(check_array(xq_dev, 16, "xq"));
      TG_TRY(check_array(xs_dev, 1, "xs"));
    } else {
      TG_TRY(check_array(x_dev, e, "x"));
    }
    TG_TRY(check_array(mean_dev, 4, "mean"));
    TG_TRY(check_array(rstd_dev, 4, "rstd"));
    TG_TRY(check_array(dx_dev, e, "dx"));
    TG_TRY(check_optional(gamma_dev, pe, "gamma"));
  }
  TG_TRY(check_optional(dgamma_dev, pe, "dgamma"));
  TG_TRY(check_optional(dbeta_dev, pe, "dbeta"));
  int sms = 0;
  TG_TRY(device_ready(&sms, nullptr));
  const bool sums = dgamma_dev || dbeta_dev;
  const int64_t need = sums && rows > 0 ? tg::norm_bwd_workspace(rows, cols, sms) : 0;
  if (need > 0) {
    if (!workspace_dev || workspace_bytes < need)
      return fail(TG_ERR_ARG, "workspace of %lld bytes; dgamma and dbeta need %lld",
                  (long long)(workspace_dev ? workspace_bytes : 0), (long long)need);
    TG_TRY(check_array(workspace_dev, 256, "workspace"));
  }
  const uint64_t stat = 4 * static_cast<uint64_t>(rows), param = pe * cols;
  const Region r[] = {matrix(rows > 0 ? dx_dev : nullptr, rows, cols, ld_dx, e, "dx"),
                      {dgamma_dev, param, "dgamma"},
                      {dbeta_dev, param, "dbeta"},
                      {need > 0 ? workspace_dev : nullptr, static_cast<uint64_t>(need), "workspace"},
                      matrix(dy_dev, rows, cols, ld_dy, e, "dy"),
                      matrix(x_dev, rows, cols, ld_x, e, "x"),
                      {xq_dev, rows * kb * 32, "xq"},
                      {xs_dev, rows * kb, "xs"},
                      {mean_dev, stat, "mean"},
                      {rstd_dev, stat, "rstd"},
                      {gamma_dev, param, "gamma"}};
  TG_TRY(check_apart(r, 4, 11));
  tg::NormBwdLaunch l;
  l.dy = dy_dev;
  l.x = x_dev;
  l.q = xq_dev;
  l.s = xs_dev;
  l.gamma = gamma_dev;
  l.mean = mean_dev;
  l.rstd = rstd_dev;
  l.dx = dx_dev;
  l.dgamma = dgamma_dev;
  l.dbeta = dbeta_dev;
  l.partials = static_cast<float*>(workspace_dev);
  l.rows = rows;
  l.cols = cols;
  l.ld_dy = ld_dy;
  l.ld_x = ld_x;
  l.ld_dx = ld_dx;
  l.dtype = dtype;
  l.param_dtype = param_dtype;
  l.sms = sms;
  const cudaError_t err = tg::launch_norm_bwd(l, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TG_OK : fail_cuda("layer norm backward launch", err);
}

int tg_ckpt8_pack(const void* x_dev, void* q_dev, void* s_dev, int64_t rows, int64_t cols,
                  int64_t ld_x, int dtype, void* stream) {
  if (!known_dtype(dtype)) return fail(TG_ERR_ARG, "unknown dtype %d", dtype);
  TG_TRY(check_sizes(rows, cols));
  TG_TRY(check_ld(ld_x, cols, "ld_x"));
  if (rows == 0 || cols == 0) return TG_OK;
  TG_TRY(check_array(x_dev, elem_bytes(dtype), "x"));
  TG_TRY(check_array(q_dev, 16, "q"));
  TG_TRY(check_array(s_dev, 1, "s"));
  const uint64_t kb = kept_blocks(cols);
  const Region r[] = {{q_dev, rows * kb * 32, "q"},
                      {s_dev, rows * kb, "s"},
                      matrix(x_dev, rows, cols, ld_x, elem_bytes(dtype), "x")};
  TG_TRY(check_apart(r, 2, 3));
  int sms = 0;
  TG_TRY(device_ready(&sms, nullptr));
  const cudaError_t err = tg::launch_ckpt8_pack(x_dev, q_dev, s_dev, rows, cols, ld_x, dtype, sms,
                                                static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TG_OK : fail_cuda("checkpoint pack launch", err);
}

int tg_ckpt8_unpack(const void* q_dev, const void* s_dev, void* out_dev, int64_t rows, int64_t cols,
                    int64_t ld_out, int dtype, void* stream) {
  if (!known_dtype(dtype)) return fail(TG_ERR_ARG, "unknown dtype %d", dtype);
  TG_TRY(check_sizes(rows, cols));
  TG_TRY(check_ld(ld_out, cols, "ld_out"));
  if (rows == 0 || cols == 0) return TG_OK;
  TG_TRY(check_array(q_dev, 16, "q"));
  TG_TRY(check_array(s_dev, 1, "s"));
  TG_TRY(check_array(out_dev, elem_bytes(dtype), "out"));
  const uint64_t kb = kept_blocks(cols);
  const Region r[] = {matrix(out_dev, rows, cols, ld_out, elem_bytes(dtype), "out"),
                      {q_dev, rows * kb * 32, "q"},
                      {s_dev, rows * kb, "s"}};
  TG_TRY(check_apart(r, 1, 3));
  int sms = 0;
  TG_TRY(device_ready(&sms, nullptr));
  const cudaError_t err = tg::launch_ckpt8_unpack(q_dev, s_dev, out_dev, rows, cols, ld_out, dtype,
                                                  sms, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? TG_OK : fail_cuda("checkpoint unpack launch", err);
}

int64_t tg_ckpt8_wgrad_workspace_bytes(int64_t rows, int64_t cols, int64_t outs) {
  TG_TRY(check_wgrad_sizes(rows, cols, outs));
  if (rows == 0 || cols == 0 || outs == 0) return 0;
  int max_pairs = 0;
  TG_TRY(wgrad_ready(nullptr, &max_pairs));
  return static_cast<int64_t>(wgrad_plan(rows, cols, outs, max_pairs).workspace);
}

int tg_ckpt8_wgrad(const void* q_dev, const void* s_dev, const void* dY_dev, void* dW_dev,
                   int64_t rows, int64_t cols, int64_t outs, int64_t ld_dy, int64_t ld_dw,
                   int dtype, void* workspace_dev, int64_t workspace_bytes, void* stream) {
  return wgrad_impl(q_dev, s_dev, dY_dev, dW_dev, rows, cols, outs, ld_dy, ld_dw, dtype,
                    workspace_dev, workspace_bytes, stream, false, 0, -1);
}

int tg_ckpt8_wgrad_debug(const void* q_dev, const void* s_dev, const void* dY_dev, void* dW_dev,
                         int64_t rows, int64_t cols, int64_t outs, int64_t ld_dy, int64_t ld_dw,
                         int dtype, void* workspace_dev, int64_t workspace_bytes, void* stream,
                         uint64_t watchdog_ns, int64_t inject_skip_phase) {
  return wgrad_impl(q_dev, s_dev, dY_dev, dW_dev, rows, cols, outs, ld_dy, ld_dw, dtype,
                    workspace_dev, workspace_bytes, stream, true, watchdog_ns, inject_skip_phase);
}

}  // extern "C"
