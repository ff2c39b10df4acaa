// tg_train.cu -- instantiations and launchers of the operators around the GEMM in training: layer
// norm forward and backward, and activation checkpoints in 8 bits.
#include <atomic>
#include <type_traits>

#include "../../include/tg.h"
#include "tg_ckpt8_kernel.cuh"
#include "tg_internal.h"
#include "tg_launch.cuh"
#include "tg_norm_kernel.cuh"
#include "tg_norm_short_kernel.cuh"

namespace tg {

namespace {

uint32_t round_up(uint64_t n, uint32_t to) { return static_cast<uint32_t>((n + to - 1) / to * to); }

// Every row starts on a 16-byte boundary (a null matrix has no say).
bool rows_aligned(const void* p, int64_t ld, uint32_t elem) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
                          static_cast<uint64_t>(ld) * elem % 16 == 0);
}

RowsOf rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t elem) {
  RowsOf r;
  r.base = static_cast<char*>(const_cast<void*>(p));
  r.end = p ? r.base + ((rows - 1) * ld + cols) * static_cast<int64_t>(elem) : r.base;
  r.pitch = ld * static_cast<int64_t>(elem);
  return r;
}

// Names a type as an argument of a generic lambda.
template <typename T>
struct Of {
  using type = T;
};

// Calls f(Of<TX>, Of<TP>) for the element type and the parameters' type.
template <typename F>
cudaError_t with_types(int dtype, int param_dtype, F&& f) {
  if (dtype == TG_F32) return f(Of<float>(), Of<float>());
  if (dtype == TG_F16)
    return param_dtype == TG_F32 ? f(Of<__half>(), Of<float>()) : f(Of<__half>(), Of<__half>());
  return param_dtype == TG_F32 ? f(Of<__nv_bfloat16>(), Of<float>())
                               : f(Of<__nv_bfloat16>(), Of<__nv_bfloat16>());
}

template <typename F>
cudaError_t with_type(int dtype, F&& f) {
  if (dtype == TG_F32) return f(Of<float>());
  return dtype == TG_F16 ? f(Of<__half>()) : f(Of<__nv_bfloat16>());
}

// ---------------------------------------------------------------- layer norm
// columns that one group of threads holds
constexpr int64_t kNormCols = kNormValues * kNormThreads;
constexpr int64_t kNormWideCols = kNormValues * kNormWideThreads;
constexpr uint32_t kLongParts = 64;
constexpr int64_t kShortBytes = 512;   // of a row that a warp holds

// Threads of a group, ``values`` columns each.
uint32_t group_threads(int64_t cols, int values) { return round_up((cols + values - 1) / values, 32); }

constexpr int kMostSmem = 224 * 1024;   // dynamic; the kernels' static share is below 3 KiB

// CTAs, and groups in each: as many groups as ``threads`` hold, no more than there are rows.
struct NormGrid {
  uint32_t g_threads, groups, ctas;
};
NormGrid norm_grid(int64_t rows, int64_t cols, int values, int threads, int sms) {
  NormGrid g;
  g.g_threads = group_threads(cols, values);
  g.ctas = static_cast<uint32_t>(rows < sms ? rows : sms);
  const int64_t per_cta = (rows + g.ctas - 1) / g.ctas;
  uint32_t most = threads / g.g_threads;
  if (most > kNormMaxGroups && g.g_threads > 32) most = kNormMaxGroups;
  g.groups = static_cast<uint32_t>(per_cta < most ? per_cta : most);
  return g;
}

// Lets kernel K use ``bytes`` of dynamic shared memory on the current device; asked of the driver
// once per device (it takes about a microsecond), as the GEMM kernels' limits are.
template <auto K>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || bytes <= 48 * 1024) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// log2 of the lanes that a short row takes: one vector each, and a checkpoint's block at least.
template <typename TX>
uint32_t short_shift(int64_t cols) {
  uint32_t shift = kVec<TX> == 8 ? 2u : 3u;
  while ((int64_t(kVec<TX>) << shift) < cols) ++shift;
  return shift;
}

// The largest of 16, 4 and the value's size that the bases, row pitches and the row's length are all
// multiples of (null matrices are zeros): passed to f as a constant.
template <typename TX, typename F>
cudaError_t with_access(int64_t cols, const RowsOf& a, const RowsOf& b, const RowsOf& c, F&& f) {
  uint64_t bits = static_cast<uint64_t>(cols) * sizeof(TX);
  for (const RowsOf* m : {&a, &b, &c})
    bits |= reinterpret_cast<uintptr_t>(m->base) | static_cast<uint64_t>(m->pitch);
  if (bits % 16 == 0) return f(std::integral_constant<int, 16>());
  if (bits % 4 == 0) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, static_cast<int>(sizeof(TX))>());
}

// kOneLead: every row starts as far into a granule in ``b`` as in ``a``.  The rows of a CTA are a
// multiple of the grid apart; where that is a multiple of 8 they start alike.
bool one_lead(const RowsOf& a, const RowsOf& b) {
  return (reinterpret_cast<uintptr_t>(a.base) - reinterpret_cast<uintptr_t>(b.base)) % 16 == 0 &&
         (a.pitch - b.pitch) % 16 == 0;
}

// Columns of a row of partial sums, in whole 128-byte lines; those of a lead, at most 7, come before.
uint32_t part_cols(int64_t cols, bool lead) { return round_up(cols + (lead ? 7 : 0), 32); }

bool wide(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_norm_fwd(const NormLaunch& l, cudaStream_t stream) {
  auto params = [&](size_t elem) {
    NormFwdParams p;
    p.x = rows_of(l.x, l.rows, l.cols, l.ld_x, elem);
    p.y = rows_of(l.y, l.rows, l.cols, l.ld_y, elem);
    p.gamma = l.gamma;
    p.beta = l.beta;
    p.wide_params = wide(l.gamma) && wide(l.beta) ? 1u : 0u;
    p.shared_params = 0;
    p.mean = l.mean;
    p.rstd = l.rstd;
    p.q = static_cast<uint8_t*>(l.q);
    p.s = static_cast<uint8_t*>(l.s);
    p.rows = static_cast<uint32_t>(l.rows);
    p.cols = static_cast<uint32_t>(l.cols);
    p.blocks = round_up(l.cols, kCkptBlock) / kCkptBlock;
    p.eps = l.eps;
    return p;
  };
  auto run_short = [&](auto tx, auto tp, auto keep) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    const NormFwdParams p = params(sizeof(TX));
    const uint32_t shift = short_shift<TX>(l.cols), per_warp = 32u >> shift;
    const int64_t turns = (l.rows + per_warp - 1) / per_warp;   // of a warp
    const int64_t most = static_cast<int64_t>(l.sms) * kShortFwdCtas;
    const int64_t ctas = turns < most ? turns : most, warps = (turns + ctas - 1) / ctas;
    constexpr int64_t kWarps = kShortFwdThreads / 32;
    const uint32_t threads = static_cast<uint32_t>(32 * (warps < kWarps ? warps : kWarps));
    return with_access<TX>(l.cols, p.x, p.y, p.y, [&](auto access) {
      return launch_pdl(
          norm_fwd_short_kernel<TX, TP, decltype(keep)::value, decltype(access)::value>,
          dim3(static_cast<uint32_t>(ctas)), threads, 0, stream, p, shift);
    });
  };
  auto run = [&](auto tx, auto tp, auto unal, auto keep) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    constexpr bool UNAL = decltype(unal)::value, KEEP = decltype(keep)::value;
    NormFwdParams p = params(sizeof(TX));
    auto grouped = [&](auto lie, auto n, auto m) -> cudaError_t {
      constexpr int kThreads = decltype(n)::value, kValues = decltype(m)::value;
      const NormGrid g = norm_grid(l.rows, l.cols, kValues, kThreads, UNAL ? l.sms & ~7 : l.sms);
      const uint32_t threads = g.groups * g.g_threads;
      size_t smem = norm_fwd_smem<TX, kThreads, kValues>(threads / 32);
      if (kValues == kFwdLongValues && l.cols <= kFwdParamCols) {
        p.shared_params = static_cast<uint32_t>(smem);
        smem += 2 * sizeof(float) * static_cast<size_t>(g.g_threads) * kValues;
      }
      constexpr auto kernel =
          norm_fwd_kernel<TX, TP, decltype(lie)::value, KEEP, kThreads, kValues>;
      cudaError_t e = allow_smem<kernel>(smem);
      if (e != cudaSuccess) return e;
      return launch_pdl(kernel, dim3(g.ctas), threads, smem, stream, p, g.g_threads);
    };
    constexpr std::integral_constant<int, UNAL ? kAnyRows : kWholeRows> kLie;
    constexpr std::integral_constant<int, kNormThreads> kOne;
    constexpr std::integral_constant<int, kNormWideThreads> kWide;
    // kOneLead where a row's last granule is still the group's
    auto held = [&](auto m) -> cudaError_t {
      constexpr int kValues = decltype(m)::value;
      if constexpr (UNAL && !KEEP)
        if (l.cols <= kNormCols && one_lead(p.x, p.y) &&
            group_threads(l.cols + kVec<TX> - 1, kValues) == group_threads(l.cols, kValues))
          return grouped(std::integral_constant<int, kOneLead>(), kOne, m);
      return grouped(kLie, kOne, m);
    };
    if constexpr (sizeof(TX) == 2)
      if (l.cols > kFwdLongCols && l.cols <= kNormWideCols &&
          l.rows * l.cols >= kFwdLongWork * l.sms)
        return held(std::integral_constant<int, kFwdLongValues>());
    constexpr std::integral_constant<int, kNormValues> kFew;
    if (l.cols <= kNormCols) return held(kFew);
    if (l.cols <= kNormWideCols) return grouped(kLie, kWide, kFew);
    return launch_pdl(norm_fwd_long_kernel<TX, TP, UNAL, KEEP>,
                      dim3(static_cast<uint32_t>(l.rows)), 1024, 0, stream, p);
  };
  return with_types(l.dtype, l.param_dtype, [&](auto tx, auto tp) -> cudaError_t {
    constexpr uint32_t kElem = sizeof(typename decltype(tx)::type);
    if (l.cols * kElem <= kShortBytes)
      return l.q ? run_short(tx, tp, std::true_type()) : run_short(tx, tp, std::false_type());
    const bool unal = l.cols * kElem % 16 != 0 || !rows_aligned(l.x, l.ld_x, kElem) ||
                      !rows_aligned(l.y, l.ld_y, kElem);
    if (l.q) return unal ? run(tx, tp, std::true_type(), std::true_type())
                         : run(tx, tp, std::false_type(), std::true_type());
    return unal ? run(tx, tp, std::true_type(), std::false_type())
                : run(tx, tp, std::false_type(), std::false_type());
  });
}

namespace {

// Rows of partial sums: one a CTA, or the row ranges of norm_bwd_cols_kernel.
uint32_t norm_bwd_parts(int64_t rows, int64_t cols, int dtype, int sms) {
  if (rows == 0) return 0;
  if (cols > (dtype == TG_F32 ? kNormCols : kNormWideCols))
    return static_cast<uint32_t>(rows < kLongParts ? rows : kLongParts);
  return static_cast<uint32_t>(rows < sms ? rows : sms);
}

}  // namespace

int64_t norm_bwd_workspace(int64_t rows, int64_t cols, int sms) {
  const uint32_t a = norm_bwd_parts(rows, cols, TG_F32, sms);
  const uint32_t b = norm_bwd_parts(rows, cols, TG_F16, sms);
  return static_cast<int64_t>(a > b ? a : b) * 2 * part_cols(cols, true) * 4;
}

cudaError_t launch_norm_bwd(const NormBwdLaunch& l, cudaStream_t stream) {
  const uint32_t parts = norm_bwd_parts(l.rows, l.cols, l.dtype, l.sms);
  const bool sums = l.dgamma != nullptr || l.dbeta != nullptr;
  uint32_t first = 0, apart = 0;   // kOneLead: of the rows
  uint32_t columns = part_cols(l.cols, false);
  auto params = [&](size_t elem) {
    NormBwdParams p;
    p.dy = rows_of(l.dy, l.rows, l.cols, l.ld_dy, elem);
    p.dx = rows_of(l.dx, l.rows, l.cols, l.ld_dx, elem);
    p.x = rows_of(l.x, l.rows, l.cols, l.x ? l.ld_x : 0, elem);
    p.q = static_cast<const uint8_t*>(l.q);
    p.s = static_cast<const uint8_t*>(l.s);
    p.gamma = l.gamma;
    p.wide_params = wide(l.gamma) ? 1u : 0u;
    p.mean = l.mean;
    p.rstd = l.rstd;
    p.partials = sums ? l.partials : nullptr;
    p.part_cols = part_cols(l.cols, false);
    p.rows = static_cast<uint32_t>(l.rows);
    p.cols = static_cast<uint32_t>(l.cols);
    p.blocks = round_up(l.cols, kCkptBlock) / kCkptBlock;
    return p;
  };
  auto run_short = [&](auto tx, auto tp, auto kept) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    const NormBwdParams p = params(sizeof(TX));
    const uint32_t shift = short_shift<TX>(l.cols), per_warp = 32u >> shift;
    // ``parts`` CTAs, each of as many warps (a power of two) as have rows
    const int64_t turns = (l.rows + per_warp - 1) / per_warp;
    uint32_t threads = 32;
    while (threads < kShortBwdThreads && int64_t(threads / 32) * parts < turns) threads *= 2;
    return with_access<TX>(l.cols, p.dy, p.dx, p.x, [&](auto access) {
      return launch_pdl(
          norm_bwd_short_kernel<TX, TP, decltype(kept)::value, decltype(access)::value>,
          dim3(parts), threads, 0, stream, p, shift);
    });
  };
  auto rows_pass = [&](auto tx, auto tp, auto unal, auto kept) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    constexpr bool UNAL = decltype(unal)::value, KEPT = decltype(kept)::value;
    NormBwdParams p = params(sizeof(TX));
    auto grouped = [&](auto n) -> cudaError_t {
      constexpr int kThreads = decltype(n)::value, kRows = UNAL ? kAnyRows : kWholeRows;
      const NormGrid g = norm_grid(l.rows, l.cols, kNormValues, kThreads, l.sms);
      const uint32_t threads = g.groups * g.g_threads;
      const size_t smem = norm_bwd_smem<TX, kThreads>(threads / 32);
      constexpr auto kernel = norm_bwd_kernel<TX, TP, kRows, KEPT, kThreads>;
      cudaError_t e = allow_smem<kernel>(smem);
      if (e != cudaSuccess) return e;
      return launch_pdl(kernel, dim3(g.ctas), threads, smem, stream, p, g.g_threads);
    };
    if constexpr (UNAL && !KEPT)
      if (l.cols + kVec<TX> - 1 <= kNormCols && one_lead(p.dy, p.x) && one_lead(p.dy, p.dx) &&
          (l.rows <= l.sms || l.sms % 8 == 0)) {
        first = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.dy.base) % 16);
        apart = static_cast<uint32_t>(p.dy.pitch % 16);
        p.part_cols = columns = part_cols(l.cols, true);
        const NormGrid g =
            norm_grid(l.rows, l.cols + kVec<TX> - 1, kNormValues, kNormThreads, l.sms);
        const uint32_t threads = g.groups * g.g_threads;
        const size_t smem = norm_bwd_smem<TX, kNormThreads>(threads / 32);
        constexpr auto kernel = norm_bwd_kernel<TX, TP, kOneLead, KEPT, kNormThreads>;
        cudaError_t e = allow_smem<kernel>(smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(g.ctas), threads, smem, stream, p, g.g_threads);
      }
    if (l.cols <= kNormCols) return grouped(std::integral_constant<int, kNormThreads>());
    if constexpr (sizeof(TX) == 2)
      if (l.cols <= kNormWideCols)
        return grouped(std::integral_constant<int, kNormWideThreads>());
    cudaError_t e = launch_pdl(norm_bwd_long_kernel<TX, TP, UNAL, KEPT>,
                               dim3(static_cast<uint32_t>(l.rows)), 1024, 0, stream, p);
    if (e != cudaSuccess || !sums) return e;
    constexpr uint32_t kCols = 128 * kVec<TX>;
    return launch_pdl(norm_bwd_cols_kernel<TX, UNAL, KEPT>,
                      dim3(round_up(l.cols, kCols) / kCols, parts), 128, 0, stream, p);
  };
  return with_types(l.dtype, l.param_dtype, [&](auto tx, auto tp) -> cudaError_t {
    using TP = typename decltype(tp)::type;
    constexpr uint32_t kElem = sizeof(typename decltype(tx)::type);
    const bool unal = l.cols * kElem % 16 != 0 || !rows_aligned(l.dy, l.ld_dy, kElem) ||
                      !rows_aligned(l.dx, l.ld_dx, kElem) || !rows_aligned(l.x, l.ld_x, kElem);
    cudaError_t e = cudaSuccess;
    if (l.rows > 0) {
      if (l.cols * kElem <= kShortBytes)
        e = l.x ? run_short(tx, tp, std::false_type()) : run_short(tx, tp, std::true_type());
      else if (l.x)
        e = unal ? rows_pass(tx, tp, std::true_type(), std::false_type())
                 : rows_pass(tx, tp, std::false_type(), std::false_type());
      else
        e = unal ? rows_pass(tx, tp, std::true_type(), std::true_type())
                 : rows_pass(tx, tp, std::false_type(), std::true_type());
    }
    if (e != cudaSuccess || !sums) return e;
    const dim3 grid(round_up(l.cols, 32) / 32, 2);
    return launch_pdl(norm_bwd_join_kernel<TP>, grid, 256, 0, stream,
                      static_cast<const float*>(l.partials), parts, columns,
                      static_cast<uint32_t>(l.cols), first, apart, kElem == 4 ? 2u : 1u,
                      static_cast<TP*>(l.dgamma), static_cast<TP*>(l.dbeta));
  });
}

// ---------------------------------------------------------------- 8-bit checkpoints
namespace {

template <typename TX, bool UNAL, bool PACK>
cudaError_t ckpt8_run(char* x, uint8_t* q, uint8_t* s, int64_t rows, int64_t cols, int64_t ld,
                      int sms, cudaStream_t stream) {
  constexpr int kN = kVec<TX>;
  Ckpt8Params p;
  p.cols = static_cast<uint32_t>(cols);
  p.blocks = round_up(cols, kCkptBlock) / kCkptBlock;
  p.per_row = UNAL ? round_up(cols, 32 * kN) / kN : p.blocks * (kCkptBlock / kN);
  p.div_shift = 0;
  while ((uint64_t(1) << p.div_shift) < p.per_row) ++p.div_shift;
  p.div_mul = static_cast<uint32_t>(
      ((uint64_t(1) << 32) * ((uint64_t(1) << p.div_shift) - p.per_row)) / p.per_row + 1);
  // rows of one launch: its units are numbered in 31 bits
  const int64_t most = (int64_t(1) << 30) / p.per_row, chunk = most < 1 ? 1 : most;
  for (int64_t r = 0; r < rows; r += chunk) {
    const int64_t n = rows - r < chunk ? rows - r : chunk;
    const int64_t elem = sizeof(TX);
    p.x = rows_of(x + r * ld * elem, n, cols, ld, sizeof(TX));
    p.q = q + r * p.blocks * kCkptBlock;
    p.s = s + r * p.blocks;
    p.units = static_cast<uint32_t>(n * p.per_row);
    const uint64_t want = (static_cast<uint64_t>(p.units) + 255) / 256;
    // 64 blocks an SM: blocks that end while others load (8192 x 8192 bf16 pack 41.6 us; 43.6 with
    // 8, a single wave; 47.8 with a block for every 512 units)
    const uint64_t cap = static_cast<uint64_t>(sms) * 64;
    const cudaError_t e =
        launch_pdl(ckpt8_kernel<TX, UNAL, PACK>, dim3(static_cast<uint32_t>(want < cap ? want : cap)),
                   256, 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool PACK>
cudaError_t ckpt8_any(void* x, void* q, void* s, int64_t rows, int64_t cols, int64_t ld, int dtype,
                      int sms, cudaStream_t stream) {
  return with_type(dtype, [&](auto tx) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    char* src = static_cast<char*>(x);
    uint8_t *q8 = static_cast<uint8_t*>(q), *s8 = static_cast<uint8_t*>(s);
    return rows_aligned(x, ld, sizeof(TX))
               ? ckpt8_run<TX, false, PACK>(src, q8, s8, rows, cols, ld, sms, stream)
               : ckpt8_run<TX, true, PACK>(src, q8, s8, rows, cols, ld, sms, stream);
  });
}

}  // namespace

cudaError_t launch_ckpt8_pack(const void* x, void* q, void* s, int64_t rows, int64_t cols,
                              int64_t ld_x, int dtype, int sms, cudaStream_t stream) {
  return ckpt8_any<true>(const_cast<void*>(x), q, s, rows, cols, ld_x, dtype, sms, stream);
}

cudaError_t launch_ckpt8_unpack(const void* q, const void* s, void* out, int64_t rows, int64_t cols,
                                int64_t ld_out, int dtype, int sms, cudaStream_t stream) {
  return ckpt8_any<false>(out, const_cast<void*>(q), const_cast<void*>(s), rows, cols, ld_out,
                          dtype, sms, stream);
}

}  // namespace tg
