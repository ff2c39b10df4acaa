// tg_train.cu -- instantiations and launchers of the operators around the GEMM in training: layer
// norm forward and backward, and activation checkpoints in 8 bits.
#include <type_traits>

#include "../../include/tg.h"
#include "tg_ckpt8_kernel.cuh"
#include "tg_internal.h"
#include "tg_launch.cuh"
#include "tg_norm_kernel.cuh"

namespace tg {

namespace {

bool aligned(const void* p, uint64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

uint32_t round_up(uint64_t n, uint32_t to) { return static_cast<uint32_t>((n + to - 1) / to * to); }

// A row (or a whole parameter vector: ld 0) can be read in 16-byte vectors of its type.
bool rows_aligned(const void* p, int64_t ld, uint32_t elem) {
  return aligned(p, 16) && static_cast<uint64_t>(ld) * elem % 16 == 0;
}

// Names a type (or a number) as an argument of a generic lambda.
template <typename T>
struct Of {
  using type = T;
};
template <int N>
using Num = std::integral_constant<int, N>;

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

// ---------------------------------------------------------------- layer norm, forward
constexpr int64_t kWarpRowCols = 1024;    // a row held by one warp, 32 values a lane
constexpr int64_t kCtaRowCols = 16384;    // a row held by one CTA, 16 values a thread

template <typename TX, typename TP, int VE, bool KEEP>
cudaError_t norm_fwd_ve(const NormLaunch& l, const NormFwdParams& p, cudaStream_t stream) {
  if (l.cols <= kWarpRowCols) {
    const dim3 grid(static_cast<uint32_t>((l.rows + 3) / 4));
    if (l.cols <= 256)
      return launch_pdl(norm_fwd_kernel<TX, TP, VE, 8 / VE, true, KEEP>, grid, 128, 0, stream, p);
    return launch_pdl(norm_fwd_kernel<TX, TP, VE, 32 / VE, true, KEEP>, grid, 128, 0, stream, p);
  }
  const dim3 grid(static_cast<uint32_t>(l.rows));
  if (l.cols <= kCtaRowCols)
    return launch_pdl(norm_fwd_kernel<TX, TP, VE, 16 / VE, false, KEEP>, grid,
                      round_up((l.cols + 15) / 16, 32), 0, stream, p);
  return launch_pdl(norm_fwd_long_kernel<TX, TP, VE, KEEP>, grid, 1024, 0, stream, p);
}

// ---------------------------------------------------------------- layer norm, backward
constexpr int64_t kBwdGroupCols = 8192;   // 16 columns a thread, 512 threads
constexpr uint32_t kBwdThreads = 512;
constexpr uint32_t kBwdLongParts = 64;

uint32_t bwd_group_threads(int64_t cols) { return round_up((cols + 15) / 16, 32); }

}  // namespace

cudaError_t launch_norm_fwd(const NormLaunch& l, cudaStream_t stream) {
  NormFwdParams p;
  p.x = l.x;
  p.gamma = l.gamma;
  p.beta = l.beta;
  p.y = l.y;
  p.mean = l.mean;
  p.rstd = l.rstd;
  p.q = static_cast<uint8_t*>(l.q);
  p.s = static_cast<uint8_t*>(l.s);
  p.rows = static_cast<uint32_t>(l.rows);
  p.cols = static_cast<uint32_t>(l.cols);
  p.blocks = round_up(l.cols, kCkptBlock) / kCkptBlock;
  p.ld_x = l.ld_x;
  p.ld_y = l.ld_y;
  p.eps = l.eps;
  return with_types(l.dtype, l.param_dtype, [&](auto tx, auto tp) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    constexpr int kVec = 16 / sizeof(TX);
    const bool vec = rows_aligned(l.x, l.ld_x, sizeof(TX)) &&
                     rows_aligned(l.y, l.ld_y, sizeof(TX)) && aligned(l.gamma, 16) &&
                     aligned(l.beta, 16);
    if (vec)
      return l.q ? norm_fwd_ve<TX, TP, kVec, true>(l, p, stream)
                 : norm_fwd_ve<TX, TP, kVec, false>(l, p, stream);
    return l.q ? norm_fwd_ve<TX, TP, 1, true>(l, p, stream)
               : norm_fwd_ve<TX, TP, 1, false>(l, p, stream);
  });
}

uint32_t norm_bwd_parts(int64_t rows, int64_t cols, int sms) {
  if (rows == 0) return 0;
  if (cols > kBwdGroupCols)
    return static_cast<uint32_t>(rows < kBwdLongParts ? rows : kBwdLongParts);
  const uint32_t groups = kBwdThreads / bwd_group_threads(cols);
  const int64_t ctas = (rows + groups - 1) / groups;
  return static_cast<uint32_t>(ctas < sms ? ctas : sms);
}

cudaError_t launch_norm_bwd(const NormBwdLaunch& l, cudaStream_t stream) {
  const uint32_t parts = norm_bwd_parts(l.rows, l.cols, l.sms);
  const bool sums = l.dgamma != nullptr || l.dbeta != nullptr;
  NormBwdParams p;
  p.dy = l.dy;
  p.x = l.x;
  p.q = static_cast<const uint8_t*>(l.q);
  p.s = static_cast<const uint8_t*>(l.s);
  p.gamma = l.gamma;
  p.mean = l.mean;
  p.rstd = l.rstd;
  p.dx = l.dx;
  p.partials = sums ? l.partials : nullptr;
  p.rows = static_cast<uint32_t>(l.rows);
  p.cols = static_cast<uint32_t>(l.cols);
  p.blocks = round_up(l.cols, kCkptBlock) / kCkptBlock;
  p.ld_dy = l.ld_dy;
  p.ld_x = l.ld_x;
  p.ld_dx = l.ld_dx;
  auto rows_pass = [&](auto tx, auto tp, auto ve, auto kept) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    constexpr int VE = decltype(ve)::value;
    constexpr bool KEPT = decltype(kept)::value;
    if (l.cols <= kBwdGroupCols) {
      const uint32_t g = bwd_group_threads(l.cols), groups = kBwdThreads / g;
      const size_t smem = groups > 1 ? 2 * sizeof(float) * static_cast<size_t>(l.cols) : 0;
      return launch_pdl(norm_bwd_kernel<TX, TP, VE, 16 / VE, KEPT>, dim3(parts), groups * g, smem,
                        stream, p, g);
    }
    cudaError_t e = launch_pdl(norm_bwd_long_kernel<TX, TP, VE, KEPT>,
                               dim3(static_cast<uint32_t>(l.rows)), 1024, 0, stream, p);
    if (e != cudaSuccess || !sums) return e;
    const dim3 grid(round_up(l.cols, 128 * VE) / (128 * VE), parts);
    return launch_pdl(norm_bwd_cols_kernel<TX, VE, KEPT>, grid, 128, 0, stream, p);
  };
  return with_types(l.dtype, l.param_dtype, [&](auto tx, auto tp) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    using TP = typename decltype(tp)::type;
    constexpr int kVec = 16 / sizeof(TX);
    const bool vec = rows_aligned(l.dy, l.ld_dy, sizeof(TX)) &&
                     rows_aligned(l.dx, l.ld_dx, sizeof(TX)) && aligned(l.gamma, 16) &&
                     (l.x == nullptr || rows_aligned(l.x, l.ld_x, sizeof(TX)));
    cudaError_t e = cudaSuccess;
    if (l.rows > 0) {
      if (l.x)
        e = vec ? rows_pass(tx, tp, Num<kVec>(), std::false_type())
                : rows_pass(tx, tp, Num<1>(), std::false_type());
      else
        e = vec ? rows_pass(tx, tp, Num<kVec>(), std::true_type())
                : rows_pass(tx, tp, Num<1>(), std::true_type());
    }
    if (e != cudaSuccess || !sums) return e;
    const dim3 grid(round_up(l.cols, 32) / 32, 2);
    return launch_pdl(norm_bwd_join_kernel<TP>, grid, 256, 0, stream,
                      static_cast<const float*>(l.partials), parts, p.cols,
                      static_cast<TP*>(l.dgamma), static_cast<TP*>(l.dbeta));
  });
}

// ---------------------------------------------------------------- 8-bit checkpoints
namespace {

// Rows in one launch, so that its units fit in 31 bits.
int64_t rows_per_launch(int64_t blocks, int per) {
  const int64_t most = (int64_t(1) << 30) / (blocks * per);
  return most < 1 ? 1 : most;
}

uint32_t ckpt8_grid(uint64_t units, int sms) {
  const uint64_t want = (units + 255) / 256, most = static_cast<uint64_t>(sms) * 32;
  return static_cast<uint32_t>(want < most ? want : most);
}

template <typename TX, int VE, bool PACK>
cudaError_t ckpt8_run(void* x, uint8_t* q, uint8_t* s, int64_t rows, int64_t cols, int64_t ld,
                      int sms, cudaStream_t stream) {
  Ckpt8Params p;
  p.cols = static_cast<uint32_t>(cols);
  p.blocks = round_up(cols, kCkptBlock) / kCkptBlock;
  p.ld = ld;
  constexpr int kPer = kCkptBlock / VE;
  const int64_t chunk = rows_per_launch(p.blocks, kPer);
  for (int64_t r = 0; r < rows; r += chunk) {
    const int64_t n = rows - r < chunk ? rows - r : chunk;
    TX* at = static_cast<TX*>(x) + r * ld;
    p.src = at;
    p.dst = at;
    p.q = q + r * p.blocks * kCkptBlock;
    p.s = s + r * p.blocks;
    p.units = static_cast<uint32_t>(n * p.blocks * kPer);
    cudaError_t e;
    if constexpr (PACK)
      e = launch_pdl(ckpt8_pack_kernel<TX, VE>, dim3(ckpt8_grid(p.units, sms)), 256, 0, stream, p);
    else
      e = launch_pdl(ckpt8_unpack_kernel<TX, VE>, dim3(ckpt8_grid(p.units, sms)), 256, 0, stream,
                     p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_ckpt8_pack(const void* x, void* q, void* s, int64_t rows, int64_t cols,
                              int64_t ld_x, int dtype, int sms, cudaStream_t stream) {
  return with_type(dtype, [&](auto tx) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    constexpr int kVec = 16 / sizeof(TX);
    void* src = const_cast<void*>(x);
    uint8_t *q8 = static_cast<uint8_t*>(q), *s8 = static_cast<uint8_t*>(s);
    return rows_aligned(x, ld_x, sizeof(TX))
               ? ckpt8_run<TX, kVec, true>(src, q8, s8, rows, cols, ld_x, sms, stream)
               : ckpt8_run<TX, 1, true>(src, q8, s8, rows, cols, ld_x, sms, stream);
  });
}

cudaError_t launch_ckpt8_unpack(const void* q, const void* s, void* out, int64_t rows, int64_t cols,
                                int64_t ld_out, int dtype, int sms, cudaStream_t stream) {
  return with_type(dtype, [&](auto tx) -> cudaError_t {
    using TX = typename decltype(tx)::type;
    constexpr int kVec = 16 / sizeof(TX);
    uint8_t* q8 = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
    uint8_t* s8 = const_cast<uint8_t*>(static_cast<const uint8_t*>(s));
    return rows_aligned(out, ld_out, sizeof(TX))
               ? ckpt8_run<TX, kVec, false>(out, q8, s8, rows, cols, ld_out, sms, stream)
               : ckpt8_run<TX, 1, false>(out, q8, s8, rows, cols, ld_out, sms, stream);
  });
}

}  // namespace tg
