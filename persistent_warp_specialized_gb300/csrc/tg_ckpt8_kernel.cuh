// tg_ckpt8_kernel.cuh -- activation checkpoints in 8 bits: pack and unpack (format: tg_rows.cuh).
//
// Both are one pass over memory and are bound by it: a 16-bit value is read (2 bytes) and 1 + 1/32
// bytes are written, or the other way round.  A block of 32 values belongs to 32 / N neighbouring
// lanes, N = 16 / size values each, so its amax takes log2(32 / N) shuffles.
//
// Rows that start on 16-byte boundaries: units of N values are numbered over all rows, so short rows
// fill warps as well as long ones.  Other rows: a warp takes strips of 32 N values of one row, and
// shifts its vectors out of the granules they lie in (tg_rows.cuh).
#pragma once

#include "tg_rows.cuh"

namespace tg {

struct Ckpt8Params {
  RowsOf x;              // pack: the source; unpack: the destination
  uint8_t* q;
  uint8_t* s;
  uint32_t cols, blocks; // blocks = ceil(cols / 32)
  uint32_t units;        // of N values, numbered over all rows (strips * 32 a row with UNAL), < 2^31
  uint32_t per_row;      // units in a row
  uint32_t div_mul, div_shift;   // u / per_row = (umulhi(u, div_mul) + u) >> div_shift, u < 2^31
};

constexpr int kCkptUnroll = 2;   // units in flight per thread

template <typename T, bool UNAL, bool PACK>
__global__ void __launch_bounds__(256) ckpt8_kernel(const Ckpt8Params p) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kN = kVec<T>;
  constexpr uint32_t kPer = kCkptBlock / kN;            // units per block of 32 values
  const uint32_t stride = gridDim.x * blockDim.x;       // a multiple of 32
  const uint32_t end = (p.units + 31u) & ~31u;          // whole warps, for the shuffles
  const int64_t row_bytes = static_cast<int64_t>(p.cols) * static_cast<int>(sizeof(T));
  for (uint32_t u0 = blockIdx.x * blockDim.x + threadIdx.x; u0 < end;
       u0 += kCkptUnroll * stride) {
    V16 r[kCkptUnroll];                                 // pack: values; unpack: bytes and scale
    uint32_t row[kCkptUnroll], v[kCkptUnroll];
#pragma unroll
    for (int k = 0; k < kCkptUnroll; ++k) {
      const uint32_t u = u0 + k * stride;
      r[k] = V16{{0u, 0u, 0u, 0u}};
      if (u >= end) continue;
      row[k] = (__umulhi(u, p.div_mul) + u) >> p.div_shift;
      v[k] = u - row[k] * p.per_row;
      const char* at = p.x.base + static_cast<int64_t>(row[k]) * p.x.pitch;
      if constexpr (PACK) {
        r[k] = load_vector<T, UNAL>(p.x, at, u < p.units ? 16 * static_cast<int64_t>(v[k]) : row_bytes,
                                    u < p.units ? row_bytes : 0);
      } else if (u < p.units && v[k] / kPer < p.blocks) {
        const uint64_t b = static_cast<uint64_t>(row[k]) * p.blocks + v[k] / kPer;
        uint32_t q[kN / 4];
        load_kept<kN>(p.q + b * kCkptBlock + (v[k] % kPer) * kN, q);
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) r[k].w[i] = q[i];
        r[k].w[2] = p.s[b];
      }
    }
#pragma unroll
    for (int k = 0; k < kCkptUnroll; ++k) {
      const uint32_t u = u0 + k * stride;
      if (u >= end) break;
      const int left = u < p.units ? values_left<kN>(v[k], p.cols) : 0;
      float f[kN];
      if constexpr (PACK) {
        values<T>(r[k], f);
        if (left < kN) {
#pragma unroll
          for (int i = 0; i < kN; ++i) f[i] = i < left ? f[i] : 0.0f;
        }
        uint32_t q[kN / 4];
        const uint32_t s = ckpt8_quantise<kN>(f, q);
        if (u < p.units && v[k] / kPer < p.blocks) {
          const uint64_t b = static_cast<uint64_t>(row[k]) * p.blocks + v[k] / kPer;
          store_kept<kN>(p.q + b * kCkptBlock + (v[k] % kPer) * kN, q);
          if (v[k] % kPer == 0) p.s[b] = static_cast<uint8_t>(s);
        }
      } else {
        kept_values<kN>(r[k].w, r[k].w[2], f);
        store_vector<T, UNAL>(p.x.base + static_cast<int64_t>(row[k]) * p.x.pitch,
                              16 * static_cast<int64_t>(v[k]), rounded<T>(f), left);
      }
    }
  }
}

}  // namespace tg
