// tg_ckpt8_kernel.cuh -- activation checkpoints in 8 bits: pack and unpack (format: tg_rows.cuh).
//
// Both are one pass over memory and are bound by it: a 16-bit value is read (2 bytes) and 1 + 1/32
// bytes are written, or the other way round.  A block of 32 values belongs to 32 / VE neighbouring
// lanes, VE values each, so its amax takes log2(32 / VE) shuffles; units of VE values are numbered
// over all rows, so short rows fill warps as well as long ones.
#pragma once

#include "tg_rows.cuh"

namespace tg {

struct Ckpt8Params {
  const void* src;       // pack: x; unpack: unused
  void* dst;             // unpack: out; pack: unused
  uint8_t* q;
  uint8_t* s;
  uint32_t cols, blocks; // blocks = ceil(cols / 32)
  int64_t ld;            // row stride of src / dst in elements
  uint32_t units;        // rows * blocks * (32 / VE), < 2^31
};

template <typename T, int VE>
__global__ void __launch_bounds__(256) ckpt8_pack_kernel(const Ckpt8Params p) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr uint32_t kPer = kCkptBlock / VE;            // units per block of 32 values
  const uint32_t stride = gridDim.x * blockDim.x;       // a multiple of 32
  const uint32_t end = (p.units + 31u) & ~31u;          // whole warps, for the shuffles
  for (uint32_t u = blockIdx.x * blockDim.x + threadIdx.x; u < end; u += stride) {
    const bool in = u < p.units;
    const uint32_t b = u / kPer;                        // block number over all rows
    const uint32_t row = b / p.blocks, j = b - row * p.blocks;
    const uint32_t col = j * kCkptBlock + (u % kPer) * VE;
    const T* src = static_cast<const T*>(p.src) + static_cast<int64_t>(row) * p.ld + col;
    const Raw<T, VE> r =
        load_some<T, VE>(src, in ? static_cast<int64_t>(p.cols) - col : 0);
    float v[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) v[i] = to_f32(r.v[i]);
    Raw<uint8_t, VE> q;
    const uint32_t s = ckpt8_quantise<VE>(v, q);
    if (in) {
      *reinterpret_cast<Raw<uint8_t, VE>*>(p.q + static_cast<uint64_t>(u) * VE) = q;
      if (u % kPer == 0) p.s[b] = static_cast<uint8_t>(s);
    }
  }
}

template <typename T, int VE>
__global__ void __launch_bounds__(256) ckpt8_unpack_kernel(const Ckpt8Params p) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr uint32_t kPer = kCkptBlock / VE;
  const uint32_t stride = gridDim.x * blockDim.x;
  for (uint32_t u = blockIdx.x * blockDim.x + threadIdx.x; u < p.units; u += stride) {
    const uint32_t b = u / kPer;
    const uint32_t row = b / p.blocks, j = b - row * p.blocks;
    const uint32_t col = j * kCkptBlock + (u % kPer) * VE;
    Kept<VE> k;
    k.q = load_raw<uint8_t, VE>(p.q + static_cast<uint64_t>(u) * VE);
    k.s = p.s[b];
    float v[VE];
    kept_values<VE>(k, v);
    Raw<T, VE> r;
#pragma unroll
    for (int i = 0; i < VE; ++i) r.v[i] = from_f32<T>(v[i]);
    store_some<T, VE>(static_cast<T*>(p.dst) + static_cast<int64_t>(row) * p.ld + col, r,
                      static_cast<int64_t>(p.cols) - col);
  }
}

}  // namespace tg
