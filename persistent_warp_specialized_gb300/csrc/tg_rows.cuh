// tg_rows.cuh -- what the row-wise kernels (layer norm, 8-bit checkpoints) share: loads and stores
// of a few neighbouring values of a row, the E4M3 / E8M0 conversions of a checkpoint, and sums over
// a warp.
//
// A checkpoint of x [rows, cols] is q [rows, 32 ceil(cols / 32)] E4M3 bytes (zero past ``cols``) and
// s [rows, ceil(cols / 32)] E8M0 bytes; it stands for q * 2^(s - 127).  The scale of 32 values is
// 2^(floor(log2 amax) - 8), 8 being E4M3's largest exponent, with amax over the block's finite
// values and the exponent clamped to [-127, 127]; the quotient is rounded to nearest even and
// saturates at 448.  NaN and infinities are kept as NaN (E4M3 has no infinity, and 448 would hide
// an overflow).  Where cols is a multiple of 32 this is the row-major operand that
// tg_mxfp8_pack_scales and tg_gemm_mxfp8 take.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "tg_ptx.cuh"

namespace tg {

constexpr int kCkptBlock = 32;   // values per scale

// ---------------------------------------------------------------- element types
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// VE values of T as they lie in memory, moved by the widest loads their size allows.
template <typename T, int VE>
struct alignas(sizeof(T) * VE <= 16 ? sizeof(T) * VE : 16) Raw {
  T v[VE];
};

template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, VE>*>(p);
}

// The first ``n`` of VE values (the others are zero); one wide load when all of them are there.
// ``n`` may be negative.
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> load_some(const T* p, int64_t n) {
  if (n >= VE) return load_raw<T, VE>(p);
  Raw<T, VE> r;
#pragma unroll
  for (int i = 0; i < VE; ++i) r.v[i] = i < n ? p[i] : from_f32<T>(0.0f);
  return r;
}

template <typename T, int VE>
__device__ __forceinline__ void store_some(T* p, const Raw<T, VE>& r, int64_t n) {
  if (n >= VE) {
    *reinterpret_cast<Raw<T, VE>*>(p) = r;
    return;
  }
#pragma unroll
  for (int i = 0; i < VE; ++i)
    if (i < n) p[i] = r.v[i];
}

// ---------------------------------------------------------------- sums over a warp
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- E4M3 and E8M0
// Scale byte of a block whose largest finite magnitude is ``amax``: the float's exponent field is
// floor(log2 amax) + 127, so the byte is that field minus 8, at least 0 (zeros and subnormals).
__device__ __forceinline__ uint32_t ckpt8_scale_byte(float amax) {
  const uint32_t e = __float_as_uint(amax) >> 23;
  return e > 8u ? e - 8u : 0u;
}

// 2^(127 - byte), the exact reciprocal of the scale; byte <= 246 for every finite amax, so the
// result is a normal number.
__device__ __forceinline__ float ckpt8_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127): the smallest is a subnormal float, and 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// two floats -> E4M3, round to nearest even, saturating; ``lo`` in the low byte.  NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// two E4M3 bytes -> two floats (exact; by way of fp16, which holds every E4M3 value)
__device__ __forceinline__ float2 e4m3x2_value(uint32_t bytes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// VE values of a checkpoint's row as they lie in memory: E4M3 bytes and their scale byte.
template <int VE>
struct Kept {
  Raw<uint8_t, VE> q;
  uint32_t s;
};

template <int VE>
__device__ __forceinline__ void kept_values(const Kept<VE>& k, float (&v)[VE]) {
  const float scale = e8m0_value(k.s);
  if constexpr (VE == 1) {
    v[0] = e4m3x2_value(k.q.v[0]).x * scale;
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 2) {
      const float2 f = e4m3x2_value(k.q.v[i] | static_cast<uint32_t>(k.q.v[i + 1]) << 8);
      v[i] = f.x * scale;
      v[i + 1] = f.y * scale;
    }
  }
}

// Quantises one block of 32 values held by 32 / VE neighbouring lanes, VE each (values past the
// row's end are zero); every lane of the warp calls it.  Returns the scale byte, and the bytes of
// this lane's values in ``q``.
template <int VE>
__device__ __forceinline__ uint32_t ckpt8_quantise(const float (&v)[VE], Raw<uint8_t, VE>& q) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < VE; ++i) amax = fmaxf(amax, fabsf(v[i]));   // fmaxf passes over NaN
#pragma unroll
  for (int o = 1; o < kCkptBlock / VE; o <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float u[VE];
#pragma unroll
  for (int i = 0; i < VE; ++i) u[i] = v[i];
  if (__any_sync(0xffffffffu, amax == INFINITY)) {   // rare: infinities become NaN, amax is redone
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
      if (fabsf(u[i]) == INFINITY) u[i] = __uint_as_float(0x7fffffffu);
      amax = fmaxf(amax, fabsf(u[i]));
    }
#pragma unroll
    for (int o = 1; o < kCkptBlock / VE; o <<= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  const uint32_t s = ckpt8_scale_byte(amax);
  const float inv = ckpt8_inverse(s);
  if constexpr (VE == 1) {
    q.v[0] = static_cast<uint8_t>(e4m3x2(u[0] * inv, 0.0f));
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 2) {
      const uint32_t b = e4m3x2(u[i] * inv, u[i + 1] * inv);
      q.v[i] = static_cast<uint8_t>(b);
      q.v[i + 1] = static_cast<uint8_t>(b >> 8);
    }
  }
  return s;
}

}  // namespace tg
