// tg_rows.cuh -- what the row-wise kernels (layer norm, 8-bit checkpoints) share: 16-byte accesses
// to rows of any alignment, the E4M3 / E8M0 conversions of a checkpoint, and sums over a warp.
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
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // values in 16 bytes

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

// 16 bytes of a row: kVec<T> values, the first in the low end of w[0].
struct alignas(16) V16 {
  uint32_t w[4];
};

// in one access, 16-byte aligned (as uint4: of the struct the compiler may make four)
__device__ __forceinline__ V16 load16(const void* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  return V16{{u.x, u.y, u.z, u.w}};
}
__device__ __forceinline__ void store16(void* p, const V16& r) {
  *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

__device__ __forceinline__ void values_of(const V16& r, float (&v)[4], float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void values_of(const V16& r, float (&v)[8], __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void values_of(const V16& r, float (&v)[8], __half) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void values(const V16& r, float (&v)[kVec<T>]) {
  values_of(r, v, T());
}

__device__ __forceinline__ V16 rounded_of(const float (&v)[4], float) {
  V16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(v[i]);
  return r;
}
__device__ __forceinline__ V16 rounded_of(const float (&v)[8], __nv_bfloat16) {
  V16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}
__device__ __forceinline__ V16 rounded_of(const float (&v)[8], __half) {
  V16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return r;
}
// the values rounded to T
template <typename T>
__device__ __forceinline__ V16 rounded(const float (&v)[kVec<T>]) {
  return rounded_of(v, T());
}

// ---------------------------------------------------------------- rows of any alignment
// A matrix's bytes, from its first value to past its last; ``pitch`` bytes between rows.
struct RowsOf {
  char* base;
  char* end;
  int64_t pitch;
};

// A row starts ``lead`` bytes into a 16-byte granule.  A warp takes 32 neighbouring vectors of 16
// bytes from it (a strip); with lead != 0 vector j lies in granules j and j + 1, so a strip needs 33
// granules, all read as they lie, and each lane shifts its vector out of two of them.  UNAL: some
// row has a lead, or rows are not whole vectors; without it every vector is a granule in the row, or
// past its end.

// Value i of the 16 bytes (i a constant), stored alone.
template <typename T>
__device__ __forceinline__ void store_one(char* p, const V16& r, int i) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<uint32_t*>(p + 4 * i) = r.w[i];
  else
    *reinterpret_cast<uint16_t*>(p + 2 * i) =
        static_cast<uint16_t>(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
}

// The 16 bytes at ``p`` (16-byte aligned); bytes outside [from, to) are not touched and read as
// zero.  For the granules at a matrix's ends.
template <typename T>
__device__ __forceinline__ V16 load_granule(const char* p, const char* from, const char* to) {
  if (p >= from && p + 16 <= to) return load16(p);
  V16 r = {{0u, 0u, 0u, 0u}};
#pragma unroll
  for (int i = 0; i < kVec<T>; ++i) {
    const char* q = p + i * static_cast<int>(sizeof(T));
    if (q < from || q >= to) continue;
    if constexpr (sizeof(T) == 4)
      r.w[i] = *reinterpret_cast<const uint32_t*>(q);
    else
      r.w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(q)) << (16 * (i & 1));
  }
  return r;
}

// 16 bytes from byte ``lead`` (a multiple of the value's size, below 16; the same in every lane) of
// a and b put together: one of four word offsets, then a shift by half a word.
template <typename T>
__device__ __forceinline__ V16 window(const V16& a, const V16& b, uint32_t lead) {
  const uint32_t bits = sizeof(T) == 4 ? 0u : (lead & 2u) * 8u;
  V16 r;
  switch (lead >> 2) {
    case 0:
      r = V16{{__funnelshift_r(a.w[0], a.w[1], bits), __funnelshift_r(a.w[1], a.w[2], bits),
               __funnelshift_r(a.w[2], a.w[3], bits), __funnelshift_r(a.w[3], b.w[0], bits)}};
      break;
    case 1:
      r = V16{{__funnelshift_r(a.w[1], a.w[2], bits), __funnelshift_r(a.w[2], a.w[3], bits),
               __funnelshift_r(a.w[3], b.w[0], bits), __funnelshift_r(b.w[0], b.w[1], bits)}};
      break;
    case 2:
      r = V16{{__funnelshift_r(a.w[2], a.w[3], bits), __funnelshift_r(a.w[3], b.w[0], bits),
               __funnelshift_r(b.w[0], b.w[1], bits), __funnelshift_r(b.w[1], b.w[2], bits)}};
      break;
    default:
      r = V16{{__funnelshift_r(a.w[3], b.w[0], bits), __funnelshift_r(b.w[0], b.w[1], bits),
               __funnelshift_r(b.w[1], b.w[2], bits), __funnelshift_r(b.w[2], b.w[3], bits)}};
  }
  return r;
}

// How many of a row's values there are from vector ``v`` of N on, as far as N: negative where the
// row ended before the vector, at least -N.
template <int N>
__device__ __forceinline__ int values_left(uint32_t v, uint32_t cols) {
  const int64_t n = static_cast<int64_t>(cols) - static_cast<int64_t>(v) * N;
  return n >= N ? N : (n <= -N ? -N : static_cast<int>(n));
}

__device__ __forceinline__ uint32_t lead_of(const char* row) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
}

// The lane's vector of a strip, straight from memory (every lane calls it).  ``row``: the row's
// first byte, ``at``: the vector's byte offset in it.  Values past the row's end are what lies
// there (or zero): the caller masks them.
template <typename T, bool UNAL>
__device__ __forceinline__ V16 load_vector(const RowsOf& m, const char* row, int64_t at,
                                           int64_t row_bytes) {
  const V16 none = {{0u, 0u, 0u, 0u}};
  if constexpr (!UNAL) {
    return at < row_bytes ? load_granule<T>(row + at, m.base, m.end) : none;
  } else {
    const uint32_t lead = lead_of(row);
    const char* p = row - lead + at;
    const V16 a = at < row_bytes + lead ? load_granule<T>(p, m.base, m.end) : none;
    V16 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = __shfl_down_sync(0xffffffffu, a.w[i], 1);
    if ((threadIdx.x & 31u) == 31u)
      b = at + 16 < row_bytes + lead ? load_granule<T>(p + 16, m.base, m.end) : none;
    return window<T>(a, b, lead);
  }
}

// Stores the lane's vector of a strip (every lane calls it); ``left``: values_left of the vector.  With lead != 0 a lane writes the granule that its vector begins
// in, with the end of the lane before's; at a strip's and the row's ends values go one by one.
template <typename T, bool UNAL>
__device__ __forceinline__ void store_vector(char* row, int64_t at, const V16& r, int left) {
  constexpr int kN = kVec<T>, kSize = sizeof(T);
  const uint32_t lead = UNAL ? lead_of(row) : 0u;
  if (!UNAL || lead == 0u) {
    if (left >= kN) {
      store16(row + at, r);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < left) store_one<T>(row + at, r, i);
    }
  } else {
    const uint32_t lane = threadIdx.x & 31u;
    V16 prev;
#pragma unroll
    for (int i = 0; i < 4; ++i) prev.w[i] = __shfl_up_sync(0xffffffffu, r.w[i], 1);
    const V16 g = window<T>(prev, r, 16u - lead);
    const int ahead = static_cast<int>(lead) / kSize;       // values of the lane before
    char* p = row + at - lead;
    const int first = lane == 0u ? ahead : 0;
    const int limit = ahead + left;   // where left < 0, -left of the lane before's are missing too
    // lane 0 begins its granule at its own first value, lane 31 also ends the next one: its values
    // from kN - ahead on.  Both ends share the stores: value i of lane 0's granule, or of lane 31's
    // vector.
    if (first == 0 && limit >= kN) store16(p, g);
    const bool tail = lane == 31u && limit >= kN;
    if (tail || first != 0 || limit < kN) {
      const int lo = tail ? kN - ahead : first, hi = tail ? left : limit;
      char* q = tail ? row + at : p;
      V16 e;
#pragma unroll
      for (int i = 0; i < 4; ++i) e.w[i] = tail ? r.w[i] : g.w[i];
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i >= lo && i < hi) store_one<T>(q, e, i);
    }
  }
}

// ---------------------------------------------------------------- staging through shared memory
// Asynchronous copy of SIZE bytes (4, 8 or 16) to shared memory, both sides aligned to SIZE.
template <int SIZE>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (SIZE == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(SIZE)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// until at most N committed groups of this thread are in flight
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ V16 ld_shared_v16(uint32_t addr) {
  V16 r;
  ld_shared_v4(addr, r.w[0], r.w[1], r.w[2], r.w[3]);
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr uint32_t kStripBytes = 33 * 16;   // a strip's granules in shared memory

// Starts the copy of the lane's granule of a strip (and, from lane 31 with UNAL, of the 33rd) to
// ``strip``; what lies past the row's end is not copied.  ``inner``: inner_vector of the vector.
template <typename T, bool UNAL>
__device__ __forceinline__ void stage_vector(uint32_t strip, const RowsOf& m, const char* row,
                                             uint32_t at, int64_t row_bytes, bool inner) {
  const uint32_t lane = threadIdx.x & 31u;
  if constexpr (!UNAL) {
    if (inner) cp_async<16>(strip + lane * 16u, row + at);
  } else {
    const uint32_t lead = lead_of(row);
    const char* p = row - lead + at;
    if (inner) {
      cp_async<16>(strip + lane * 16u, p);
      if (lane == 31u) cp_async<16>(strip + 32u * 16u, p + 16);
      return;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j == 1 && lane != 31u) break;
      if (at + 16u * j >= row_bytes + lead) break;
      const char* q = p + 16 * j;
      const uint32_t dst = strip + (lane + j) * 16u;
      if (q >= m.base && q + 16 <= m.end) {
        cp_async<16>(dst, q);
      } else {   // at the matrix's ends
        const V16 r = load_granule<T>(q, m.base, m.end);
        st_shared_v4(dst, r.w[0], r.w[1], r.w[2], r.w[3]);
      }
    }
  }
}

// Whether a vector's granules lie within every row, so that nothing has to be checked: with UNAL
// not the first (with a lead it begins before the row) nor the last ones.
template <bool UNAL>
__device__ __forceinline__ bool inner_vector(uint32_t at, int64_t row_bytes) {
  return UNAL ? at >= 16u && at + 32u <= row_bytes : at + 16u <= row_bytes;
}

// The lane's vector of a staged strip (the warp's copies have landed).
template <typename T, bool UNAL>
__device__ __forceinline__ V16 staged_vector(uint32_t strip, uint32_t lead) {
  const uint32_t lane = threadIdx.x & 31u;
  const V16 a = ld_shared_v16(strip + lane * 16u);
  if constexpr (!UNAL) {
    return a;
  } else {
    return window<T>(a, ld_shared_v16(strip + lane * 16u + 16u), lead);
  }
}

// ---------------------------------------------------------------- parameters
// kVec<TX> parameters from column ``col`` on (values past ``cols`` read as zero): 16-byte loads
// where the array and the column allow them.
template <typename TP, int N>
__device__ __forceinline__ void load_params(const TP* p, uint32_t col, uint32_t cols, bool wide,
                                            float (&v)[N]) {
  if (wide && col + N <= cols) {
    if constexpr (sizeof(TP) * N >= 16) {
#pragma unroll
      for (int j = 0; j < N; j += kVec<TP>) {
        float u[kVec<TP>];
        values<TP>(load16(p + col + j), u);
#pragma unroll
        for (int i = 0; i < kVec<TP>; ++i) v[j + i] = u[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = col + i < cols ? to_f32(p[col + i]) : 0.0f;
}

// ---------------------------------------------------------------- sums over a warp
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of V (2 or 4) values over a warp at once: the lanes share the values out as they add, in
// V - 1 + log2(32 / V) shuffles instead of 5 V.  Returns the sum of value lane / (32 / V).
template <int V>
__device__ __forceinline__ float warp_sums(const float (&v)[V]) {
  const uint32_t lane = threadIdx.x & 31u;
  float u[V];
#pragma unroll
  for (int i = 0; i < V; ++i) u[i] = v[i];
  int o = 16;
#pragma unroll
  for (int n = V; n > 1; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = upper ? u[i + n / 2] : u[i], give = upper ? u[i] : u[i + n / 2];
      u[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) u[0] += __shfl_xor_sync(0xffffffffu, u[0], o);
  return u[0];
}
// the sum of value i of warp_sums, from the lanes that have it
template <int V>
__device__ __forceinline__ float sum_of(float sums, int i) {
  return __shfl_sync(0xffffffffu, sums, i * (32 / V));
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

// two E4M3 bytes (the low 16 bits) -> two floats (exact; by way of fp16, which holds every E4M3
// value)
__device__ __forceinline__ float2 e4m3x2_value(uint32_t bytes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// N (4 or 8) values of a checkpoint from their bytes (q[0] first) and scale byte
template <int N>
__device__ __forceinline__ void kept_values(const uint32_t* q, uint32_t s, float (&v)[N]) {
  const float scale = e8m0_value(s);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 f = e4m3x2_value(q[i / 4] >> (8 * (i & 2)));
    v[i] = f.x * scale;
    v[i + 1] = f.y * scale;
  }
}

// kept_values less ``mean``, rounded once (a byte times its scale is exact)
template <int N>
__device__ __forceinline__ void kept_less(const uint32_t* q, uint32_t s, float mean,
                                          float (&v)[N]) {
  const float scale = e8m0_value(s);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 f = e4m3x2_value(q[i / 4] >> (8 * (i & 2)));
    v[i] = fmaf(f.x, scale, -mean);
    v[i + 1] = fmaf(f.y, scale, -mean);
  }
}

// Quantises one block of 32 values held by 32 / N neighbouring lanes, N (4 or 8) each (values past
// the row's end are zero); every lane of the warp calls it.  Returns the scale byte, and this
// lane's bytes in ``q``.
template <int N>
__device__ __forceinline__ uint32_t ckpt8_quantise(const float (&v)[N], uint32_t (&q)[N / 4]) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));   // fmaxf passes over NaN
#pragma unroll
  for (int o = 1; o < kCkptBlock / N; o <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float u[N];
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] = v[i];
  if (__any_sync(0xffffffffu, amax == INFINITY)) {   // rare: infinities become NaN, amax is redone
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (fabsf(u[i]) == INFINITY) u[i] = __uint_as_float(0x7fffffffu);
      amax = fmaxf(amax, fabsf(u[i]));
    }
#pragma unroll
    for (int o = 1; o < kCkptBlock / N; o <<= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  const uint32_t s = ckpt8_scale_byte(amax);
  const float inv = ckpt8_inverse(s);
#pragma unroll
  for (int i = 0; i < N; i += 4)
    q[i / 4] = e4m3x2(u[i] * inv, u[i + 1] * inv) | e4m3x2(u[i + 2] * inv, u[i + 3] * inv) << 16;
  return s;
}

// This lane's bytes of a checkpoint's row, N (4 or 8) at p (aligned to N).
template <int N>
__device__ __forceinline__ void store_kept(uint8_t* p, const uint32_t (&q)[N / 4]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = q[0];
}
template <int N>
__device__ __forceinline__ void load_kept(const uint8_t* p, uint32_t (&q)[N / 4]) {
  if constexpr (N == 8) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    q[0] = r.x;
    q[1] = r.y;
  } else {
    q[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

}  // namespace tg
