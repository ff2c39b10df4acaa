// tg_api_checks.h -- the checks of arguments that the training operators' C-ABI translation units
// share: sizes, strides, arrays, and outputs that must not overlap what else a call is given.
#pragma once

#include <cstdint>

#include "../../include/tg.h"
#include "tg_api_common.h"

#define TG_TRY(call)                 \
  do {                               \
    const int rc_ = (call);          \
    if (rc_ != TG_OK) return rc_;    \
  } while (0)

namespace tg {
namespace abi {

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

inline bool known_dtype(int d) { return d == TG_F16 || d == TG_BF16 || d == TG_F32; }
inline uint64_t elem_bytes(int d) { return d == TG_F32 ? 4 : 2; }

inline bool off_by(const void* p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// bytes from the first to the last element of a [rows, cols] matrix with row stride ld
inline uint64_t span(int64_t rows, int64_t cols, int64_t ld, uint64_t elem) {
  return rows == 0 ? 0 : ((static_cast<uint64_t>(rows) - 1) * ld + cols) * elem;
}

inline int check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim)
    return fail(TG_ERR_ARG, "sizes must be in [0, 2^31): rows=%lld cols=%lld", (long long)rows,
                (long long)cols);
  return TG_OK;
}

inline int check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols || ld > kMaxDim)
    return fail(TG_ERR_ARG, "%s=%lld must be at least the row's %lld values and below 2^31", name,
                (long long)ld, (long long)cols);
  return TG_OK;
}

// A required device array of ``elem``-byte elements.
inline int check_array(const void* p, uint64_t elem, const char* name) {
  if (!p) return fail(TG_ERR_ARG, "null pointer: %s", name);
  if (off_by(p, elem))
    return fail(TG_ERR_ALIGN, "%s must be %llu-byte aligned", name, (unsigned long long)elem);
  return check_device_ptr(p, name);
}

// The array ``p`` if the caller gave it.
inline int check_optional(const void* p, uint64_t elem, const char* name) {
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

inline Region matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, uint64_t elem,
              const char* name) {
  return {p, span(rows, cols, ld, elem), name, cols * elem, ld * elem};
}

// Whether two arrays share no byte.  Matrices of one pitch may lie in each other's gaps, as column
// slices of one buffer do: their rows then take separate parts of every ``pitch`` bytes.  Anything
// else is told apart by where it begins and ends.
inline bool apart(const Region& a, const Region& b) {
  if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return true;
  if (a.pitch == 0 || a.pitch != b.pitch) return false;
  const uint64_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  // how far into a's rows b's begin
  const uint64_t at = b0 >= a0 ? (b0 - a0) % a.pitch : a.pitch - 1 - (a0 - b0 - 1) % a.pitch;
  return at >= a.row && at + b.row <= a.pitch;
}

// No output may overlap an input or another output (regions [0, outs) are the outputs).
inline int check_apart(const Region* r, int outs, int n) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (r[i].p && r[j].p && !apart(r[i], r[j]))
        return fail(TG_ERR_ARG, "%s overlaps %s", r[i].name, r[j].name);
  return TG_OK;
}

}  // namespace abi
}  // namespace tg
