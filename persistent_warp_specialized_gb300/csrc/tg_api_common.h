// tg_api_common.h -- what the C-ABI translation units share: error reporting, pointer checks,
// device set-up and TMA descriptors.  Defined in tg_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tg {
namespace abi {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// Sets the calling thread's error message and returns ``code``.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail_cuda(const char* what, cudaError_t e);

// Sets the current device up on its first use (TG_ERR_CUDA if it is not sm_103).  Either pointer
// may be null: the SM count, and the CTA pairs of the pair kernels that are resident at once.
int device_ready(int* sms_out, int* max_pairs_out);

// device_ready, and the weight gradient's kernels set up on the device's first weight gradient (the
// other calls neither wait for them nor depend on their occupancy).  max_pairs_out: its own CTA pairs
// that are resident at once, at least one.
int wgrad_ready(int* sms_out, int* max_pairs_out);

// The same for the products with fused epilogues, on the device's first of them.
int linear_ready(int* sms_out, int* max_pairs_out);

// TG_OK if ``p`` is device memory of the current device (TMA reads it directly).
int check_device_ptr(const void* p, const char* name);

bool overlaps(const void* a, uint64_t abytes, const void* b, uint64_t bbytes);

// A row-major [outer, inner] matrix of ``elem_bytes``-byte elements, boxes of box_outer rows x
// box_inner elements landing with the 128-byte swizzle (or none).  pitch_bytes: bytes between rows
// (0: rows are contiguous).
int encode_tiled(CUtensorMap* map, CUtensorMapDataType dt, uint32_t elem_bytes, const void* base,
                 uint64_t inner, uint64_t outer, uint32_t box_inner, uint32_t box_outer,
                 const char* name, bool swizzle = true, uint64_t pitch_bytes = 0);

// The default limit of every bounded wait in the kernels when the caller gives none: the
// fixed kDefaultWatchdogNs plus 2 us per k-block of K.  The longest legitimate wait spans one
// unit's whole K (the epilogue waiting for its accumulator), and a k-block takes at most about
// 0.5 us on GB300 even on a CTA pair's half-width unit, so with K near 2^31 (2^25 k-blocks of
// 64, ~12 s per unit, measured) a fixed limit of ~4 s stopped a correct GEMM.
uint64_t default_watchdog_ns(uint32_t k_blocks);

}  // namespace abi
}  // namespace tg
