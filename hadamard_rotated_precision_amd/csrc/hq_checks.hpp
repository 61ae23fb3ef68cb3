// hq_checks.hpp — what the C-ABI layers of libhq_train.so and libhq_mx.so share: limits, alignment
// and device checks (plain host C++).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hq_internal.hpp"

namespace hq {

inline int64_t pitch16(int64_t n) { return (n + 15) / 16 * 16; }
inline size_t align256(size_t n) { return (n + 255) / 256 * 256; }
inline bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool valid_dt(int32_t dt) { return dt == HQ_F32 || dt == HQ_F16 || dt == HQ_BF16; }
// matrices and vectors of floating-point elements may start at any element
inline bool element_aligned(const void* p, int32_t dt) { return aligned(p, dt == HQ_F32 ? 4 : 2); }

// Largest extent of a matrix axis, and 2^38 elements in all: tiles are addressed with 32-bit
// offsets inside a row block, and workgroup counts stay inside a grid.
constexpr int64_t kMaxDim = int64_t{1} << 22;

inline bool dims_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && a <= kMaxDim && b <= kMaxDim &&
         ((a + 127) / 128) * ((b + 127) / 128) <= (int64_t{1} << 24);
}

#define HQ_CHECK(expr)             \
  do {                             \
    hq_status s_ = (expr);         \
    if (s_ != HQ_OK) return s_;    \
  } while (0)
#define HQ_TRY(expr)                                  \
  do {                                                \
    if ((expr) != hipSuccess) return HQ_ERR_LAUNCH;   \
  } while (0)

// The library's device checks, and the stream's device: a kernel must not be launched on a
// stream of another device than the current one.
inline hq_status stream_ok(void* stream) {
  HQ_CHECK(device_ready());
  if (!stream) return HQ_OK;
  int cur = 0;
  hipDevice_t of = 0;
  if (hipGetDevice(&cur) != hipSuccess) return HQ_ERR_DEVICE;
  if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &of) != hipSuccess) return HQ_ERR_DEVICE;
  return of == cur ? HQ_OK : HQ_ERR_DEVICE;
}

inline hq_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return HQ_OK;
  if (!ws || have < need) return HQ_ERR_WORKSPACE;
  return aligned(ws, 16) ? HQ_OK : HQ_ERR_ALIGN;
}

}  // namespace hq
