// abi.hpp - what the C-ABI sources share: the thread-local last error and the
// pointer checks.  The state itself lives in paro_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "paro.h"

namespace paro {

// Records the message for paro_last_error() and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the message and returns PARO_OK.
int ok();
int hip_fail(hipError_t e, const char *what);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool overlap(const void *a, size_t an, const void *b, size_t bn) {
  const char *pa = (const char *)a, *pb = (const char *)b;
  return an && bn && pa < pb + bn && pb < pa + an;
}

inline bool act_dtype(int dt) { return dt == PARO_F16 || dt == PARO_BF16; }

constexpr int64_t kMaxOut = int64_t(1) << 21;
// Every workspace of the linears, the decode attention and the cache's pages
// starts with a fixed counter area: for the split-K reduction one 32-bit
// counter on its own 128-byte line per 128-column tile, at most kMaxOut/128
// tiles; for the attention's join its first kDecodeCounters words.  A
// zero-filled workspace stays valid across shapes, paths and these calls: none
// ever writes anything but zeros-at-exit into it.
constexpr size_t kCounterBytes = (size_t)(kMaxOut / 128) * 128;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace paro
