// abi.hpp - what the C-ABI sources share: the thread-local last error and the
// pointer checks.  The state itself lives in paro_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

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

// Whether two tensors [rows][heads][dim bytes] of the same strides (in bytes, at
// least 0; that of a single row or head does not matter) share a byte: for each
// distance in heads, the distances in rows that bring them closest together.
inline bool strided_overlap(const void *a, const void *b, int64_t rows, int heads, int64_t dim, int64_t row,
                            int64_t head) {
  const int64_t delta = (int64_t)((uintptr_t)b - (uintptr_t)a), most = rows - 1;
  for (int64_t h = 1 - heads; h < heads; ++h) {
    const int64_t at = delta + (heads > 1 ? h * head : 0), near = rows > 1 && row > 0 ? -at / row : 0;
    for (int64_t r = near - 1; r <= near + 1; ++r) {
      const int64_t d = at + (rows > 1 ? std::max(-most, std::min(most, r)) * row : 0);
      if (d > -dim && d < dim) return true;
    }
  }
  return false;
}

inline bool act_dtype(int dt) { return dt == PARO_F16 || dt == PARO_BF16; }

constexpr int64_t kMaxOut = int64_t(1) << 21;
// Every workspace of the linears, the decode attention and the cache's pages
// starts with a fixed counter area: for the split-K reduction one 32-bit
// counter on its own 128-byte line per 128-column tile, at most kMaxOut/128
// tiles; for the attention's join its first kDecodeCounters (over four bits
// kDecode4Counters) words.  A zero-filled workspace stays valid across shapes,
// paths and these calls: none ever writes anything but zeros-at-exit into it.
constexpr size_t kCounterBytes = (size_t)(kMaxOut / 128) * 128;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

}  // namespace paro
