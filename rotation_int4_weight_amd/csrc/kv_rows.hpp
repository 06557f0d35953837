// kv_rows.hpp - where a packed row stands in the paged cache: shared by the
// calls that write rows into the pages and that read them back.  Each function
// is called by a whole wave for one row.
#pragma once

#include "attention.hpp"
#include "common.hpp"

namespace paro {

// The entry i of a packed row, whose rows are low..high.
struct Entry {
  int i;
  int64_t low, high;
};

// The last entry with cu[i] <= row, found by 64-way steps (cu null: one row per
// entry); false for a row outside every entry.
__device__ __forceinline__ bool entry_of(const int64_t *__restrict__ cu, int n, int64_t row, int64_t tokens, int lane,
                                         Entry &e) {
  e.i = (int)row;
  e.low = row;
  e.high = row + 1;
  if (!cu) return true;
  // narrow [a, b) to one
  int a = 0, b = n;
  while (b - a > 1) {
    const int step = (b - a + 63) / 64;
    const int at = a + lane * step;
    const uint64_t le = __ballot(at < b && cu[at < b ? at : a] <= row);
    if (!(le & 1)) return false;  // before the first sequence
    const int last = 63 - __clzll(le);
    a += last * step;
    b = min(b, a + step);
  }
  e.i = a;
  e.low = cu[a];
  e.high = cu[a + 1];
  if (e.low < 0) e.low = 0;
  if (e.high > tokens) e.high = tokens;
  return row >= e.low && row < e.high;
}

// Whether an entry before the i-th names its slot.
__device__ __forceinline__ bool named_before(const int32_t *__restrict__ slots, int i, int lane) {
  const int s = slots[i];
  bool earlier = false;
#pragma unroll 8
  for (int j = lane; j < i; j += 64) earlier |= slots[j] == s;
  return __any(earlier);
}

// The position of a row where its entry's rows are the newest of slot s (inside
// the cache); negative: there is none.
__device__ __forceinline__ int64_t newest_position(const KvLayer &kv, int s, const Entry &e, int64_t row) {
  const int len = min(kv.lengths[s], kv.max_pages << kv.page_shift);
  return len <= 0 ? -1 : (int64_t)len - (e.high - row);
}

// The page of position pos >= 0 (inside max_pages) of slot s, -1 if it is none.
__device__ __forceinline__ int page_at(const KvLayer &kv, int s, int64_t pos) {
  const int page = kv.table[(int64_t)s * kv.max_pages + (pos >> kv.page_shift)];
  return page < 0 || page >= kv.num_pages ? -1 : page;
}

}  // namespace paro
