// kv_pages.hip - the pages of the key-value cache: writing new rows
// (paro_kv_append), granting pages with copy on write (paro_kv_reserve),
// sharing (paro_kv_fork), giving up (paro_kv_free) and compacting
// (paro_kv_compact).
//
// The bookkeeping is decided on the device, so that a serving step needs no
// host round trip and can be captured into a graph.  Decisions that depend on
// all entries (which page is free, who is first) are made by one workgroup of
// 1024 threads; the data then moves in a second, wide launch that reads the
// list of page copies the first one left in the workspace (short forks need no
// second one).  Free pages are taken in ascending order and ties go to the
// earliest entry, so the same state and call give the same result.
//
// Measured in a graph (8 heads of 128 channels, 16-position pages of 32 KB per
// K or V and layer): eight branches of a 1000-position slot in 32 layers, fork,
// reserve with eight copied pages and free, 21.5 us, of which a launch after
// the other takes about 3 us each; moving 500 of 1200 pages in 4 layers 56 us,
// 4.7 TB/s; appending 64 rows 3.2 us (a launch), 4096 rows 6.7 us, 5.0 TB/s of
// rows read and written (a copy of 1 GiB: 4.8).
#include <algorithm>

#include "attention.hpp"
#include "common.hpp"
#include "kv_rows.hpp"

namespace paro {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPagesPerLane = 16;  // refs one lane looks at per step of the page scan
constexpr int kScanStep = kPlanThreads * kPagesPerLane;

// Workspace (int32): [0] number of page copies, [kSrc..] sources, [dst..]
// targets, [list..] pages found by the scan, [map..] where a page went.
constexpr int kSrc = 16;
struct Work {
  int32_t *copies, *src, *dst, *list, *map;
};
__host__ __device__ inline Work work_of(int32_t *w, int64_t num_pages) {
  const int64_t most = num_pages > kMaxSlots ? num_pages : kMaxSlots;  // pages, or entries of a call
  return Work{w, w + kSrc, w + kSrc + most, w + kSrc + 2 * most, w + kSrc + 3 * most};
}

struct Pool {
  int32_t *refs, *table, *lengths;
  int num_pages, slots, max_pages, page_shift;
  __device__ int held(int len) const {  // pages of a slot of this length
    const int most = max_pages << page_shift;
    len = len < 0 ? 0 : len > most ? most : len;
    return (len + (1 << page_shift) - 1) >> page_shift;
  }
};

// Exclusive prefix sum of v over the workgroup; total: the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *wave_sums, T &total) {
  T incl = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_up(incl, d, 64);
    if (lane_id() >= d) incl += o;
  }
  __syncthreads();  // wave_sums may still be read from the call before
  if (lane_id() == 63) wave_sums[wave_id()] = incl;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const T s = wave_sums[w];
    before += w < wave_id() ? s : 0;
    total += s;
  }
  return before + incl - v;
}

// Calls take(rank, page) for the pages that pick(page, refs[page]) chooses, in
// ascending order of the page, ranks 0, 1, ..., until `want` are found or the
// pages end; returns the number found (it may pass `want` by a step).  Each
// lane looks at kPagesPerLane pages, 64 apart, all loads in flight together.
template <class Pick, class Take>
__device__ __forceinline__ int scan_pages(const Pool &p, int want, int *wave_sums, Pick pick, Take take) {
  int found = 0;
  for (int base = 0; base < p.num_pages && found < want; base += kScanStep) {
    const int first = base + wave_id() * 64 * kPagesPerLane + lane_id();
    int r[kPagesPerLane];
#pragma unroll
    for (int j = 0; j < kPagesPerLane; ++j) {
      const int page = first + 64 * j;
      r[j] = page < p.num_pages ? p.refs[page] : 0;
    }
    uint64_t hit[kPagesPerLane];
    int count = 0;
#pragma unroll
    for (int j = 0; j < kPagesPerLane; ++j) {
      const int page = first + 64 * j;
      hit[j] = __ballot(page < p.num_pages && pick(page, r[j]));
      count += __popcll(hit[j]);
    }
    int total;
    int rank = found + block_scan(lane_id() == 0 ? count : 0, wave_sums, total);
    rank = __shfl(rank, 0, 64);  // lane 0: what lies before this wave
#pragma unroll
    for (int j = 0; j < kPagesPerLane; ++j) {
      const uint64_t below = hit[j] & ((1ull << lane_id()) - 1ull);
      if ((hit[j] >> lane_id()) & 1ull) take(rank + __popcll(below), first + 64 * j);
      rank += __popcll(hit[j]);
    }
    found += total;
  }
  return found;
}

// first[s] = the first entry that names slot s (kPlanThreads threads).
__device__ __forceinline__ void first_entries(const int32_t *slots, int n, int num_slots, int *first) {
  for (int s = threadIdx.x; s < num_slots; s += kPlanThreads) first[s] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = slots[i];
    if (s >= 0 && s < num_slots) atomicMin(&first[s], i);
  }
  __syncthreads();
}

// ---- reserve ----

// Bound by latency: the slot, its length, its last page and that page's count
// are loads that wait for each other, then the scan of the counts (16384 pages a
// step), the table and the counts are written.
constexpr int kEntriesPerThread = kMaxSlots / kPlanThreads;

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(Pool p, const int32_t *__restrict__ slots,
                                                                   const int32_t *__restrict__ grow, int n,
                                                                   int32_t *__restrict__ granted, Work w) {
  __shared__ int first[kMaxSlots];  // first entry of a slot, then the first new position of an entry's pages
  __shared__ int ends[kMaxSlots];   // pages that an entry and those before it need
  __shared__ int wave_sums[kPlanWaves];
  __shared__ int64_t long_sums[kPlanWaves];
  __shared__ int copies;
  if (threadIdx.x == 0) copies = 0;
  first_entries(slots, n, p.slots, first);

  // what each entry needs, 1024 entries at a time (thread: one entry); the
  // sums stop at num_pages + 1 (more is never granted)
  int need[kEntriesPerThread], at[kEntriesPerThread], newlen[kEntriesPerThread], shared[kEntriesPerThread];
  int64_t run = 0;
#pragma unroll
  for (int u = 0; u < kEntriesPerThread; ++u) {
    const int i = u * kPlanThreads + (int)threadIdx.x;
    need[u] = 0;
    newlen[u] = -1;  // refused
    shared[u] = -1;
    at[u] = 0;
    if (u * kPlanThreads >= n) continue;
    const int s = i < n ? slots[i] : -1, g = i < n ? grow[i] : 0;
    if (s >= 0 && s < p.slots && first[s] == i && g >= 0) {
      const int len = p.lengths[s];
      if (len >= 0 && (int64_t)len + g <= ((int64_t)p.max_pages << p.page_shift)) {
        newlen[u] = len + g;
        const int have = p.held(len);
        at[u] = have;
        if (g > 0 && (len & ((1 << p.page_shift) - 1)) != 0) {
          const int last = p.table[(int64_t)s * p.max_pages + have - 1];
          if (last >= 0 && last < p.num_pages && p.refs[last] > 1) {
            shared[u] = last;
            at[u] = have - 1;
          }
        }
        need[u] = p.held(newlen[u]) - at[u];
      }
    }
    int64_t all;
    const int64_t end = run + block_scan((int64_t)need[u], long_sums, all) + need[u];
    run += all;
    if (i < n) ends[i] = (int)min(end, (int64_t)p.num_pages + 1);
  }
  const int total = (int)min(run, (int64_t)p.num_pages);
  __syncthreads();  // first[] is read no more as entries
#pragma unroll
  for (int u = 0; u < kEntriesPerThread; ++u) {
    const int i = u * kPlanThreads + (int)threadIdx.x;
    if (i < n) first[i] = at[u];
  }
  const int found = scan_pages(
      p, total, wave_sums, [](int, int r) { return r == 0; },
      [&](int rank, int page) {
        if (rank < total) w.list[rank] = page;
      });
  const int free = min(found, total);
  __syncthreads();  // the list is written, and every refs value that decides has been read
#pragma unroll
  for (int u = 0; u < kEntriesPerThread; ++u) {
    const int i = u * kPlanThreads + (int)threadIdx.x;
    if (i >= n) continue;
    const bool yes = newlen[u] >= 0 && (need[u] == 0 || ends[i] <= free);
    granted[i] = yes;
    if (!yes) {
      if (need[u] > 0) first[i] = -1;
      continue;
    }
    p.lengths[slots[i]] = newlen[u];
    if (shared[u] >= 0) {
      atomicSub(&p.refs[shared[u]], 1);
      const int c = atomicAdd(&copies, 1);
      w.src[c] = shared[u];
      w.dst[c] = w.list[ends[i] - need[u]];
    }
  }
  __syncthreads();
  // page rank r belongs to the first entry with ends > r (binary search)
  for (int r = threadIdx.x; r < free; r += kPlanThreads) {
    int low = 0, high = n - 1;
    while (low < high) {
      const int mid = (low + high) >> 1;
      if (ends[mid] > r) high = mid;
      else low = mid + 1;
    }
    if (first[low] < 0 || ends[low] <= r) continue;  // not granted
    const int before = low ? ends[low - 1] : 0, page = w.list[r];
    p.table[(int64_t)slots[low] * p.max_pages + first[low] + (r - before)] = page;
    p.refs[page] = 1;
  }
  if (threadIdx.x == 0) w.copies[0] = copies;
}

// ---- page copies, K and V of every layer ----

// Work items: copy x layer x {K, V} x 16 KB piece; the number of copies is
// read on the device, so a launch with none ends at once.  Each lane keeps
// four 16-byte loads in flight.  Bound by HBM: 4.7 TB/s where many pages move.
constexpr int kPiece = 16384;

// MOVED: the pages leave their places for good, so the tables are rewritten too
// (every workgroup takes some slots first).
template <bool MOVED>
__global__ void __launch_bounds__(256) copy_pages_kernel(char *__restrict__ k, char *__restrict__ v, Pool p,
                                                         const int32_t *__restrict__ used_in, Work w, int layers,
                                                         int64_t num_pages, int64_t page_bytes) {
  if constexpr (MOVED) {
    const int used = used_in[0];
    for (int s = blockIdx.x; s < p.slots; s += gridDim.x) {
      const int pages = p.held(p.lengths[s]);
      int32_t *row = p.table + (int64_t)s * p.max_pages;
      for (int j = threadIdx.x; j < pages; j += 256) {
        const int page = row[j];
        if (page >= used && page < p.num_pages) row[j] = w.map[page];
      }
    }
  }
  const int64_t copies = w.copies[0];
  const int pieces = (int)((page_bytes + kPiece - 1) / kPiece);
  const int64_t items = copies * layers * 2 * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = (int)(it % pieces);
    int64_t r = it / pieces;
    char *base = (r & 1) ? v : k;
    r >>= 1;
    const int64_t layer = r % layers, c = r / layers;
    const int64_t src = w.src[c], dst = w.dst[c];
    const char *from = base + (layer * num_pages + src) * page_bytes + (int64_t)piece * kPiece;
    char *to = base + (layer * num_pages + dst) * page_bytes + (int64_t)piece * kPiece;
    const int bytes = (int)min((int64_t)kPiece, page_bytes - (int64_t)piece * kPiece);
    u32x4 t[kPiece / 4096];
#pragma unroll
    for (int j = 0; j < kPiece / 4096; ++j) {
      const int o = (j * 256 + (int)threadIdx.x) * 16;
      if (o < bytes) t[j] = *reinterpret_cast<const u32x4 *>(from + o);
    }
#pragma unroll
    for (int j = 0; j < kPiece / 4096; ++j) {
      const int o = (j * 256 + (int)threadIdx.x) * 16;
      if (o < bytes) *reinterpret_cast<u32x4 *>(to + o) = t[j];
    }
  }
}

// ---- fork ----

// Rows are shared in the planning launch where its 16 waves need at most this
// many steps of 64 table entries, were every row full (fork and free in one
// launch less / with it, us: 8 rows of 64 5.8 / 6.9, 16 of 256 (4 steps) 7.3 /
// 7.1, 16 of 512 10.0 / 7.7, 64 of 128 11.4 / 8.8; a launch is 3 us of host time).
constexpr int kForkSteps = 4;

// pages of a parent's row to the child's, by `threads` threads from `thread` on
__device__ __forceinline__ void share_pages(const Pool &p, int parent, int child, int pages, int thread, int threads) {
  const int32_t *from = p.table + (int64_t)parent * p.max_pages;
  int32_t *to = p.table + (int64_t)child * p.max_pages;
  for (int j = thread; j < pages; j += threads) {
    const int page = from[j];
    to[j] = page;
    if (page >= 0 && page < p.num_pages) atomicAdd(&p.refs[page], 1);
  }
}

// APPLY: the rows are shared here too, a wave taking an entry; otherwise
// w.src[i] leaves the number of pages to share to fork_apply_kernel.
template <bool APPLY>
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Pool p, const int32_t *__restrict__ parents,
                                                                const int32_t *__restrict__ children, int n,
                                                                int32_t *__restrict__ granted, Work w) {
  __shared__ int first[kMaxSlots];
  first_entries(children, n, p.slots, first);
  int len[kEntriesPerThread];
  bool yes[kEntriesPerThread];
#pragma unroll
  for (int u = 0; u < kEntriesPerThread; ++u) {
    const int i = u * kPlanThreads + threadIdx.x;
    yes[u] = false;
    len[u] = 0;
    if (i >= n) continue;
    const int a = parents[i], c = children[i];
    if (a < 0 || a >= p.slots || c < 0 || c >= p.slots || a == c || first[c] != i || p.lengths[c] != 0) continue;
    yes[u] = true;
    len[u] = p.lengths[a];
  }
  __syncthreads();  // lengths as they were before the call have been read
#pragma unroll
  for (int u = 0; u < kEntriesPerThread; ++u) {
    const int i = u * kPlanThreads + threadIdx.x;
    if (i >= n) continue;
    granted[i] = yes[u];
    const int pages = yes[u] ? p.held(len[u]) : 0;
    if constexpr (APPLY) first[i] = pages;
    else w.src[i] = pages;
    if (yes[u]) p.lengths[children[i]] = len[u];
  }
  if constexpr (APPLY) {
    __syncthreads();
    for (int i = wave_id(); i < n; i += kPlanWaves)
      if (first[i] > 0) share_pages(p, parents[i], children[i], first[i], lane_id(), 64);
  }
}

// A child that is another entry's parent had no pages before the call, so no
// row is read and written at once.
__global__ void __launch_bounds__(256) fork_apply_kernel(Pool p, const int32_t *__restrict__ parents,
                                                         const int32_t *__restrict__ children, Work w) {
  const int i = blockIdx.y, pages = w.src[i];
  if (pages == 0) return;
  share_pages(p, parents[i], children[i], pages, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

// ---- free ----

__global__ void __launch_bounds__(256) free_kernel(Pool p, const int32_t *__restrict__ slots) {
  const int i = blockIdx.x, s = slots[i];
  if (s < 0 || s >= p.slots) return;
  bool earlier = false;  // an earlier entry names the slot: that one frees it
#pragma unroll 4
  for (int j = threadIdx.x; j < i; j += 256) earlier |= slots[j] == s;
  if (__syncthreads_or(earlier)) return;
  const int pages = p.held(p.lengths[s]);
  int32_t *row = p.table + (int64_t)s * p.max_pages;
  for (int j = threadIdx.x; j < pages; j += 256) {
    const int page = row[j];
    row[j] = -1;
    if (page >= 0 && page < p.num_pages) atomicSub(&p.refs[page], 1);
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) p.lengths[s] = 0;
}

// ---- compact ----

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Pool p, int32_t *__restrict__ used_out, Work w) {
  __shared__ int wave_sums[kPlanWaves];
  const int used = scan_pages(
      p, INT_MAX, wave_sums, [](int, int r) { return r > 0; }, [](int, int) {});
  // one scan numbers the free pages below `used` and, after them, the used
  // ones at or above it: as many of either
  const int found = scan_pages(
      p, INT_MAX, wave_sums, [used](int page, int r) { return page < used ? r <= 0 : r > 0; },
      [&](int rank, int page) { w.list[rank] = page; });
  const int moves = found / 2;
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kPlanThreads) {
    const int to = w.list[i], from = w.list[moves + i];
    w.src[i] = from;
    w.dst[i] = to;
    w.map[from] = to;
    p.refs[to] = p.refs[from];
    p.refs[from] = 0;
  }
  if (threadIdx.x == 0) {
    w.copies[0] = moves;
    used_out[0] = used;
  }
}

// ---- append ----

// A wave writes one row of K and of V.  Its sequence is found by a 64-way
// search of the offsets; a row whose entry is not the first to name its slot,
// or was refused its room, or whose position or page does not exist, is skipped.
__global__ void __launch_bounds__(256) append_kernel(KvLayer kv, int kv_heads, int dim_shift, const uint16_t *__restrict__ k,
                                                     int64_t k_token, int64_t k_head, const uint16_t *__restrict__ v,
                                                     int64_t v_token, int64_t v_head, const int32_t *__restrict__ slots,
                                                     const int64_t *__restrict__ cu, const int32_t *__restrict__ granted, int n,
                                                     int64_t tokens) {
  const int64_t row = (int64_t)blockIdx.x * 4 + wave_id();
  if (row >= tokens) return;
  const int lane = lane_id();
  Entry e;
  if (!entry_of(cu, n, row, tokens, lane, e)) return;
  const int s = slots[e.i];
  if (s < 0 || s >= kv.slots || (granted && granted[e.i] == 0) || named_before(slots, e.i, lane)) return;
  const int64_t pos = newest_position(kv, s, e, row);
  if (pos < 0) return;
  const int page = page_at(kv, s, pos);
  if (page < 0) return;
  const int dim = 1 << dim_shift;
  const int64_t base = (int64_t)page * kv.page_stride + ((pos & ((1 << kv.page_shift) - 1)) << dim_shift);
  const int64_t head_stride = (int64_t)dim << kv.page_shift;
  for (int c = lane * 8; c < kv_heads * dim; c += 512) {
    const int h = c >> dim_shift, d = c & (dim - 1);
    const u32x4 kk = *reinterpret_cast<const u32x4 *>(k + row * k_token + h * k_head + d);
    const u32x4 vv = *reinterpret_cast<const u32x4 *>(v + row * v_token + h * v_head + d);
    *reinterpret_cast<u32x4 *>(kv.k + base + h * head_stride + d) = kk;
    *reinterpret_cast<u32x4 *>(kv.v + base + h * head_stride + d) = vv;
  }
}

Pool pool_of(const paro_kv_cache &c) {
  Pool p;
  p.refs = c.refs;
  p.table = c.table;
  p.lengths = c.lengths;
  p.num_pages = (int)c.num_pages;
  p.slots = c.slots;
  p.max_pages = c.max_pages;
  p.page_shift = __builtin_ctz((unsigned)c.page_size);
  return p;
}

// used: compaction's; null for copies that leave their sources in place
hipError_t launch_copies(const paro_kv_cache &c, const Work &w, int64_t most_copies, const int32_t *used,
                         hipStream_t st) {
  const int64_t page_bytes = kv_page_units(c) * 2;
  const int64_t items = most_copies * c.layers * 2 * ((page_bytes + kPiece - 1) / kPiece);
  const dim3 grid((unsigned)std::min<int64_t>(std::max<int64_t>(items, used ? c.slots : 1), 2048)), block(256);
  if (used)
    hipLaunchKernelGGL(copy_pages_kernel<true>, grid, block, 0, st, (char *)c.k, (char *)c.v, pool_of(c), used, w,
                       c.layers, c.num_pages, page_bytes);
  else
    hipLaunchKernelGGL(copy_pages_kernel<false>, grid, block, 0, st, (char *)c.k, (char *)c.v, pool_of(c), used, w,
                       c.layers, c.num_pages, page_bytes);
  return hipGetLastError();
}

}  // namespace

size_t kv_work_ints(const paro_kv_cache &c) {
  const size_t most = (size_t)std::max<int64_t>(c.num_pages, kMaxSlots);
  return kSrc + 4 * most;
}

hipError_t launch_kv_reserve(const paro_kv_cache &c, const int32_t *slots, const int32_t *grow, int n,
                             int32_t *granted, int32_t *work, hipStream_t st) {
  const Work w = work_of(work, c.num_pages);
  hipLaunchKernelGGL(reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, pool_of(c), slots, grow, n, granted, w);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_copies(c, w, n, nullptr, st);
}

hipError_t launch_kv_fork(const paro_kv_cache &c, const int32_t *parents, const int32_t *children, int n,
                          int32_t *granted, int32_t *work, hipStream_t st) {
  const Work w = work_of(work, c.num_pages);
  const Pool p = pool_of(c);
  const int steps = ((n + kPlanWaves - 1) / kPlanWaves) * ((c.max_pages + 63) / 64);
  if (steps <= kForkSteps) {
    hipLaunchKernelGGL(fork_plan_kernel<true>, dim3(1), dim3(kPlanThreads), 0, st, p, parents, children, n, granted, w);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(fork_plan_kernel<false>, dim3(1), dim3(kPlanThreads), 0, st, p, parents, children, n, granted, w);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned blocks = (unsigned)std::min((c.max_pages + 255) / 256, 16);
  hipLaunchKernelGGL(fork_apply_kernel, dim3(blocks, (unsigned)n), dim3(256), 0, st, p, parents, children, w);
  return hipGetLastError();
}

hipError_t launch_kv_free(const paro_kv_cache &c, const int32_t *slots, int n, hipStream_t st) {
  hipLaunchKernelGGL(free_kernel, dim3((unsigned)n), dim3(256), 0, st, pool_of(c), slots);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const paro_kv_cache &c, int32_t *used, int32_t *work, hipStream_t st) {
  const Work w = work_of(work, c.num_pages);
  const Pool p = pool_of(c);
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p, used, w);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_copies(c, w, c.num_pages / 2, used, st);
}

hipError_t launch_kv_append(const KvLayer &kv, int kv_heads, int head_dim, const uint16_t *k, int64_t k_token,
                            int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head, const int32_t *slots,
                            const int64_t *cu, const int32_t *granted, int n, int64_t tokens, hipStream_t st) {
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)((tokens + 3) / 4)), dim3(256), 0, st, kv, kv_heads,
                     __builtin_ctz((unsigned)head_dim), k, k_token, k_head, v, v_token, v_head, slots, cu, granted,
                     n, tokens);
  return hipGetLastError();
}

}  // namespace paro
