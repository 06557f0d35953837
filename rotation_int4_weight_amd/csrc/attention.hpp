// attention.hpp - internal host launchers of the attention and key-value
// cache kernels.  attention_abi.cpp validates every argument before calling
// these; all pointers are device pointers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "paro.h"

namespace paro {

constexpr int kMaxSlots = 4096;      // the planning kernels keep per-slot tables in LDS
constexpr int kMaxSequences = 16384;  // with 256 heads and the most rows, under 2^32 threads a launch
constexpr int kMaxDecodeRows = 32768;  // a grid dimension

// Caches in four bits (include/paro.h gives the layout): 64 channels share a
// scale and a lowest value.
constexpr int kKv4Group = 64;
inline bool kv4(int dt) { return dt == PARO_KV4_F16 || dt == PARO_KV4_BF16; }
// the type of the rows, queries and outputs of a cache
inline int kv_row_dtype(int dt) { return dt == PARO_KV4_F16 ? PARO_F16 : dt == PARO_KV4_BF16 ? PARO_BF16 : dt; }
// 16-bit units of a page of K (or V) of one layer: elements, or codes and pairs
inline int64_t kv_page_units(const paro_kv_cache &c) {
  const int64_t n = (int64_t)c.kv_heads * c.page_size * c.head_dim;
  return kv4(c.dt) ? n * 9 / 32 : n;
}

// One layer of a paged cache as the kernels see it.
struct KvLayer {
  uint16_t *k, *v;         // the layer's pages [num_pages][kv_heads][page_size][head_dim], or in four bits
  const int32_t *table;    // [slots][max_pages]
  const int32_t *lengths;  // [slots]
  int64_t page_stride;     // 16-bit units per page (kv_page_units)
  int num_pages, max_pages, slots;
  int page_shift;          // log2(page_size)
  // positions that a slot holds (0 for one outside the cache)
  __device__ int length(int slot) const {
    if (slot < 0 || slot >= slots) return 0;
    const int n = lengths[slot], most = max_pages << page_shift;
    return n < 0 ? 0 : n > most ? most : n;
  }
};

struct AttentionArgs {
  const uint16_t *q, *k, *v;  // k, v: packed prompts only
  uint16_t *y;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, y_token, y_head;  // elements
  int q_heads, kv_heads, group;  // group = q_heads / kv_heads
  int head_dim, dt, causal;
  float scale;
  int64_t q_tokens, k_tokens;
  const int64_t *cu_q, *cu_k;
  const int32_t *slots;  // cache forms
  int sequences;         // prompts: sequences; decode: rows
  KvLayer kv;            // cache forms
};

// A finite output stays finite in fp16: rounded weights may carry a sum of
// values of 65504 past the type by up to 2^-11.  Infinities and NaN stay.
constexpr float kMaxF16 = 65504.f;
template <bool FP16>
__device__ __forceinline__ float within_type(float x) {
  if constexpr (!FP16) return x;
  return __builtin_fabsf(x) < __builtin_inff() ? __builtin_amdgcn_fmed3f(x, -kMaxF16, kMaxF16) : x;
}

// Prompts: K and V packed (cached = false) or in the cache's pages.  Over the
// cache, few rows may have their keys split over `splits` workgroups (at most
// attention_prompt_splits; then there are fewer than kDecodeCounters of them).
int attention_prompt_splits(int64_t q_tokens, int64_t sequences, int q_heads, int kv_heads, int64_t max_len);
size_t attention_prompt_partial_bytes(int splits, int64_t q_tokens, int64_t sequences, int q_heads, int kv_heads,
                                      int head_dim);
hipError_t launch_attention_prompt(const AttentionArgs &a, bool cached, int splits, uint32_t *counters, float *sums,
                                   hipStream_t st);

// One token per row over the cache.  The length of a row is split over
// `splits` workgroups where there are fewer than kDecodeCounters (row,
// key-value head, head tile) items, so a fixed counter area at the start of
// every workspace serves all shapes and stays zero between calls.
constexpr int kDecodeCounters = 512;
struct DecodeAttentionPlan {
  int splits;
  int head_tiles;  // workgroups per key-value head: its query heads in tiles of 16
};
DecodeAttentionPlan plan_attention_decode(int64_t rows, int q_heads, int kv_heads, int64_t max_len);
size_t attention_decode_partial_bytes(const DecodeAttentionPlan &p, int64_t rows, int kv_heads, int head_dim);
hipError_t launch_attention_decode(const AttentionArgs &a, const DecodeAttentionPlan &p, uint32_t *counters,
                                   float *partials, hipStream_t st);

// The same over a cache in four bits: the keys of all rows together are dealt
// out to the workgroups that the card holds at once (two per CU), a counter and
// two slots for parts each.
constexpr int kMaxDealtRows = 4096;
constexpr int kDecode4Resident = 2;  // workgroups per CU
constexpr int kDecode4Counters = 256 * kDecode4Resident;
struct Decode4Plan {
  int head_tiles;  // as above
  int workgroups;
  bool dealt;      // false: a workgroup per output, that is row, key-value head and head tile
  int whole;       // the same where no row has more units than this; 0: more outputs than workgroups
};
Decode4Plan plan_attention_decode4(int64_t rows, int q_heads, int kv_heads, int64_t max_len);
// for any number of rows, so that a workspace serves fewer of them too
size_t attention_decode4_partial_bytes(int q_heads, int kv_heads, int head_dim);
hipError_t launch_attention_decode4(const AttentionArgs &a, const Decode4Plan &p, uint32_t *counters,
                                    float *partials, hipStream_t st);

hipError_t launch_kv_append(const KvLayer &kv, int kv_heads, int head_dim, const uint16_t *k, int64_t k_token,
                            int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head, const int32_t *slots,
                            const int64_t *cu, const int32_t *granted, int n, int64_t tokens, hipStream_t st);

// The same into a cache in four bits; dt: the rows' type.
hipError_t launch_kv_append4(const KvLayer &kv, int kv_heads, int head_dim, int dt, const uint16_t *k,
                             int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                             const int32_t *slots, const int64_t *cu, const int32_t *granted, int n, int64_t tokens,
                             hipStream_t st);
// Rows out of the pages; k or v may be null.  four: the cache is in four bits.
struct KvReadArgs {
  KvLayer kv;
  int kv_heads, head_dim, dt, out_dt;  // dt: the rows' type; out_dt: dt or kF32
  bool four;
  void *k, *v;
  int64_t k_token, k_head, v_token, v_head;  // elements
  const int32_t *slots, *first;              // first may be null
  const int64_t *cu;                         // may be null
  int n;
  int64_t tokens;
};
hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t st);

// Page bookkeeping.  work: kv_work_ints(c) int32.
size_t kv_work_ints(const paro_kv_cache &c);
hipError_t launch_kv_reserve(const paro_kv_cache &c, const int32_t *slots, const int32_t *grow, int n,
                             int32_t *granted, int32_t *work, hipStream_t st);
hipError_t launch_kv_fork(const paro_kv_cache &c, const int32_t *parents, const int32_t *children, int n,
                          int32_t *granted, int32_t *work, hipStream_t st);
hipError_t launch_kv_free(const paro_kv_cache &c, const int32_t *slots, int n, hipStream_t st);
hipError_t launch_kv_compact(const paro_kv_cache &c, int32_t *used, int32_t *work, hipStream_t st);

}  // namespace paro
