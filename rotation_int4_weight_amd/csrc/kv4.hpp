// kv4.hpp - the layout of the pages of a cache in four bits (paro_kv_cache with
// PARO_KV4_F16 or PARO_KV4_BF16), as device code sees it: one head of one page
// holds its codes, then a {scale, low} pair of 16-bit values per position and
// 64 channels.
#pragma once

#include "attention.hpp"
#include "common.hpp"

namespace paro {

template <int DIM>
struct Kv4 {
  static constexpr int kGroups = DIM / kKv4Group;  // pairs per position
  static constexpr int kRow = DIM / 2;             // bytes of codes per position
  static constexpr int kSteps = DIM / 32;          // contraction steps of K, words per lane group and position
  // bytes of one head's page of P positions, and where its pairs begin
  static __host__ __device__ constexpr int64_t head_bytes(int page) { return (int64_t)page * DIM * 9 / 16; }
  static __host__ __device__ constexpr int pairs_at(int page) { return page * kRow; }
  // byte of the 32-bit K word with channels 8 c8 .. 8 c8 + 7 of position p
  static __device__ __forceinline__ int k_word(int p, int c8) { return 4 * ((p * 4 + (c8 & 3)) * kSteps + (c8 >> 2)); }
  // byte of the 16-bit V word with channels 4 c4 .. 4 c4 + 3 of position p
  static __device__ __forceinline__ int v_word(int p, int c4) {
    return 2 * ((((p >> 2) * 16 + (c4 & 15)) * kGroups + (c4 >> 4)) * 4 + (p & 3));
  }
};

}  // namespace paro
