// attention_prompt.hip - attention over prompts (paro_attention_prompt over
// packed K and V, paro_attention_prompt_cached over the cache's pages).
//
// A workgroup takes 128 rows of one key-value head, a row being a (token,
// query head of the group) pair, so that the heads that share K and V share
// their tiles, short prompts fill a tile and the diagonal wastes little.  K
// and V stream through LDS in tiles of 64 keys (two buffers, loaded straight
// into LDS), and a wave keeps everything of its 32 rows in registers:
//   S^T = K Q^T and O^T = V^T P^T on v_mfma_f32_32x32x16.  Both have the row
//   in lane%32, so maxima and sums need one swap of lane halves.  S^T leaves
//   half h of a wave with the keys 8n + 4h + 0..3 of each 32; the second
//   product's contraction is numbered the same way, so the weights go from
//   one product to the other without leaving their lane.  V^T fragments are
//   read from row-major V by the transposing LDS read (16 lanes receive 16
//   channels of 4 keys).
//   Running maximum m and sum l: a tile's weights are exp2((s - m) scale2),
//   relative to an m that is only moved (and what was summed before scaled)
//   when some row's maximum rose by more than 2^8 over it: any m gives the
//   same quotient.  fp16 weights are 2^7 larger (up to 2^15, inside the type),
//   so that those down to 2^-21 of the largest stay above its subnormals.
// LDS rows are 16-byte chunks, chunk c of row r stored at c ^ f(r), so that
// both reads touch every bank once.
//
// A masked key has weight 0, but 0 times a V that is not finite is NaN: a wave
// whose sums are not all finite at the end looks for such values among the
// keys that some of its rows may not see (at most the last tiles'), and if
// there are any computes its rows again, one by one, with masked keys left out
// (a prompt of 8192 with one in its last key: 38 ms instead of 0.56; one that
// all rows see costs 0.1 ms).  Searching every tile with masked keys beforehand
// cost each prompt 1 to 2 us.
//
// What bounds it: 16.9 million MFMAs of 32 cycles each for a causal prompt of
// 8192 (32 heads over 8, 128 channels) are 220 us at 2.4 GHz, but with random
// data two waves per SIMD that issue nothing else run at 1.56 GHz (the power
// limit), 338 us, and with the 5 FMA-like instructions and the exp2 that go
// with each MFMA here, 393 us.  Measured 526 to 567 us on different cards, 970
// to 1046 TFLOP/s (1222 for a library GEMM of 8192^3); counters: MFMA busy
// 53 % of the cycles, no LDS bank conflict, 157 MB read from HBM for 100 MB of
// input.  Interleaving the next tile's scores with the weights by hand took
// the same time at a lower clock.  With one wave per SIMD a tile takes 3500
// cycles: scores 1160, weights 940, values 790, the next loads' issue and the
// barrier 580 (1024 tokens: 25 us so, 22 with two, see kHalvesKeys).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attention.hpp"
#include "common.hpp"
#include "mfma.hpp"

namespace paro {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void *lds_ptr;
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;

constexpr int kKeys = 64;  // keys per tile
// With at most this many workgroups of 128 rows the keys are split between the
// waves of smaller ones (see the SPLIT kernel).  Whole and split, us: 64 rows
// over 8064 cached keys (24 workgroups) 189 and 50, 256 over 8256 (72) 195 and
// 62; eight waves in halves (see kHalvesKeys) and split: 500 over 8500 (128) 139
// and 107, 400 over 1400 (104) 28 and 26, but 600 over 8600 (152) 142 and 155,
// and 8 x 30 over 60 (120) 6.7 and 8.3 (lengths are not known on the host).  A
// causal prompt's rows see half the keys: 256 (72) whole and split 9.9 and 9.4,
// 512 (136) 14.5 and 16.2.  One of one key tile has nothing to split (17 tokens:
// 5.8 us, 6.5 split).
constexpr int few_tiles(bool cached) { return cached ? 128 : 96; }
// With a workspace the parts of few rows' keys fill the 256 CUs once (one
// workgroup of the SPLIT kernel fits a CU), no part shorter than this: it is
// two tiles per wave, and joining costs 2 to 3 us (4 rows over 1000 keys, one
// part and two: 11.8 and 12.1 us; over 500, parts of 256: 9.0 and 10.9).  8 rows
// over 32768 keys 186 and 40 us, over 131072 1216 and 135, 64 over 8064 51 and
// 32.
constexpr int kPartKeys = 512;
constexpr int64_t kCus = 256;
// Workgroups of 128 rows have eight waves, in two halves that take the key
// tiles in turn, where there is about one of them per CU: alone there, four
// waves wait for their own results most of the time.  Four waves and eight, us:
// 1024 rows over 9024 cached keys (256 workgroups) 217 and 157, 16 x 64 over
// 4064 (256) 128 and 101, but 1500 over 5500 (368) 141 and 155.  A causal
// prompt's workgroups end at different times, so there up to two per CU: 2048
// tokens (512) 49.4 and 47.0, 2 x 1000 34.4 and 30.4, 2 x 2000 with 16 heads over
// 16 58.5 and 46; 2500 (624) 63 and 70.  Short sequences have no tiles to share:
// 2 x 700 20.6 and 21.1, 4 x 400 18.3 and 22.9.
constexpr int64_t kHalvesKeys = 768;

template <int DT>
__device__ __forceinline__ f32x16 mfma32x32x16(const u32x4 &a, const u32x4 &b, const f32x16 &c) {
  if constexpr (DT == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
}

// Two floats to the type, rounded to nearest even, by one instruction.
template <int DT>
__device__ __forceinline__ uint32_t pack2_rne(float lo, float hi) {
  if constexpr (DT == kF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// The chunk permutation of LDS row r (see the header).
template <int DIM>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (DIM == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
  else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// One sequence's part in a tile of rows.
struct Rows {
  int64_t q0;  // its first query row
  int64_t k0;  // its first key (packed)
  int n_q, n_k;
  int index;            // tile of BM rows within the sequence and head
  const int32_t *table; // cache
};

// The sequence of row tile t, by a scan of the sequences (ceil(n_q * group /
// BM) tiles each), 256 at a time, a lane taking four.  False: no such tile.
template <bool CACHED, int BM>
__device__ __forceinline__ bool find_tile(const AttentionArgs &a, int t, Rows &r) {
  const int lane = lane_id();
  const auto bound = [&](int s) {  // cu_q[s] in range; the end again past the last sequence
    const int64_t v = a.cu_q[min(s, a.sequences)];
    return (int)(v < 0 ? 0 : v > a.q_tokens ? a.q_tokens : v);
  };
  for (int s0 = 0; s0 < a.sequences; s0 += 256) {
    int tiles[4], q[5], ends = 0;
#pragma unroll
    for (int u = 0; u < 5; ++u) q[u] = bound(s0 + 4 * lane + u);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      tiles[u] = (max(q[u + 1] - q[u], 0) * a.group + BM - 1) / BM;
      ends += tiles[u];
    }
    int before = ends;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(ends, d, 64);
      if (lane >= d) ends += o;
    }
    before = ends - before;
    const uint64_t past = __ballot(ends > t);
    if (past) {
      const int j = __builtin_ctzll(past);
      int index = t - __builtin_amdgcn_readfirstlane(__shfl(before, j, 64)), u = 0;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int n = __builtin_amdgcn_readfirstlane(__shfl(tiles[i], j, 64));
        if (u == i && index >= n) {
          index -= n;
          ++u;
        }
      }
      const int sq = s0 + 4 * j + u, q0 = bound(sq);
      r.index = __builtin_amdgcn_readfirstlane(index);
      r.q0 = __builtin_amdgcn_readfirstlane(q0);
      r.n_q = __builtin_amdgcn_readfirstlane(bound(sq + 1) - q0);
      if constexpr (CACHED) {
        const int slot = a.slots[sq];
        r.n_k = __builtin_amdgcn_readfirstlane(a.kv.length(slot));
        r.table = a.kv.table + (int64_t)(r.n_k > 0 ? slot : 0) * a.kv.max_pages;
        r.k0 = 0;
      } else {
        const int64_t k0 = a.cu_k[sq] < 0 ? 0 : a.cu_k[sq];
        const int64_t k1 = a.cu_k[sq + 1] > a.k_tokens ? a.k_tokens : a.cu_k[sq + 1];
        r.n_k = __builtin_amdgcn_readfirstlane(k1 > k0 ? (int)(k1 - k0) : 0);
        r.k0 = __builtin_amdgcn_readfirstlane(k1 > k0 ? (int)k0 : 0);
        r.table = nullptr;
      }
      return true;
    }
    t -= __builtin_amdgcn_readfirstlane(__shfl(ends, 63, 64));
  }
  return false;
}

__device__ __forceinline__ int64_t page_base(const AttentionArgs &a, const Rows &r, int kvh, int dim, int64_t pos) {
  int page = r.table[pos >> a.kv.page_shift];
  page = page < 0 ? 0 : page >= a.kv.num_pages ? a.kv.num_pages - 1 : page;
  return (int64_t)page * a.kv.page_stride +
         (((int64_t)kvh << a.kv.page_shift) + (pos & ((1 << a.kv.page_shift) - 1))) * dim;
}

template <int DIM, bool CACHED>
__device__ __forceinline__ const uint16_t *v_row(const AttentionArgs &a, const Rows &r, int kvh, int j) {
  return CACHED ? a.kv.v + page_base(a, r, kvh, DIM, j) : a.v + (r.k0 + j) * a.v_token + kvh * a.v_head;
}

// Whether V holds a value that is not finite among the keys that a wave's rows
// had in their tiles (up to the end of the tile with key most - 1) and that not
// all of them see (from key least on).  A tile's rows past the sequence's end
// are zeros only as far as they lie behind its last row: where packed rows
// overlap (a token stride under DIM), they hold parts of the last rows, at most
// DIM / 8 of them, so those are searched too.
template <int DT, int DIM, bool CACHED>
__device__ __forceinline__ bool masked_not_finite(const AttentionArgs &a, const Rows &r, int kvh, int least, int most) {
  constexpr uint32_t kInf = DT == kF16 ? 0x7c00u : 0x7f80u;
  const int tiles_end = (most + kKeys - 1) / kKeys * kKeys, end = min(r.n_k, tiles_end);
  if (!CACHED && a.v_token < DIM && tiles_end > r.n_k) least = max(0, min(least, r.n_k - DIM / 8));
  bool bad = false;
  for (int j = least; j < end; ++j) {
    const uint16_t *v = v_row<DIM, CACHED>(a, r, kvh, j);
    for (int c = lane_id(); c < DIM; c += 64) bad |= (v[c] & kInf) == kInf;
  }
  return __any(bad);
}

// One row by one wave with masked keys left out: the way around values that
// are not finite.  Keys 64 at a time, lane j with key j's score; the output's
// channels lie over the lanes.
template <int DT, int DIM, bool CACHED>
__device__ __forceinline__ void row_by_wave(const AttentionArgs &a, const Rows &r, int kvh, int token,
                                                      int head) {
  const int lane = lane_id();
  const int64_t row = r.q0 + token;
  const int seen = a.causal ? min(r.n_k, token + 1 + r.n_k - r.n_q) : r.n_k;
  const uint16_t *q = a.q + row * a.q_token + head * a.q_head;
  float m = -INFINITY, l = 0.f, acc[DIM / 64] = {};
  for (int j0 = 0; j0 < seen; j0 += 64) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < seen) {
      const uint16_t *k = CACHED ? a.kv.k + page_base(a, r, kvh, DIM, j) : a.k + (r.k0 + j) * a.k_token + kvh * a.k_head;
      s = 0.f;
      for (int d = 0; d < DIM; d += 8) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(q + d), z = *reinterpret_cast<const u32x4 *>(k + d);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          s = fmaf(act_to_f32<DT>((uint16_t)(x[c >> 1] >> (16 * (c & 1)))),
                   act_to_f32<DT>((uint16_t)(z[c >> 1] >> (16 * (c & 1)))), s);
      }
      s *= a.scale;
    }
    float top = s;
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float p = j < seen ? expf(s - ref) : 0.f, keep = expf(m - ref);
    l = l * keep + p;
    m = mn;
    for (int c = 0; c < DIM / 64; ++c) acc[c] *= keep;
    const int n = min(64, seen - j0);
    for (int jj = 0; jj < n; ++jj) {
      const float w = __shfl(p, jj, 64);
      const uint16_t *v = v_row<DIM, CACHED>(a, r, kvh, j0 + jj);
      for (int c = 0; c < DIM / 64; ++c) acc[c] = fmaf(w, act_to_f32<DT>(v[c * 64 + lane]), acc[c]);
    }
  }
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, 64);
  uint16_t *y = a.y + row * a.y_token + head * a.y_head;
  for (int c = 0; c < DIM / 64; ++c)
    y[c * 64 + lane] = (uint16_t)(pack2<DT>(within_type<DT == kF16>(seen > 0 ? acc[c] / l : 0.f), 0.f) & 0xffffu);
}

// One wave instruction of 64 x 16 bytes into LDS.  As asm where a wave counts
// its own loads: for builtin loads the compiler makes every transposing LDS
// read wait for all that are in flight.  There is no output register, the
// tile loop waits by itself, and the wait states cover a descriptor or m0
// written just before.  m0 is named as written: the compiler keeps its own
// value there from one builtin load into LDS to the next.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register, which it warns of
__device__ __forceinline__ void load_lds(const uint16_t *base, uint32_t bytes, char *lds, uint32_t off) {
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr)lds);
  const uint64_t b = (uint64_t)base;
  const u32x4 r = {(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b),
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xffffu),
                   (uint32_t)__builtin_amdgcn_readfirstlane(bytes), (uint32_t)kRawBufferWord3};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(r)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// All but the last n of this wave's vector-memory operations have completed.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Loads of a tile's K and V into LDS, 1 KB (kRowsPer rows) per wave
// instruction; rows past the sequence's end are filled with zeros.  Packed
// tiles are one buffer; in the cache a buffer is up to 16 rows, which lie in
// one page, and the page's index is looked up a tile ahead.
template <int DIM, bool CACHED, int NW, int KEYS>
struct Loader {
  static constexpr int kRowsPer = 512 / DIM;
  static constexpr int kLoads = KEYS * DIM * 2 / 1024 / NW;  // per wave and tile, NW waves sharing it
  static constexpr int kRowStep = kRowsPer * NW;             // rows between a wave's loads
  static constexpr int kPerBuffer = !CACHED ? kLoads : kRowStep < 16 ? 16 / kRowStep : 1;
  static constexpr int kBuffers = kLoads / kPerBuffer;
  const uint16_t *k, *v;      // packed: the head's first key; cache: the head in page 0
  uint32_t k_off[kPerBuffer], v_off[CACHED ? 1 : kPerBuffer];  // this lane's byte offsets in a buffer
  int pages[kBuffers];

  __device__ __forceinline__ void init(const AttentionArgs &a, const Rows &r, int kvh, int j0, int wave, int lane) {
    constexpr int kChunks = DIM / 8;
    const int64_t in_page = ((int64_t)kvh << a.kv.page_shift) * DIM;
    k = CACHED ? a.kv.k + in_page : a.k + r.k0 * a.k_token + kvh * a.k_head;
    v = CACHED ? a.kv.v + in_page : a.v + r.k0 * a.v_token + kvh * a.v_head;
#pragma unroll
    for (int n = 0; n < kPerBuffer; ++n) {
      const int row = wave * kRowsPer + n * kRowStep + lane / kChunks;
      const int chunk = ((lane % kChunks) ^ swizzle<DIM>(row)) * 16;
      if constexpr (CACHED) {
        k_off[n] = (uint32_t)((n * kRowStep + lane / kChunks) * DIM * 2 + chunk);
      } else {
        k_off[n] = (uint32_t)(row * a.k_token * 2 + chunk);
        v_off[n] = (uint32_t)(row * a.v_token * 2 + chunk);
      }
    }
    if constexpr (CACHED) look_up(a, r, j0, wave);
  }
  __device__ __forceinline__ void look_up(const AttentionArgs &a, const Rows &r, int j0, int wave) {
#pragma unroll
    for (int b = 0; b < kBuffers; ++b)
      pages[b] = r.table[min(j0 + wave * kRowsPer + b * kPerBuffer * kRowStep, r.n_k - 1) >> a.kv.page_shift];
  }
  // first element of buffer b's rows in the tile at key j0, and the bytes of its K or V rows there are
  __device__ __forceinline__ int64_t buffer_at(const AttentionArgs &a, int j0, int b, int wave) const {
    if constexpr (!CACHED) return j0;  // in keys
    const int row = j0 + wave * kRowsPer + b * kPerBuffer * kRowStep;
    const int page = min(max(pages[b], 0), a.kv.num_pages - 1);
    return page * a.kv.page_stride + (row & ((1 << a.kv.page_shift) - 1)) * DIM;
  }
  __device__ __forceinline__ uint32_t buffer_bytes(const Rows &r, int j0, int b, int wave, int64_t token) const {
    const int left = CACHED ? min(kPerBuffer == 1 ? kRowsPer : 16, r.n_k - (j0 + wave * kRowsPer + b * kPerBuffer * kRowStep))
                            : min(KEYS, r.n_k - j0);
    return left > 0 ? (uint32_t)((left - 1) * (CACHED ? DIM : token) * 2 + DIM * 2) : 0u;
  }
  // the tile at key j0 (after look_up of it), and the look-up of the one at key next
  __device__ __forceinline__ void load(const AttentionArgs &a, const Rows &r, int j0, int next, char *to_k, char *to_v,
                                       int wave) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know the buffer type
#pragma unroll
    for (int b = 0; b < kBuffers; ++b) {
      const int64_t at = buffer_at(a, j0, b, wave);
      const __amdgpu_buffer_rsrc_t rk =
          raw_rsrc(k + (CACHED ? at : at * a.k_token), buffer_bytes(r, j0, b, wave, a.k_token));
      const __amdgpu_buffer_rsrc_t rv =
          raw_rsrc(v + (CACHED ? at : at * a.v_token), buffer_bytes(r, j0, b, wave, a.v_token));
#pragma unroll
      for (int n = 0; n < kPerBuffer; ++n) {
        const int to = 1024 * (wave + NW * (b * kPerBuffer + n));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (lds_ptr)(to_k + to), 16, k_off[n], 0, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (lds_ptr)(to_v + to), 16, CACHED ? k_off[n] : v_off[n], 0, 0, 0);
      }
    }
    if constexpr (CACHED) look_up(a, r, next, wave);
#endif
  }
  // K or V alone by asm loads (kLoads of them)
  template <bool V>
  __device__ __forceinline__ void load_one(const AttentionArgs &a, const Rows &r, int j0, char *to) {
#pragma unroll
    for (int b = 0; b < kBuffers; ++b) {
      const int64_t at = buffer_at(a, j0, b, 0), token = V ? a.v_token : a.k_token;
      const uint16_t *base = (V ? v : k) + (CACHED ? at : at * token);
      const uint32_t bytes = buffer_bytes(r, j0, b, 0, token);
#pragma unroll
      for (int n = 0; n < kPerBuffer; ++n)
        load_lds(base, bytes, to + 1024 * (b * kPerBuffer + n), V && !CACHED ? v_off[n] : k_off[n]);
    }
  }
};

// What a workgroup of the SPLIT kernel has of its rows' keys, and where the
// parts of other workgroups meet (parts == 1: nowhere).
struct Part {
  int index, parts;
  float *sums;        // the parts of these rows: [parts][32][DIM + 4]
  uint32_t *counter;  // workgroups that have stored theirs; zero between calls
};
// Two floats that another XCD will read or wrote: past the L2s.
__device__ __forceinline__ void store_coherent(float *p, float x, float y) {
  __hip_atomic_store(reinterpret_cast<uint64_t *>(p), (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 load_coherent(const float *p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return f32x2{__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))};
}

// Joins the waves' sums of the same 32 rows (each relative to its own m2, the
// maximum times scale2) and writes the rows: thread (row, 8 channels).  Where
// the keys are in parts, each workgroup stores its joined sums and the last one
// to arrive joins them, in their order.
template <int DT, int DIM, bool CACHED, int NW, bool PARTS>
__device__ __forceinline__ void join_waves(const AttentionArgs &a, const Rows &r, int kvh, int base, int rows,
                                           int least, int most, const f32x16 (&o)[DIM / 32], float m2, float l,
                                           float *lds, const Part &part) {
  constexpr int RS = DIM + 4;  // row of sums: its channels, then m2 and l
  const int lane = lane_id(), wave = wave_id(), h = lane >> 5, col = lane & 31;
  __syncthreads();  // every wave is done with its tiles
  float *mine = lds + (wave * 32 + col) * RS;
#pragma unroll
  for (int db = 0; db < DIM / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<f32x4 *>(mine + 32 * db + 2 * i + 4 * h) =
          f32x4{o[db][i], o[db][i + 1], o[db][i + 2], o[db][i + 3]};
  if (h == 0) {
    mine[DIM] = m2;
    mine[DIM + 1] = l;
  }
  __syncthreads();
  bool bad = false;
  const auto write = [&](int row, int c, f32x4 x0, f32x4 x1, float sum) {
    const int token = (base + row) / a.group, head = kvh * a.group + (base + row) % a.group;
    const bool any = r.n_k > 0 && (!a.causal || token + 1 + r.n_k - r.n_q > 0);
    const float inv = any ? 1.f / sum : 0.f;
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x0[i] *= inv;
      x1[i] *= inv;
      worst = __builtin_fmaf(x0[i], 0.f, __builtin_fmaf(x1[i], 0.f, worst));
    }
    bad |= worst != 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x0[i] = within_type<DT == kF16>(x0[i]);
      x1[i] = within_type<DT == kF16>(x1[i]);
    }
    const u32x4 y = {pack2_rne<DT>(x0[0], x0[1]), pack2_rne<DT>(x0[2], x0[3]), pack2_rne<DT>(x1[0], x1[1]),
                     pack2_rne<DT>(x1[2], x1[3])};
    *reinterpret_cast<u32x4 *>(a.y + (r.q0 + token) * a.y_token + head * a.y_head + c) = any ? y : u32x4{0, 0, 0, 0};
  };
  for (int e = threadIdx.x; e < 32 * DIM / 8; e += 64 * NW) {
    const int row = e / (DIM / 8), c = e % (DIM / 8) * 8;
    if (base + row >= rows) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, lds[(w * 32 + row) * RS + DIM]);
    float sum = 0.f;
    f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0;
#pragma unroll 2
    for (int w = 0; w < NW; ++w) {
      const float *from = lds + (w * 32 + row) * RS;
      const float keep = from[DIM] == top ? 1.f : __builtin_amdgcn_exp2f(from[DIM] - top);
      sum += keep * from[DIM + 1];
      x0 += keep * *reinterpret_cast<const f32x4 *>(from + c);
      x1 += keep * *reinterpret_cast<const f32x4 *>(from + c + 4);
    }
    if (!PARTS || part.parts == 1) {
      write(row, c, x0, x1, sum);
    } else {
      float *to = part.sums + ((int64_t)part.index * 32 + row) * RS;
      store_coherent(to + c, x0[0], x0[1]);
      store_coherent(to + c + 2, x0[2], x0[3]);
      store_coherent(to + c + 4, x1[0], x1[1]);
      store_coherent(to + c + 6, x1[2], x1[3]);
      if (c == 0) store_coherent(to + DIM, top, sum);
    }
  }
  if (PARTS && part.parts > 1) {
    __builtin_amdgcn_s_waitcnt(0);  // this thread's sums have been stored
    __syncthreads();
    int *last = reinterpret_cast<int *>(lds);
    if (threadIdx.x == 0) {
      const uint32_t old = __hip_atomic_fetch_add(part.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *last = old == (uint32_t)(part.parts - 1);
    }
    __syncthreads();
    if (!*last) return;
    for (int e = threadIdx.x; e < 32 * DIM / 8; e += 64 * NW) {
      const int row = e / (DIM / 8), c = e % (DIM / 8) * 8;
      if (base + row >= rows) continue;
      float top = -INFINITY, sum = 0.f;
      f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0;
#pragma unroll 4
      for (int i = 0; i < part.parts; ++i) {
        const float *from = part.sums + ((int64_t)i * 32 + row) * RS;
        const f32x2 ml = load_coherent(from + DIM), y0 = load_coherent(from + c), y1 = load_coherent(from + c + 2),
                    y2 = load_coherent(from + c + 4), y3 = load_coherent(from + c + 6);
        const float mn = fmaxf(top, ml[0]);
        const float ka = top == mn ? 1.f : __builtin_amdgcn_exp2f(top - mn),
                    kb = ml[0] == mn ? 1.f : __builtin_amdgcn_exp2f(ml[0] - mn);
        top = mn;
        sum = sum * ka + ml[1] * kb;
        x0 = x0 * ka + f32x4{y0[0], y0[1], y1[0], y1[1]} * kb;
        x1 = x1 * ka + f32x4{y2[0], y2[1], y3[0], y3[1]} * kb;
      }
      write(row, c, x0, x1, sum);
    }
    if (threadIdx.x == 0) __hip_atomic_store(part.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // tiles are 32 keys here, the search's 64: it may find a value that no tile held
  if (__syncthreads_or(bad) && masked_not_finite<DT, DIM, CACHED>(a, r, kvh, least, most)) {
#pragma unroll 1
    for (int i = wave; i < 32 && base + i < rows; i += NW)
      row_by_wave<DT, DIM, CACHED>(a, r, kvh, (base + i) / a.group, kvh * a.group + (base + i) % a.group);
  }
}

// SPLIT: the waves share 32 rows and take tiles of 32 keys in turn, each with
// LDS buffers of its own (one for K, one for V, so that twice as many waves
// fit: the next K is loaded once the scores are formed, the next V once the
// values are summed); their sums are joined at the end.  PARTS: the keys go to
// gridDim.z workgroups first (apart, since the one more range costs the SPLIT
// kernel registers: 64 rows over 8064 keys 58 instead of 50 us).
template <int DT, int DIM, bool CACHED, int NW, bool SPLIT, bool PARTS>
__global__ void __launch_bounds__(64 * NW, 2) prompt_attention_kernel(AttentionArgs a, int row_tiles,
                                                                      uint32_t *counters, float *sums) {
  constexpr bool HALVES = !SPLIT && NW == 8;  // waves 0..3 and 4..7 take tiles in turn
  constexpr int BM = SPLIT ? 32 : 128, KS = DIM / 16, DB = DIM / 32;
  constexpr int KEYS = SPLIT ? 32 : kKeys, KB = KEYS / 32;
  constexpr int kTileBytes = KEYS * DIM * 2;
  constexpr int kBuffers = SPLIT ? 1 : 2;  // of K, then of V
  constexpr int kJoinBytes = SPLIT ? NW * 32 * (DIM + 4) * 4 : 0, kAllBytes = (SPLIT ? NW : NW / 4) * 2 * kBuffers * kTileBytes;
  __shared__ __align__(1024) char all_lds[kJoinBytes > kAllBytes ? kJoinBytes : kAllBytes];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  const int h = lane >> 5, col = lane & 31;
  const int half = HALVES ? wave / 4 : 0;
  char *const lds = all_lds + (SPLIT ? wave * 2 : half * 4) * kTileBytes;
  const int stride = SPLIT ? NW * KEYS : NW / 4 * KEYS;  // between this wave's tiles
  const int share = SPLIT ? 0 : wave - 4 * half;          // of a tile's loads and rows
  // key-value heads next to each other in the launch order: workgroups go to
  // the XCDs in turn, so with 8 heads each XCD's L2 holds one head's K and V;
  // the longest tiles (a sequence's last) first
  const int kvh = (int)(blockIdx.x % a.kv_heads);
  const int t = row_tiles - 1 - (int)(blockIdx.x / a.kv_heads);
  Rows r;
  if (!find_tile<CACHED, BM>(a, t, r)) return;
  const int rows = r.n_q * a.group;  // rows of the sequence and key-value head
  const int base = r.index * BM + 32 * share;
  const int mine = min(base + col, rows - 1);  // rows past the end repeat the last one and are not stored
  const int token = mine / a.group, head = kvh * a.group + mine % a.group;
  const int shift = r.n_k - r.n_q;
  // keys that a row sees, and the fewest and most of the wave's and the workgroup's rows
  const auto seen_by = [&](int row) {
    const int n = a.causal ? min(r.n_k, row / a.group + 1 + shift) : r.n_k;
    return max(n, 0);
  };
  const int seen = seen_by(mine);
  const int wave_least = seen_by(min(base, rows - 1)), wave_most = seen_by(min(base + 31, rows - 1));
  const int most = __builtin_amdgcn_readfirstlane(seen_by(min((r.index + 1) * BM, rows) - 1));
  // this workgroup's part of the keys, and this wave's first tile
  int begin = SPLIT ? wave * KEYS : half * KEYS, end = most, keys = 0;
  if constexpr (PARTS) {
    const int splits = (int)gridDim.z, index = (int)blockIdx.z;
    keys = max(kPartKeys, ((most + splits - 1) / splits + stride - 1) / stride * stride);
    if (index > 0 && index * keys >= most) return;
    begin += index * keys;
    end = min(most, index * keys + keys);
  }

  // Q^T fragments: row lane%32, channels 16 s + 8 h..; a negative scale goes to Q
  u32x4 q[KS];
  {
    const uint16_t *qp = a.q + (r.q0 + token) * a.q_token + head * a.q_head + 8 * h;
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      q[s] = *reinterpret_cast<const u32x4 *>(qp + 16 * s);
#pragma unroll
      for (int c = 0; c < 4; ++c) q[s][c] ^= flip;
    }
  }
  // not zero (0 times the -infinity of a masked score is NaN), but so small that no finite product matters
  const float scale2 = fmaxf(fabsf(a.scale) * 1.44269504088896340736f, 0x1p-149f);

  // LDS addresses: K fragment s at k_at[s] (+ 32 rows), V^T fragment (db, half) at v_at (+ 16 rows per step)
  uint32_t k_at[KS], v_at[DB][2];
#pragma unroll
  for (int s = 0; s < KS; ++s) k_at[s] = (uint32_t)(col * DIM * 2 + (((2 * s + h) ^ swizzle<DIM>(col)) << 4));
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 8 * u + 4 * h + ((lane >> 2) & 3);
      const int chunk = 4 * db + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
      v_at[db][u] = (uint32_t)(kBuffers * kTileBytes + row * DIM * 2 + ((chunk ^ swizzle<DIM>(row)) << 4) + 8 * (lane & 1));
    }

  f32x16 o[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[db][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  Loader<DIM, CACHED, SPLIT ? 1 : 4, KEYS> loader;
  if (begin < end) {
    loader.init(a, r, kvh, begin, share, lane);
    if constexpr (SPLIT) {
      loader.template load_one<false>(a, r, begin, lds);
      loader.template load_one<true>(a, r, begin, lds + kTileBytes);
      if constexpr (CACHED) loader.look_up(a, r, begin + stride, share);
    } else {
      loader.load(a, r, begin, begin + stride, lds, lds + 2 * kTileBytes, share);
    }
  }
  const auto step = [&](int j0, auto which) __attribute__((always_inline)) {
    constexpr int buf = decltype(which)::value;
    const bool more = j0 + stride < end;
    if constexpr (SPLIT) {
      wait_loads<decltype(loader)::kLoads>();  // K has landed; V may be on its way
    } else {
      // this tile has landed, and every wave is done with the other buffer
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (more)
        loader.load(a, r, j0 + stride, j0 + 2 * stride, lds + (buf ^ 1) * kTileBytes,
                    lds + (2 + (buf ^ 1)) * kTileBytes, share);
    }
    if (!SPLIT && j0 >= wave_most) return;  // no row of this wave sees the tile
    const char *tile = lds + buf * kTileBytes;
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const u32x4 k = *reinterpret_cast<const u32x4 *>(tile + k_at[x] + kb * 32 * DIM * 2);
        s[kb] = mfma32x32x16<DT>(k, q[x], s[kb]);
      }
    if constexpr (SPLIT) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // K has been read
      if (more) loader.template load_one<false>(a, r, j0 + stride, lds);
    }
    if (j0 + KEYS > wave_least) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j0 + 32 * kb + 8 * (i >> 2) + 4 * h + (i & 3) >= seen) s[kb][i] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
    {
      const uint32_t u = __float_as_uint(top);
      const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      top = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
    }
    // true too where m is still -infinity and top is not
    if (__any((top - m) * scale2 > 8.f)) {
      const float mn = fmaxf(m, top);
      const float keep = m == mn ? 1.f : __builtin_amdgcn_exp2f((m - mn) * scale2);
      m = mn;
      l *= keep;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] *= keep;
    }
    const float ref = m == -INFINITY ? 0.f : m * scale2 - (DT == kF16 ? 7.f : 0.f);
    u32x4 p[2 * KB];
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], scale2, -ref));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i + 1], scale2, -ref));
        sums[(i >> 1) & 3] += e0 + e1;
        p[2 * kb + (i >> 3)][(i & 7) >> 1] = pack2_rne<DT>(e0, e1);
      }
    l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
    if constexpr (SPLIT) {  // V has landed; the next K may be on its way
      if (more) wait_loads<decltype(loader)::kLoads>();
      else wait_loads<0>();
    }
#pragma unroll
    for (int ks = 0; ks < 2 * KB; ++ks)
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        const char *vt = tile + ks * 16 * DIM * 2;
        const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(vt + v_at[db][0]));
        const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(vt + v_at[db][1]));
        const u32x2 w0 = __builtin_bit_cast(u32x2, v0), w1 = __builtin_bit_cast(u32x2, v1);
        o[db] = mfma32x32x16<DT>(u32x4{w0[0], w0[1], w1[0], w1[1]}, p[ks], o[db]);
      }
    if constexpr (SPLIT) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // V has been read
      if (more) {
        loader.template load_one<true>(a, r, j0 + stride, lds + kTileBytes);
        if constexpr (CACHED) loader.look_up(a, r, j0 + 2 * stride, share);
      }
    }
  };
  if constexpr (SPLIT) {
    for (int j0 = begin; j0 < end; j0 += stride) step(j0, std::integral_constant<int, 0>());
  } else {
    // (with halves both take as many steps, since they meet at each one's barrier)
    for (int j0 = 0; j0 < most; j0 += 2 * stride) {
      step(j0 + begin, std::integral_constant<int, 0>());
      if (j0 + stride < most) step(j0 + stride + begin, std::integral_constant<int, 1>());
    }
  }

  {
    const uint32_t u = __float_as_uint(l);
    const auto w = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    l = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
  if constexpr (SPLIT) {
    Part part = {0, 1, nullptr, nullptr};
    if constexpr (PARTS) {
      part.index = (int)blockIdx.z;
      part.parts = max(1, (most + keys - 1) / keys);
      part.sums = sums + (int64_t)blockIdx.x * gridDim.z * 32 * (DIM + 4);
      part.counter = counters + blockIdx.x;
    }
    join_waves<DT, DIM, CACHED, NW, PARTS>(a, r, kvh, base, rows, wave_least, wave_most, o, m * scale2, l, reinterpret_cast<float *>(all_lds),
                                     part);
    return;
  }
  if constexpr (HALVES) {
    // the second half's sums come to the first, lane for lane
    __syncthreads();
    float *const at = reinterpret_cast<float *>(all_lds) + share * (DIM / 2 + 2) * 64;
    if (half) {
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<f32x4 *>(at + ((4 * db + i / 4) * 64 + lane) * 4) =
              f32x4{o[db][i], o[db][i + 1], o[db][i + 2], o[db][i + 3]};
      at[DIM / 2 * 64 + lane] = m * scale2;
      at[(DIM / 2 + 1) * 64 + lane] = l;
    }
    __syncthreads();
    if (half) return;
    const float m1 = at[DIM / 2 * 64 + lane], m0 = m * scale2, top = fmaxf(m0, m1);
    const float k0 = m0 == top ? 1.f : __builtin_amdgcn_exp2f(m0 - top), k1 = m1 == top ? 1.f : __builtin_amdgcn_exp2f(m1 - top);
    l = l * k0 + at[(DIM / 2 + 1) * 64 + lane] * k1;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(at + ((4 * db + i / 4) * 64 + lane) * 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[db][i + c] = o[db][i + c] * k0 + x[c] * k1;
      }
  }
  const bool stored = base + col < rows;
  const float inv = seen > 0 ? 1.f / l : 0.f;
  float worst = 0.f;  // NaN as soon as one value is not finite (x * 0 is NaN then)
  float most_f16 = 0.f;
  uint16_t *y = a.y + (r.q0 + token) * a.y_token + head * a.y_head + 8 * h;
  const auto store = [&](auto clamped) __attribute__((always_inline)) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int n = 0; n < 2; ++n) {  // channels 32 db + 16 n: half h holds 4 h.. and 8 + 4 h..
        uint32_t w[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x0 = o[db][8 * n + 4 * u + 2 * c] * inv, x1 = o[db][8 * n + 4 * u + 2 * c + 1] * inv;
            if constexpr (decltype(clamped)::value) {
              x0 = within_type<true>(x0);
              x1 = within_type<true>(x1);
            } else {
              worst = __builtin_fmaf(x0, 0.f, worst);
              worst = __builtin_fmaf(x1, 0.f, worst);
              if constexpr (DT == kF16) most_f16 = fmaxf(most_f16, fmaxf(fabsf(x0), fabsf(x1)));
            }
            w[u][c] = seen > 0 ? pack2_rne<DT>(x0, x1) : 0u;
          }
        // lanes 0..31 take the lower 8 channels of their row, lanes 32..63 the upper
        const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        if (stored) *reinterpret_cast<u32x4 *>(y + 32 * db + 16 * n) = u32x4{lo[0], hi[0], lo[1], hi[1]};
      }
  };
  store(std::false_type());
  // other rows pay one instruction for two values (17 tokens 5.7 -> 5.9 us, 8192 527 and 528)
  if (DT == kF16 && __any(stored && most_f16 > kMaxF16)) store(std::true_type());
  if (__any(stored && worst != 0.f) && masked_not_finite<DT, DIM, CACHED>(a, r, kvh, wave_least, wave_most)) {
#pragma unroll 1
    for (int i = 0; i < 32 && base + i < rows; ++i)
      row_by_wave<DT, DIM, CACHED>(a, r, kvh, (base + i) / a.group, kvh * a.group + (base + i) % a.group);
  }
}

// Workgroups of `rows` rows that sequences of so many tokens in all take at most, per key-value head.
int64_t row_tiles(int64_t q_tokens, int64_t sequences, int group, int rows) {
  return q_tokens * group / rows + sequences;
}

template <int DT, int DIM, bool CACHED>
hipError_t launch_typed(const AttentionArgs &a, int splits, uint32_t *counters, float *sums, hipStream_t st) {
  const int64_t tiles = row_tiles(a.q_tokens, a.sequences, a.group, 128);
  if (tiles * a.kv_heads <= few_tiles(CACHED) && (CACHED || a.k_tokens > kKeys)) {
    constexpr int SW = 8;
    const int64_t small = row_tiles(a.q_tokens, a.sequences, a.group, 32);
    const dim3 grid((unsigned)(small * a.kv_heads), 1, (unsigned)splits), block(64 * SW);
    if constexpr (CACHED) {
      if (splits > 1) {
        hipLaunchKernelGGL((prompt_attention_kernel<DT, DIM, CACHED, SW, true, true>), grid, block, 0, st, a,
                           (int)small, counters, sums);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((prompt_attention_kernel<DT, DIM, CACHED, SW, true, false>), grid, block, 0, st, a, (int)small,
                       counters, sums);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(tiles * a.kv_heads));
  const bool few = row_tiles(a.q_tokens, 0, a.group, 128) * a.kv_heads <= (CACHED || !a.causal ? 1 : 2) * kCus;
  if (few && (CACHED || a.k_tokens >= a.sequences * kHalvesKeys))
    hipLaunchKernelGGL((prompt_attention_kernel<DT, DIM, CACHED, 8, false, false>), grid, dim3(512), 0, st, a,
                       (int)tiles, nullptr, nullptr);
  else
    hipLaunchKernelGGL((prompt_attention_kernel<DT, DIM, CACHED, 4, false, false>), grid, dim3(256), 0, st, a,
                       (int)tiles, nullptr, nullptr);
  return hipGetLastError();
}

template <bool CACHED>
hipError_t launch(const AttentionArgs &a, int splits, uint32_t *counters, float *sums, hipStream_t st) {
  if (a.dt == kF16)
    return a.head_dim == 64 ? launch_typed<kF16, 64, CACHED>(a, splits, counters, sums, st)
                            : launch_typed<kF16, 128, CACHED>(a, splits, counters, sums, st);
  return a.head_dim == 64 ? launch_typed<kBF16, 64, CACHED>(a, splits, counters, sums, st)
                          : launch_typed<kBF16, 128, CACHED>(a, splits, counters, sums, st);
}

}  // namespace

int attention_prompt_splits(int64_t q_tokens, int64_t sequences, int q_heads, int kv_heads, int64_t max_len) {
  const int group = q_heads / kv_heads;
  if (row_tiles(q_tokens, sequences, group, 128) * kv_heads > few_tiles(true)) return 1;
  const int64_t items = row_tiles(q_tokens, sequences, group, 32) * kv_heads;
  return (int)std::max<int64_t>(1, std::min(kCus / items, (max_len + kPartKeys - 1) / kPartKeys));
}

size_t attention_prompt_partial_bytes(int splits, int64_t q_tokens, int64_t sequences, int q_heads, int kv_heads,
                                      int head_dim) {
  if (splits == 1) return 0;
  return (size_t)row_tiles(q_tokens, sequences, q_heads / kv_heads, 32) * kv_heads * splits * 32 * (head_dim + 4) * 4;
}

hipError_t launch_attention_prompt(const AttentionArgs &a, bool cached, int splits, uint32_t *counters, float *sums,
                                   hipStream_t st) {
  return cached ? launch<true>(a, splits, counters, sums, st) : launch<false>(a, 1, nullptr, nullptr, st);
}

}  // namespace paro
