// attention_decode4.hip - attention of one new token per sequence over a paged
// cache in four bits (paro_attention_decode with PARO_KV4_F16 / PARO_KV4_BF16).
//
// A key is k_c = low_u + s_u * code_c, u = c / 64 its group, so
//   q . k = sum_u ( s_u * sum_{c in u} q_c code_c  +  low_u * sum_{c in u} q_c ):
// the matrix cores multiply by the codes and the pairs come in afterwards, in
// fp32.  For the values, with weights p_j = exp(score_j - max) and
// mid_u = low_u + 8 s_u,
//   sum_j p_j v_jc = sum_j (p_j s_ju) (code_jc - 8)  +  sum_j p_j mid_ju:
// the first sum runs on the matrix cores with p s rounded to fp16, the second in
// fp32.  The 8 is taken off the operand: with products of one sign the matrix
// cores' sums come out low by about 2^-18 of their terms, which in a row of
// 100000 keys, whose terms cancel, was twice the rounding of an fp16 output
// (taken off after the product, by a second one or by the sum of the weights:
// 2.5 times further from the exact values).
//   - Codes are made operands by one AND: the bits 0..3 (or 4..7) of a 16-bit
//     half are the fp16 number code * 2^-24 (16 code * 2^-24), a subnormal, which
//     the matrix cores take as it is.  Queries are scaled to fp16 by a power of
//     two of their row's, those that meet bits 4..7 by 1/16 of it.
//   - The layout of the pages (include/paro.h) is the order of the operands: a
//     lane's 16 bytes of K are its share of one key's channels for every
//     contraction step, its 16 bytes of V four keys of eight channels.
//   - The first product has the key in lane % 16 and heads in its registers, so
//     that a lane has the pairs of its own keys only: each lane loads one key's
//     pairs of K or of V, and swaps of lane halves and quarters spread them.  The
//     second has the head in lane % 16; the weights change places in LDS.
//   - Running maximum m of score * log2 e, moved when one is more than kSlack over
//     it, and sum of the weights, both fp32.
//   - What is rounded to fp16 is p s 2^(kTop - ev), with 2^ev over the p s of a
//     head and 64 channels so far: off by 2^-11 of itself, or by 2^-(22 + kTop) of
//     the largest of them.  An ev over the scales alone would lose every other key to
//     one that has a huge scale and no weight.
// Work is dealt out in units (kUnit keys of an output, an output being a row and
// up to 16 query heads of a key-value head), so that the 512 workgroups that the
// card holds end together whatever the rows' lengths are.  A workgroup's four waves
// share an output and join their sums; where there are many short ones each wave
// takes outputs of its own, with nothing to join.  See kOutputUnits, kLoneShare and
// plan_attention_decode4.
// What bounds it, with 8 key-value heads of 128 channels and 32 query heads: where
// rows are long the bytes, 9/8 per key and channel (9/32 of the 16-bit cache's).
// Two rows of 131072 and 100001 keys (266 MB) take 66 us, 64 rows of up to 4096 (141
// MB) 40, with caches in turn whose bytes together are past the last-level cache's
// 256 MB: 4.8 TB/s, as a copy, and about 10 us of start, join and uneven ends.  On
// the same cache again, which that cache then holds in part, 52 to 59 and 33 to 36.
// With 8, 16 heads per key-value head the 64 rows take 35, 44 us where 4 take 32:
// the vector instructions of the weights.  One row of 777 keys, 8 outputs over 56
// workgroups of one step each, 8.2 us: slot and length 1.2, table 1.0, queries and
// first keys 0.7, the step 1.3, a part stored and counted 1.3, the parts joined 1.6,
// the rest a launch.  One row of 131072 36 us: 64 parts an output.
// Both sides of the choices, us, on the same cache again, when each was made:
//   - two workgroups per CU and one: 37 and 52 (64 rows), 59 and 77 (two rows);
//     three: 43 and 67, the registers of two tiles and the sums no longer fit.
//   - a ring of two tiles and of three: 37.4 and 37.6, 59.2 and 60.4.
//   - the younger workgroup of a CU ahead in every other step (s_setprio), and
//     never: 37.4 and 38.5, 59.3 and 60.6.  The older one's waves go first
//     otherwise, and ended after 41 us of a 51 us loop.
//   - a lane with the pairs of its own four keys loaded, and spread by swaps from
//     one load: the same time.
//   - heads in every fourth row of the first product's operand, N registers of
//     them, and four registers whatever the heads: 37.4 and 39.2, 300 rows of up
//     to 1000 47 and 50.4.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attention.hpp"
#include "attention_join.hpp"
#include "common.hpp"
#include "kv4.hpp"
#include "mfma.hpp"

namespace paro {
namespace {

constexpr int kStep = 32;                    // keys per wave and step
constexpr int kUnit = kStep * kDecodeWaves;  // keys per workgroup and step
// What an output costs beside its steps, in steps: its start and its end (0, 3
// and 6: 47.5, 37.4 and 39.2 us for 64 rows of up to 4096, 62, 47 and 50.5 for 300
// of up to 1000; 2 and 4 as 3).
constexpr int kOutputUnits = 3;
// Waves have outputs of their own where there are more outputs than workgroups and
// the longest has at most two thirds of the units of a wave's share.  Shared by
// four waves and one each, us: 300 rows of up to 300 keys 33 and 25, 1000 of up to
// 500 104 and 91, 1000 of 500 148 and 121; but 300 of up to 1000 (longest 8, share
// 9) 46 and 52.
constexpr uint32_t kLoneShare = 2, kLoneLongest = 3;
constexpr int kTiles = 2;                    // of a wave's ring
// The maxima move when a weight is over 2^kSlack: with 3, 4 and 5 64 rows of up to
// 4096 keys take 32.6, 32.2 and 32.1 us with 4 heads per key-value head, 45.6, 43.9
// and 42.5 with 16, and two rows of 131072 and 100001 keys in fp16 are off by 2.49,
// 2.51 and 2.54e-4 (the largest weight is 1 just after a move, and then exact).
constexpr float kSlack = 4.f;
constexpr int kTop = 8;                      // weights times scales are under 2^kTop in fp16 when their exponent is set,
constexpr float kMost = 0x1p15f;             // and under this afterwards
constexpr float kLeastMaximum = -3e38f;      // scores that fp32 does not hold weigh nothing, also among themselves
constexpr int kLeastExponent = -110;         // of a weight times a scale: 2^(kTop - ev) is one fp32 number

template <int N>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N)));
};

// 32 keys: a lane's codes of K and V, [16-key block], and one key's pairs: key
// lane % 16 of K's first and second block (lanes 0.., 16..) and of V's.
template <int DIM>
struct Tile {
  typedef typename Words<DIM / 32>::type Codes;
  Codes k[2], v[2];
  typename Words<DIM / 64>::type pairs;
};

// Where a wave's keys lie: byte offsets, in a layer's K or V, of the codes of 16
// consecutive positions (they lie in one page).  They are looked up for 32 steps
// at a time, a lane for each 16-key block, so that no step waits for the table.
template <int DIM>
struct Window {
  uint32_t low, high;  // of this lane's block
  __device__ __forceinline__ void look_up(const int32_t *__restrict__ table, int64_t page_bytes, int64_t head_offset,
                                          int last, int num_pages, int shift, int pos, int stride, int lane) {
    const int p = pos + stride * (lane >> 1) + 16 * (lane & 1);
    int page = table[min(p >> shift, last)];
    page = page < 0 ? 0 : page >= num_pages ? num_pages - 1 : page;
    const int64_t at = (int64_t)page * page_bytes + head_offset + (p & ((1 << shift) - 1)) * Kv4<DIM>::kRow;
    low = (uint32_t)at;
    high = (uint32_t)(at >> 32);
  }
  __device__ __forceinline__ int64_t block(int i) const {
    const uint32_t l = __builtin_amdgcn_readlane(low, i), h = __builtin_amdgcn_readlane(high, i);
    return (int64_t)((uint64_t)h << 32 | l);
  }
};

// The pairs of key lane % 16 for every lane, [block].
template <int DIM>
struct Pairs {
  uint32_t k[2][DIM / 64], v[2][DIM / 64];
};
template <int DIM>
__device__ __forceinline__ Pairs<DIM> spread(const typename Words<DIM / 64>::type &p) {
  Pairs<DIM> out;
#pragma unroll
  for (int u = 0; u < DIM / 64; ++u) {
    const auto half = __builtin_amdgcn_permlane32_swap(p[u], p[u], false, false);  // lanes 0..31, 32..63 twice
    const auto k = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
    const auto v = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
    out.k[0][u] = k[0];
    out.k[1][u] = k[1];
    out.v[0][u] = v[0];
    out.v[1][u] = v[1];
  }
  return out;
}

// A lane's head in the second product is lane % 16; in the first one a lane has
// key lane % 16 and N heads, g, g + 4, .. with g = lane / 16: head h of the queries
// is row 4 (h % 4) + h / 4 of the operand, so that few heads fill few registers.
template <int DIM, int N>
struct State {
  static constexpr int G = DIM / 64;
  // o[u][n][i]: the first sum of channel 64 u + 16 g + 4 i + n of head lane % 16,
  // times 2^(kTop - ev - 24) (n odd: 2^(kTop - ev - 20))
  f32x4 o[G][4];
  // of heads g + 4 i, over keys lane % 16 of each block: sums of weights times mid, and of weights
  float mids[G][N], l[N];
  float m[N];      // weights are exp2(score * log2 e - m), at most 2^kSlack
  float up[G][N];  // 2^(kTop - ev), with 2^ev over weights times scales, to kMost
};

// Weights of one u for the second product, [head][key], keys in the order in
// which a lane takes them: 4 g .. 4 g + 3 of the first block, then of the second.
constexpr int kWeightRow = 40;  // halves: what 16 lanes read together lies on different banks

// A row's queries: their fp16 fragments (head query_of(lane)), and for heads g + 4 i
// 2^-24 times their sums by group, and what makes scores * log2 e of a product: a
// factor >= 0, times 2^rest where `more` (for the wave) says that it is not 1.
template <int DIM, int N>
struct Query {
  u32x4 w[DIM / 32];
  float sum[DIM / 64][N], factor[N];
  int rest[N];
  bool more;
};
__device__ __forceinline__ int query_of(int lane) { return (lane >> 2 & 3) + 4 * (lane & 3); }

// codes of the even (bits 0..3, 8..11) or odd (4..7, 12..15) nibble of 16-bit
// halves as fp16: n = 0..3 from the lowest
__device__ __forceinline__ uint32_t nibbles(uint32_t w, int n) {
  return (n & 2 ? w >> 8 : w) & (n & 1 ? 0x00f000f0u : 0x000f000fu);
}

// the same codes less 8
__device__ __forceinline__ uint32_t centred(uint32_t w, int n) {
  const f16x2 off = __builtin_bit_cast(f16x2, n & 1 ? 0x00800080u : 0x00080008u);
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, nibbles(w, n)) - off);
}

// The greatest of 16 lanes.
__device__ __forceinline__ float max16(float x) {
  const auto turn = [](float v, auto by) {
    const int u = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, 0x120 + decltype(by)::value, 0xf, 0xf, false));
  };
  x = fmaxf(x, turn(x, std::integral_constant<int, 8>()));
  x = fmaxf(x, turn(x, std::integral_constant<int, 4>()));
  x = fmaxf(x, turn(x, std::integral_constant<int, 2>()));
  return fmaxf(x, turn(x, std::integral_constant<int, 1>()));
}

__device__ __forceinline__ float sum16(float x) {
  const auto turn = [](float v, auto by) {
    const int u = __builtin_bit_cast(int, v);
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, 0x120 + decltype(by)::value, 0xf, 0xf, false));
  };
  x += turn(x, std::integral_constant<int, 8>());
  x += turn(x, std::integral_constant<int, 4>());
  x += turn(x, std::integral_constant<int, 2>());
  return x + turn(x, std::integral_constant<int, 1>());
}

// The products of one step's 32 keys with the queries, times `factor` (and
// 2^rest): x[b][i] of key 16 b + lane % 16 and head g + 4 i.
template <int DT, int DIM, int N>
__device__ __forceinline__ void scores(float (&x)[2][N], const Tile<DIM> &t, const Pairs<DIM> &p,
                                       const Query<DIM, N> &q) {
  constexpr int G = DIM / 64;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 c[G];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      c[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 2 * u; y < 2 * u + 2; ++y) {
        const uint32_t w = t.k[b][y];
        const u32x4 a = {nibbles(w, 0), nibbles(w, 1), nibbles(w, 2), nibbles(w, 3)};
        c[u] = mfma16x16x32<kF16>(q.w[y], a, c[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const float low = act_to_f32<DT>(p.k[b][u] >> 16);
        s = u ? __builtin_fmaf(low, q.sum[u][i], s) : low * q.sum[u][i];
      }
#pragma unroll
      for (int u = 0; u < G; ++u) s = __builtin_fmaf(act_to_f32<DT>(p.k[b][u] & 0xffffu), c[u][i], s);
      x[b][i] = s;
    }
  }
}

// Weights of the scores x; dead keys have none.  Returns the lane's greatest
// exponent of one.
template <int DIM, int N>
__device__ __forceinline__ float weights_of(float (&w)[2][N], const float (&x)[2][N], const Query<DIM, N> &q,
                                            const float (&m)[N], bool end, int live, int lane) {
  float top = -INFINITY;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[b][i] = __builtin_fmaf(x[b][i], q.factor[i], -m[i]);
      top = fmaxf(top, w[b][i]);
      w[b][i] = __builtin_amdgcn_exp2f(w[b][i]);
    }
  if (end) {
    asm volatile("");
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < N; ++i) w[b][i] = 16 * b + (lane & 15) >= live ? 0.f : w[b][i];
  }
  return top;
}

// ev of 2^(kTop - ev)
__device__ __forceinline__ int exponent_of(float up) { return kTop + 1 - __builtin_amdgcn_frexp_expf(up); }

// The sums of weights times scales times factor, of heads g + 4 i.  room: 16 G
// floats of the wave's.
template <int DIM, int N>
__device__ __forceinline__ void multiply(State<DIM, N> &st, const float (&factor)[DIM / 64][N], float *room, int lane) {
  constexpr int G = DIM / 64;
#pragma unroll
  for (int u = 0; u < G; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((lane & 15) == 0) room[16 * u + (lane >> 4) + 4 * i] = factor[u][i];
  wave_lds_sync();
  float f[G];  // of head lane % 16 (other lanes' sums are not used)
#pragma unroll
  for (int u = 0; u < G; ++u) f[u] = room[16 * u + ((lane & 15) & (4 * N - 1))];
  wave_lds_sync();
#pragma unroll
  for (int u = 0; u < G; ++u)
#pragma unroll
    for (int n = 0; n < 4; ++n) st.o[u][n] *= f[u];
}

// The maxima rise: the sums so far are made relative to the new ones.  The
// exponents of weights times scales fall by the whole part of that, as those
// weights do; one that is then too low for the new keys is set by set_exponents.
template <int DIM, int N>
__device__ __forceinline__ void raise(State<DIM, N> &st, const float (&x)[2][N], const Query<DIM, N> &q, float *room,
                                      int lane) {
  float factor[DIM / 64][N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float m = fmaxf(st.m[i], max16(fmaxf(x[0][i], x[1][i])) * q.factor[i]);
    const float rise = m == st.m[i] ? 0.f : m - st.m[i], keep = __builtin_amdgcn_exp2f(-rise);
    const int whole = (int)fminf(rise, 1024.f);
    st.m[i] = m;
    st.l[i] *= keep;
#pragma unroll
    for (int u = 0; u < DIM / 64; ++u) {
      st.mids[u][i] *= keep;
      const int ev = exponent_of(st.up[u][i]), now = max(ev - whole, kLeastExponent);
      st.up[u][i] = ldexpf(1.f, kTop - now);
      factor[u][i] = ldexpf(keep, ev - now);
    }
  }
  multiply<DIM, N>(st, factor, room, lane);
}

// Exponents over the present keys' weights times scales (NaN leaves them) and, but
// for the FRESH ones, over those so far.
template <int DIM, int N, bool FRESH>
__device__ __forceinline__ void set_exponents(State<DIM, N> &st, const float (&w)[2][N], const float (&vs)[2][DIM / 64],
                                              float *room, int lane) {
  float factor[DIM / 64][N];
#pragma unroll
  for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float most = max16(fmaxf(w[0][i] * vs[0][u], w[1][i] * vs[1][u]));
      int ev = most > 0.f ? max(__builtin_amdgcn_frexp_expf(most), kLeastExponent) : kLeastExponent;
      if constexpr (!FRESH) {
        const int old = exponent_of(st.up[u][i]);
        ev = max(ev, old);
        factor[u][i] = ldexpf(1.f, old - ev);
      }
      st.up[u][i] = ldexpf(1.f, kTop - ev);
    }
  if constexpr (!FRESH) multiply<DIM, N>(st, factor, room, lane);
}

// Weights of the scores x, into the sums and, times the scales of V, into `lds`
// (2^(kTop - ev) p s in fp16).  FRESH: the first step.
template <int DT, int DIM, int N, bool FRESH>
__device__ __forceinline__ void weigh(State<DIM, N> &st, float (&x)[2][N], const Pairs<DIM> &pairs,
                                      const Query<DIM, N> &q, uint16_t *lds, bool end, int live, int lane) {
  constexpr int G = DIM / 64;
  float vs[2][G], mid[2][G];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int u = 0; u < G; ++u) {
      vs[b][u] = act_to_f32<DT>(pairs.v[b][u] & 0xffffu);
      mid[b][u] = __builtin_fmaf(8.f, vs[b][u], act_to_f32<DT>(pairs.v[b][u] >> 16));
    }
  if (q.more) {  // (uniform) a factor that one fp32 number does not hold
    asm volatile("");
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < N; ++i) x[b][i] = ldexpf(x[b][i], q.rest[i]);
  }
  if (end) {  // (uniform) dead keys do not raise a maximum
    asm volatile("");
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < N; ++i) x[b][i] = 16 * b + (lane & 15) >= live ? -3e38f : x[b][i];
  }
  float w[2][N];
  _Float16 h[2][G][N];  // 2^(kTop - ev) p s
  // whether (for the wave) one of them is too large (NaN is not)
  const auto round = [&]() {
    _Float16 most = 0;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          h[b][u][i] = (_Float16)__builtin_fmaf(w[b][i] * st.up[u][i], vs[b][u], 0.f);
          most = __builtin_fmaxf16(most, h[b][u][i]);
        }
    return most >= (_Float16)kMost;
  };
  float *const room = reinterpret_cast<float *>(lds);
  if constexpr (FRESH) {
#pragma unroll
    for (int i = 0; i < N; ++i) st.m[i] = fmaxf(max16(fmaxf(x[0][i], x[1][i])) * q.factor[i], kLeastMaximum);
    (void)weights_of<DIM, N>(w, x, q, st.m, end, live, lane);
    set_exponents<DIM, N, true>(st, w, vs, room, lane);
    (void)round();
  } else {
    const float top = weights_of<DIM, N>(w, x, q, st.m, end, live, lane);
    bool over = round();
    if (__any(top > kSlack || over)) {  // seldom
      raise<DIM, N>(st, x, q, room, lane);
      (void)weights_of<DIM, N>(w, x, q, st.m, end, live, lane);
      over = round();
      if (__any(over)) {
        set_exponents<DIM, N, false>(st, w, vs, room, lane);
        (void)round();
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) st.l[i] += w[0][i] + w[1][i];
  // key 16 b + 4 j + k of a block stands at 8 j + 4 b + k
  uint16_t *to = lds + (lane >> 4) * kWeightRow + 8 * (lane >> 2 & 3) + (lane & 3);
#pragma unroll
  for (int u = 0; u < G; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      st.mids[u][i] = __builtin_fmaf(w[0][i], mid[0][u], __builtin_fmaf(w[1][i], mid[1][u], st.mids[u][i]));
#pragma unroll
      for (int b = 0; b < 2; ++b)
        to[(16 * u + 4 * i) * kWeightRow + 4 * b] = __builtin_bit_cast(uint16_t, h[b][u][i]);
    }
}

// The second product.
template <int DIM, int N>
__device__ __forceinline__ void add_values(State<DIM, N> &st, const typename Words<DIM / 32>::type (&codes)[2],
                                           const uint16_t *lds, int lane) {
#pragma unroll
  for (int u = 0; u < DIM / 64; ++u) {
    const u32x4 p = *reinterpret_cast<const u32x4 *>(lds + (16 * u + (lane & 15)) * kWeightRow + 8 * (lane >> 4));
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const u32x4 a = {centred(codes[0][2 * u], n), centred(codes[0][2 * u + 1], n), centred(codes[1][2 * u], n),
                       centred(codes[1][2 * u + 1], n)};
      st.o[u][n] = mfma16x16x32<kF16>(a, p, st.o[u][n]);
    }
  }
}

// Lane: head query_of(lane), channels 32 x + 8 g..; unused heads repeat the last one.
template <int DIM>
__device__ __forceinline__ void load_query(u32x4 (&raw)[DIM / 32], const AttentionArgs &a, int64_t row, int head0,
                                           int heads, int lane) {
  const uint16_t *qp =
      a.q + row * a.q_token + (int64_t)(head0 + min(query_of(lane), heads - 1)) * a.q_head + 8 * (lane >> 4);
#pragma unroll
  for (int x = 0; x < DIM / 32; ++x) raw[x] = *reinterpret_cast<const u32x4 *>(qp + 32 * x);
}

template <int DT, int DIM, int N>
__device__ __forceinline__ void open_query(Query<DIM, N> &q, const u32x4 (&raw)[DIM / 32], float scale, int heads,
                                           int lane) {
  constexpr int G = DIM / 64, KS = DIM / 32;
  float most = 0.f;
#pragma unroll
  for (int x = 0; x < KS; ++x) {
    q.w[x] = query_of(lane) < heads ? raw[x] : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(act_to_f32<DT>(q.w[x][j / 2] >> (16 * (j & 1)) & 0xffffu)));
  }
  most = max_over_groups(most);
  int e = 0;
  if (most < INFINITY) (void)frexpf(most, &e);  // most < 2^e
  const float sign = scale < 0.f ? -1.f : 1.f;
  float sum[G];
#pragma unroll
  for (int u = 0; u < G; ++u) sum[u] = 0.f;
#pragma unroll
  for (int x = 0; x < KS; ++x)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f0 = ldexpf(act_to_f32<DT>(q.w[x][j] & 0xffffu), 15 - e) * sign;
      const float f1 = ldexpf(act_to_f32<DT>(q.w[x][j] >> 16), 15 - e) * sign;
      sum[x / 2] += f0 + f1;
      const float part = j & 1 ? 0x1p-4f : 1.f;
      q.w[x][j] = pack2<kF16>(f0 * part, f1 * part);
    }
  // |scale| log2 e 2^shift: in one number where that is neither too large nor
  // too small for one; the products then take 2^rest
  const float scale2 = fabsf(scale) * 1.44269504088896340736f;
  const int shift = 24 - 15 + e;
  int es;
  (void)frexpf(scale2, &es);
  const int part = max(-100 - es, min(shift, 100 - es));
  const int rest = scale2 > 0.f ? shift - part : 0;
  const float factor = scale2 > 0.f ? ldexpf(scale2, part) : 0.f;
  q.more = __any(rest != 0);
  // from rows lane % 16 to rows 4 g + i, heads g + 4 i
#pragma unroll
  for (int u = 0; u < G; ++u) {
    const float all = sum_over_groups(sum[u]) * 0x1p-24f;
#pragma unroll
    for (int i = 0; i < N; ++i) q.sum[u][i] = __shfl(all, 4 * (lane >> 4) + i, 64);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q.factor[i] = __shfl(factor, 4 * (lane >> 4) + i, 64);
    q.rest[i] = __shfl(rest, 4 * (lane >> 4) + i, 64);
  }
}

// How a call's work is dealt out (see plan_attention_decode4): rows one after
// another, each row's outputs (key-value heads, head tiles) one after another, an
// output being kOutputUnits for its start and end and a unit per kUnit keys (an
// empty row has one).  A workgroup takes `share` units one after another; the
// steps of an output begin kOutputUnits behind its first unit.
__device__ __forceinline__ int units_of(int len) { return max(1, (len + kUnit - 1) / kUnit); }

// The sum of the lanes up to this one.
__device__ __forceinline__ int inclusive_sum(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // the row before's last lane
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // the first half's last lane
  return x;
}

// The slots of an output's parts: a workgroup's second slot has what it began
// and did not end, its first what it went on with.
struct DealtParts {
  int first;  // the workgroup with part 0
  __device__ __forceinline__ int operator()(int p) const { return p ? 2 * (first + p) : 2 * first + 1; }
};

// A workgroup's piece of one output.
struct Piece {
  int row, slot, len;
  int steps;           // of the row
  int begin, end;      // the piece's keys
  int kvh, heads, head0;
  uint32_t first;      // the output's first step, in units
  bool whole, none;    // none: only units that stand for an output's start
};

// MANY: more outputs than workgroups, or not dealt (a kernel of its own, since the
// other's code is shorter and its calls are: one row of 777 keys 8.2 us, 9.1 with
// both in one).
template <int DT, int DIM, int N, bool MANY>
__global__ void __launch_bounds__(256, kDecode4Resident)
decode4_attention_kernel(AttentionArgs a, Decode4Plan plan, uint32_t *__restrict__ counters,
                         float *__restrict__ partials) {
  constexpr int G = DIM / 64;
  __shared__ DecodeJoin<DIM> lds;
  static_assert(sizeof(lds.o[0]) >= (DIM / 64) * 16 * kWeightRow * 2, "a wave's weights lie where its sums will");
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  const int outputs = a.kv_heads * plan.head_tiles;  // of a row
  const int rows = a.sequences;
  // a CU's second workgroup, which takes the lead in every other step (see the header)
  const bool young = blockIdx.x >= 256;
  // this workgroup's (or wave's) units at..until, in row `row`, whose first is before * outputs
  // (the host has seen that all of a call's units are fewer than 2^31)
  uint32_t at, until, share = 1, before = 0;
  bool whole = true;  // outputs are not cut
  bool lone = false;  // each wave has outputs of its own, those whose first unit is in its share
  int row, row0 = 0, lane_slot = 0, lane_len = 0;  // lane: row row0 + lane
  const auto look_at = [&](int first) {
    row0 = first;
    lane_slot = a.slots[min(first + lane, rows - 1)];
    lane_len = a.kv.length(lane_slot);
  };
  const int per = plan.dealt ? (rows + 63) >> 6 : 2;  // rows that a lane looks up
  int units = 0, longest = 0;
  if (plan.dealt) {  // every wave for itself
    const int first = lane * per;
    constexpr int kRows = MANY ? 8 : 4;  // looked up together
    for (int j0 = 0; j0 < per; j0 += kRows) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = first + j0 + j;
        if (j0 + j < per && r < rows) {
          lane_slot = a.slots[r];
          lane_len = a.kv.length(lane_slot);
          const int n = units_of(lane_len);
          units += n + kOutputUnits;
          longest = max(longest, n);
        }
      }
    }
  }
  if (MANY ? !plan.dealt : !__any(longest > plan.whole)) {
    // a workgroup per output
    if (blockIdx.x >= (uint32_t)(rows * outputs)) return;
    row = (int)(blockIdx.x / (uint32_t)outputs);
    if (per > 1) look_at(row);
    const int n = units_of(__builtin_amdgcn_readlane(lane_len, row - row0)) + kOutputUnits;
    at = (blockIdx.x - (uint32_t)(row * outputs)) * (uint32_t)n;
    until = at + n;
  } else {
    const int sum = inclusive_sum(units);
    const uint32_t total = (uint32_t)__builtin_amdgcn_readlane(sum, 63) * outputs;
    share = (total + gridDim.x - 1) / gridDim.x;
    uint32_t worker = blockIdx.x;
    const uint32_t of_wave = (share + kDecodeWaves - 1) / kDecodeWaves;
    lone = MANY && !__any((uint32_t)longest * kLoneLongest > of_wave * kLoneShare);
    if (lone) {
      share = of_wave;
      worker = blockIdx.x * kDecodeWaves + wave;
    }
    whole = lone;
    at = worker * share;
    until = min(total, at + share);
    if (at >= total) return;
    // the lane that has the row of the first unit, then the row
    const int unit = (int)(at / (uint32_t)outputs);
    int who = __ffsll((unsigned long long)__ballot(sum > unit)) - 1;
    int end = sum;
    if (per > 1) {
      const int begin = __builtin_amdgcn_readlane(sum - units, who);
      look_at(who * per);
      units = row0 + lane < rows ? units_of(lane_len) + kOutputUnits : 0;
      end = begin + inclusive_sum(units);
      who = __ffsll((unsigned long long)__ballot(end > unit)) - 1;
    }
    who = max(who, 0);  // (no lane, should lengths change while they are read)
    row = min(row0 + who, rows - 1);
    before = __builtin_amdgcn_readlane(end - units, who);
    if (lone) {
      const uint32_t all = __builtin_amdgcn_readlane(units_of(lane_len), who) + kOutputUnits;
      const uint32_t skip = (at - before * outputs) % all;
      at += skip ? all - skip : 0;
      if (at >= until) return;
      if (at >= (before + all) * outputs) {
        before += all;
        row = min(row + 1, rows - 1);
      }
    }
  }
  // (twice, so that the strides are constants: 300 rows of up to 1000 keys 46 us, 49 at run time)
  const auto run = [&](auto alone) __attribute__((always_inline)) {
    constexpr bool LONE = decltype(alone)::value;
    const __amdgpu_buffer_rsrc_t rs =
        raw_rsrc(partials, plan.dealt ? 2u * gridDim.x * (uint32_t)part_floats(a.group, DIM) * 4u : 0u);

    // the piece at `at`, which moves to the next one
    const auto next_piece = [&]() {
      Piece p;
      p.row = row;
      if (row - row0 >= 64) look_at(row);
      p.slot = __builtin_amdgcn_readlane(lane_slot, row - row0);
      p.len = __builtin_amdgcn_readlane(lane_len, row - row0);
      p.steps = units_of(p.len);
      const int all = p.steps + kOutputUnits;
      const uint32_t rel = at - before * outputs;
      const int output = (int)(rel / (uint32_t)all), skip = (int)(rel - (uint32_t)output * all);
      const int take = LONE || whole ? all : (int)min((uint32_t)(all - skip), until - at);
      const int step0 = max(0, skip - kOutputUnits), step1 = skip + take - kOutputUnits;
      p.none = step1 <= 0;
      p.whole = step1 - step0 == p.steps;
      p.begin = step0 * kUnit;
      p.end = min(p.len, step1 * kUnit);
      const int tile = output % plan.head_tiles;
      p.kvh = output / plan.head_tiles;
      p.heads = min(16, a.group - 16 * tile);
      p.head0 = p.kvh * a.group + 16 * tile;
      p.first = before * outputs + (uint32_t)output * all + kOutputUnits;
      at += take;
      if (at >= (before + all) * outputs) {
        before += all;
        row = min(row + 1, rows - 1);
      }
      return p;
    };

    // the loads of a wave's tiles of a piece; a ring of tiles: one is worked on
    // while the others are loaded
    constexpr int stride = LONE ? kStep : kUnit;  // between a wave's steps
    const char *const k = (const char *)a.kv.k, *const v = (const char *)a.kv.v;
    constexpr uint32_t kCodes = sizeof(typename Tile<DIM>::Codes);
    const uint32_t k_lane = (lane & 15) * Kv4<DIM>::kRow + (lane >> 4) * kCodes, v_lane = lane * kCodes;
    const char *const p_lane = (lane & 32 ? v : k) + (lane & 15) * (4 * G);
    const int shift = a.kv.page_shift;
    Piece piece;
    Window<DIM> win;
    Tile<DIM> t[kTiles];
    int pos, loaded;  // of the piece: the next step's first key, the steps loaded
    const auto load = [&](Tile<DIM> &t, int p) {
      if ((loaded & 31) == 0)
        win.look_up(a.kv.table + (int64_t)piece.slot * a.kv.max_pages, a.kv.page_stride * 2,
                    piece.kvh * Kv4<DIM>::head_bytes(1 << shift), (piece.len - 1) >> shift, a.kv.num_pages, shift, p,
                    stride, lane);
      const int64_t c0 = win.block(2 * (loaded & 31)), c1 = win.block(2 * (loaded & 31) + 1);
      // from a block's codes to its pairs
      const int mask = (1 << shift) - 1, ends = Kv4<DIM>::pairs_at(1 << shift);
      const int64_t p0 = c0 + ends - (p & mask) * (Kv4<DIM>::kRow - 4 * G);
      const int64_t p1 = c1 + ends - ((p + 16) & mask) * (Kv4<DIM>::kRow - 4 * G);
      t.pairs = *reinterpret_cast<const typename Words<G>::type *>(p_lane + (lane & 16 ? p1 : p0));
      t.k[0] = *reinterpret_cast<const typename Tile<DIM>::Codes *>(k + c0 + k_lane);
      t.k[1] = *reinterpret_cast<const typename Tile<DIM>::Codes *>(k + c1 + k_lane);
      t.v[0] = *reinterpret_cast<const typename Tile<DIM>::Codes *>(v + c0 + v_lane);
      t.v[1] = *reinterpret_cast<const typename Tile<DIM>::Codes *>(v + c1 + v_lane);
      ++loaded;
    };
    u32x4 raw[DIM / 32];
    const auto start = [&]() {
      piece = next_piece();
      if (piece.none) return;
      load_query<DIM>(raw, a, piece.row, piece.head0, piece.heads, lane);
      pos = piece.begin + (LONE ? 0 : wave * kStep);
      loaded = 0;
#pragma unroll
      for (int d = 0; d + 1 < kTiles; ++d)
        if (pos + d * stride < piece.end) load(t[d], pos + d * stride);
    };
    start();
    while (true) {
      const int end = piece.end;
      const bool none = piece.none;
      if (!none) {
        State<DIM, N> st;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          st.m[i] = -INFINITY;
          st.l[i] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
#pragma unroll
          for (int i = 0; i < N; ++i) st.mids[u][i] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) st.o[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int i = 0; i < N; ++i) st.up[u][i] = 1.f;
        if (pos < end) {
          uint16_t *weights = reinterpret_cast<uint16_t *>(&lds.o[wave][0][0]);
          Query<DIM, N> q;
          open_query<DT, DIM, N>(q, raw, a.scale, piece.heads, lane);
          bool more = true;
          const auto turn = [&](Tile<DIM> &now, Tile<DIM> &ahead, auto fresh) {
            const int live = end - pos;  // keys of this step: more than there are but at the end
            const bool tail = live < kStep;
            if (live > (kTiles - 1) * stride) load(ahead, pos + (kTiles - 1) * stride);
            if (tail) {  // (uniform) what the page holds behind the end does not count
              asm volatile("");
              if ((lane & 31) >= live)
#pragma unroll
                for (int u = 0; u < G; ++u) now.pairs[u] = 0;
            }
            const Pairs<DIM> pairs = spread<DIM>(now.pairs);
            if (young) {
              if (&now == &t[0]) __builtin_amdgcn_s_setprio(1);
              else __builtin_amdgcn_s_setprio(0);
            }
            float x[2][N];
            scores<DT, DIM, N>(x, now, pairs, q);
            weigh<DT, DIM, N, decltype(fresh)::value>(st, x, pairs, q, weights, tail, live, lane);
            wave_lds_sync();
            add_values<DIM, N>(st, now.v, weights, lane);
            wave_lds_sync();
            pos += stride;
            more = live > stride;
          };
          turn(t[0], t[kTiles - 1], std::true_type());
          while (more) {
#pragma unroll
            for (int d = 1; d <= kTiles; ++d) {
              turn(t[d % kTiles], t[(d + kTiles - 1) % kTiles], std::false_type());
              if (!more) break;
            }
          }
        }
        // ---- a wave's sums ----
        {
          // heads g + 4 i, over 16 lanes; then head lane % 16
          float *own = &lds.o[wave][0][0];  // [quantity][head]: sums of mids, up
          const int h = lane & 15, g = lane >> 4;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float l = sum16(st.l[i]);
            float mids[G];
#pragma unroll
            for (int u = 0; u < G; ++u) mids[u] = sum16(st.mids[u][i]);
            if (h == 0) {
              lds.m[wave][g + 4 * i] = st.m[i];
              lds.l[wave][g + 4 * i] = l;
#pragma unroll
              for (int u = 0; u < G; ++u) {
                own[16 * u + g + 4 * i] = mids[u];
                own[16 * (G + u) + g + 4 * i] = st.up[u][i];
              }
            }
          }
          wave_lds_sync();
          float mids[G];
          int ev[G];
#pragma unroll
          for (int u = 0; u < G; ++u) {
            mids[u] = own[16 * u + (h & (4 * N - 1))];
            ev[u] = exponent_of(own[16 * (G + u) + (h & (4 * N - 1))]);
          }
          const float inv = piece.len > 0 ? 1.f / lds.l[wave][h & (4 * N - 1)] : 0.f;
          wave_lds_sync();
          if (h < piece.heads) {
            uint16_t *const out = a.y + piece.row * a.y_token + (int64_t)(piece.head0 + h) * a.y_head;
#pragma unroll
            for (int u = 0; u < G; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int c = 64 * u + 16 * g + 4 * i;
                f32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = ldexpf(st.o[u][j][i], (j & 1 ? 20 : 24) - kTop + ev[u]) + mids[u];
                if (LONE) *reinterpret_cast<u32x2 *>(out + c) = piece.len > 0 ? pack_row<DT>(y, inv) : u32x2{0, 0};
                else *reinterpret_cast<f32x4 *>(&lds.o[wave][h][c]) = y;
              }
          }
        }
      }
      if (LONE) {
        if (at >= until) break;
        start();
        continue;
      }
      const Piece done = piece;
      const bool more = at < until;
      if (more) start();  // (its loads pass while the waves are joined)
      if (!none) {
        int part = 0, parts = 1;
        DealtParts place = {0};
        if (!done.whole) {
          place.first = (int)min(done.first / share, gridDim.x - 1);
          part = (int)blockIdx.x - place.first;
          parts = (int)((done.first + done.steps - 1) / share) - place.first + 1;
        }
        join_parts<DT, DIM, false>(a, lds, counters + place.first, rs, place, done.row, done.head0, done.heads, part,
                                   parts, done.len > 0);
      }
      if (!more) break;
      __syncthreads();  // the join's reads of lds are done
    }
  };
  if constexpr (MANY) {
    if (lone) {
      run(std::true_type());
      return;
    }
  }
  run(std::false_type());
}

}  // namespace

// Rows of up to kMaxDealtRows have their units dealt out in equal shares to as
// many workgroups as the card holds at once, so that the longest row ends with
// the others; more rows than that, whose lengths take too long to look up in
// every workgroup, are a workgroup for each output.  So are outputs that the card
// holds at once where none has more than `whole` units, which grows with their
// number, since the shares do.  Dealt and not, us: 64 rows of up to 4096 37 and 44,
// rows of 131072 and 100001 59 and 1014, one of 777 9 and 10.8, 300 of up to 1000
// 46 and 49, 2000 of up to 300 120 and 182, 4000 of up to 200 181 and 324; but 64 of
// up to 700 16.8 and 11.7, 64 of up to 1500 20.8 and 18.3, 30 of up to 400 10.8 and
// 8.3, one of 512 9.2 and 8.8.
Decode4Plan plan_attention_decode4(int64_t rows, int q_heads, int kv_heads, int64_t max_len) {
  Decode4Plan p;
  p.head_tiles = (q_heads / kv_heads + 15) / 16;
  const int64_t outputs = rows * kv_heads * p.head_tiles;
  const int64_t units = std::max<int64_t>(1, (max_len + kUnit - 1) / kUnit), most = outputs * (units + kOutputUnits);
  p.dealt = rows <= kMaxDealtRows && most < int64_t(1) << 30;  // (the sums' type)
  p.workgroups = (int)(p.dealt ? std::min<int64_t>(most, 256 * kDecode4Resident) : outputs);
  p.whole = outputs <= p.workgroups ? 5 + (int)outputs / 48 : 0;
  return p;
}

size_t attention_decode4_partial_bytes(int q_heads, int kv_heads, int head_dim) {
  return (size_t)2 * 256 * kDecode4Resident * part_floats(q_heads / kv_heads, head_dim) * 4;
}

hipError_t launch_attention_decode4(const AttentionArgs &a, const Decode4Plan &p, uint32_t *counters,
                                    float *partials, hipStream_t st) {
  const dim3 grid((unsigned)p.workgroups);
  const int heads = std::min(a.group, 16);
  const bool many = !p.dealt || p.whole == 0;
#define PARO_DECODE4_MANY(DT, DIM, N, MANY) \
  hipLaunchKernelGGL((decode4_attention_kernel<DT, DIM, N, MANY>), grid, dim3(256), 0, st, a, p, counters, partials)
#define PARO_DECODE4(DT, DIM, N)             \
  if (many) {                                \
    PARO_DECODE4_MANY(DT, DIM, N, true);     \
  } else {                                   \
    PARO_DECODE4_MANY(DT, DIM, N, false);    \
  }
#define PARO_DECODE4_HEADS(DT, DIM) \
  if (heads <= 4) {                 \
    PARO_DECODE4(DT, DIM, 1)        \
  } else if (heads <= 8) {          \
    PARO_DECODE4(DT, DIM, 2)        \
  } else {                          \
    PARO_DECODE4(DT, DIM, 4)        \
  }
  if (a.dt == kF16) {
    if (a.head_dim == 64) {
      PARO_DECODE4_HEADS(kF16, 64)
    } else {
      PARO_DECODE4_HEADS(kF16, 128)
    }
  } else {
    if (a.head_dim == 64) {
      PARO_DECODE4_HEADS(kBF16, 64)
    } else {
      PARO_DECODE4_HEADS(kBF16, 128)
    }
  }
#undef PARO_DECODE4_HEADS
#undef PARO_DECODE4
#undef PARO_DECODE4_MANY
  return hipGetLastError();
}

}  // namespace paro
