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
//     contraction step, its 16 bytes of V four keys of eight channels.  S^T and
//     O^T fragments lie as in attention_decode.hip, with the head in lane % 16.
//   - Pairs are loaded a word per lane and step, opened and shared through LDS.
//   - What is rounded to fp16 is p s 2^(15 - ev), with 2^ev over every scale of V
//     so far (and 2^-16 of every |low|: smaller scales than that add nothing).
#include <math.h>

#include <algorithm>

#include "attention.hpp"
#include "attention_join.hpp"
#include "common.hpp"
#include "kv4.hpp"
#include "mfma.hpp"

namespace paro {
namespace {

constexpr int kStep = 32;                    // keys per wave and step
constexpr int kUnit = kStep * kDecodeWaves;  // keys per workgroup and step
constexpr int kWhole = 3 * kUnit;            // rows up to this length are not cut
constexpr int kLeastExponent = -126;         // of the values' scale

template <int N>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N)));
};

// 32 keys of K and V: [16-key block]
template <int DIM>
struct Tile {
  typedef typename Words<DIM / 32>::type Codes;
  Codes k[2], v[2];
  uint32_t pk, pv;  // this lane's pair of either
};

// Byte offset, in a layer's K or V, of 16 consecutive positions (they lie in one
// page): their codes, and their pairs.
template <int DIM>
struct Pages {
  const int32_t *table;
  int64_t page_bytes, head_offset;
  int last, num_pages, shift;
  struct At {
    int64_t codes, pairs;
  };
  __device__ __forceinline__ At at(int pos) const {
    const int j = min(pos >> shift, last);
    int page = table[j];
    page = page < 0 ? 0 : page >= num_pages ? num_pages - 1 : page;
    const int64_t base = (int64_t)page * page_bytes + head_offset;
    const int p = pos & ((1 << shift) - 1);
    return At{base + p * Kv4<DIM>::kRow, base + Kv4<DIM>::pairs_at(1 << shift) + p * Kv4<DIM>::kGroups * 4};
  }
};

template <int DIM>
__device__ __forceinline__ void load_tile(Tile<DIM> &t, const char *__restrict__ k, const char *__restrict__ v,
                                          const typename Pages<DIM>::At &a0, const typename Pages<DIM>::At &a1,
                                          int lane) {
  typedef typename Tile<DIM>::Codes Codes;
  constexpr int G = Kv4<DIM>::kGroups, W = 16 * G;  // pair words of a block
  const int ko = (lane & 15) * Kv4<DIM>::kRow + (lane >> 4) * (int)sizeof(Codes), vo = lane * (int)sizeof(Codes);
  t.k[0] = *reinterpret_cast<const Codes *>(k + a0.codes + ko);
  t.k[1] = *reinterpret_cast<const Codes *>(k + a1.codes + ko);
  t.v[0] = *reinterpret_cast<const Codes *>(v + a0.codes + vo);
  t.v[1] = *reinterpret_cast<const Codes *>(v + a1.codes + vo);
  const int64_t pairs = ((lane / W) & 1 ? a1.pairs : a0.pairs) + (lane & (W - 1)) * 4;
  t.pk = *reinterpret_cast<const uint32_t *>(k + pairs);
  t.pv = *reinterpret_cast<const uint32_t *>(v + pairs);
}

// {scale, low} of K and {scale * 2^(15 - ev), mid} of V for the 32 keys of a step
template <int DIM>
struct Shared {
  f32x2 k[32 * Kv4<DIM>::kGroups], v[32 * Kv4<DIM>::kGroups];
};

template <int DIM>
struct State {
  static constexpr int G = DIM / 64;
  // o[u][n][i]: the first sum of channel 64 u + 16 g + 4 i + n of the lane's head,
  // times 2^(15 - ev - 24) (n odd: 2^(15 - ev - 20))
  f32x4 o[G][4];
  float mids[G];  // this lane's share of the sum of weights times mid
  float m, l;     // maximum of scores * log2 e, this lane's share of the sum of weights
  int ev;         // 2^ev: over the scales of V
};

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

// One step: 32 keys, `live` of them in the sequence (>= 32 but at its end).
template <int DT, int DIM>
__device__ __forceinline__ void step(State<DIM> &st, Tile<DIM> &t, Shared<DIM> &lds, const u32x4 (&q)[DIM / 32],
                                     const float (&qsum)[DIM / 64], float scale2, int shift, int live, int lane) {
  constexpr int G = DIM / 64, W = 16 * G;
  const int g = lane >> 4;
  const bool end = live < kStep;  // what the page holds behind the end does not count
  if (end && (lane & (2 * W - 1)) / G >= live) t.pk = t.pv = 0;
  const float vs = act_to_f32<DT>(t.pv & 0xffffu), vlow = act_to_f32<DT>(t.pv >> 16);
  const float size = fmaxf(vs, fabsf(vlow) * 0x1p-16f);
  if (__any(size >= ldexpf(1.f, st.ev))) {  // seldom but in the first step
    float most = size;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
    int e;
    (void)frexpf(most, &e);
    e = max(st.ev, min(e, 128));
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[u][n][i] = ldexpf(st.o[u][n][i], st.ev - e);
    st.ev = e;
  }
  if (lane < 2 * W) {
    lds.k[lane] = f32x2{act_to_f32<DT>(t.pk & 0xffffu), act_to_f32<DT>(t.pk >> 16)};
    lds.v[lane] = f32x2{ldexpf(vs, 15 - st.ev), __builtin_fmaf(8.f, vs, vlow)};
  }
  wave_lds_sync();
  float s[8];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 c[G];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      c[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 2 * u; x < 2 * u + 2; ++x) {
        const uint32_t w = t.k[b][x];
        const u32x4 a = {nibbles(w, 0), nibbles(w, 1), nibbles(w, 2), nibbles(w, 3)};
        c[u] = mfma16x16x32<kF16>(a, q[x], c[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = 0.f;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const f32x2 p = lds.k[(16 * b + 4 * g + i) * G + u];
        x = __builtin_fmaf(p[0], c[u][i], x);
        x = __builtin_fmaf(p[1], qsum[u], x);
      }
      s[4 * b + i] = ldexpf(x * scale2, shift);
    }
  }
  if (end) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (16 * (u >> 2) + 4 * g + (u & 3) >= live) s[u] = -INFINITY;
  }
  float top = s[0];
#pragma unroll
  for (int u = 1; u < 8; ++u) top = fmaxf(top, s[u]);
  const float m = fmaxf(st.m, max_over_groups(top));
  const float ref = m == -INFINITY ? 0.f : m;
  const float keep = __builtin_amdgcn_exp2f(st.m - ref);
  st.m = m;
  float w[8];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    w[u] = __builtin_amdgcn_exp2f(s[u] - ref);
    sum += w[u];
  }
  st.l = st.l * keep + sum;
  u32x4 p[G];
#pragma unroll
  for (int u = 0; u < G; ++u) {
    float mids = st.mids[u] * keep;
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const f32x2 pair = lds.v[(16 * (j >> 2) + 4 * g + (j & 3)) * G + u];
      r[j] = w[j] * pair[0];
      mids = __builtin_fmaf(w[j], pair[1], mids);
    }
    st.mids[u] = mids;
#pragma unroll
    for (int x = 0; x < 4; ++x) p[u][x] = pack2<kF16>(r[2 * x], r[2 * x + 1]);
  }
  if (__any(keep != 1.f)) {
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int n = 0; n < 4; ++n) st.o[u][n] *= keep;
  }
#pragma unroll
  for (int u = 0; u < G; ++u) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const u32x4 a = {centred(t.v[0][2 * u], n), centred(t.v[0][2 * u + 1], n), centred(t.v[1][2 * u], n),
                       centred(t.v[1][2 * u + 1], n)};
      st.o[u][n] = mfma16x16x32<kF16>(a, p[u], st.o[u][n]);
    }
  }
  wave_lds_sync();  // the pairs have been read
}

template <int DT, int DIM>
__global__ void __launch_bounds__(256, 2) decode4_attention_kernel(AttentionArgs a, DecodeAttentionPlan plan,
                                                                   uint32_t *__restrict__ counters,
                                                                   float *__restrict__ partials) {
  constexpr int G = DIM / 64, KS = DIM / 32;
  __shared__ DecodeJoin<DIM> lds;
  __shared__ __align__(16) Shared<DIM> pairs[kDecodeWaves];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  // (the order of the workgroups as in attention_decode.hip)
  const int split = blockIdx.z;
  const int tile = (int)(blockIdx.x % plan.head_tiles), kvh = (int)(blockIdx.x / plan.head_tiles);
  const int64_t row = blockIdx.y;
  const int heads = min(16, a.group - 16 * tile);  // query heads of this workgroup
  const int head0 = kvh * a.group + 16 * tile;
  const int slot = a.slots[row];
  // Q^T fragments: lane: head lane%16, channels 32 x + 8 g..; unused heads zero
  u32x4 q[KS];
  float qsum[G];
  int shift;  // scores are 2^shift times the products' sums
  {
    const int h = lane & 15;
    const uint16_t *qp = a.q + row * a.q_token + (int64_t)(head0 + min(h, heads - 1)) * a.q_head + 8 * (lane >> 4);
    float most = 0.f;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      q[x] = *reinterpret_cast<const u32x4 *>(qp + 32 * x);
      if (h >= heads) q[x] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(act_to_f32<DT>(q[x][j / 2] >> (16 * (j & 1)) & 0xffffu)));
    }
    most = max_over_groups(most);
    int e = 0;
    if (most < INFINITY) (void)frexpf(most, &e);  // most < 2^e
#pragma unroll
    for (int u = 0; u < G; ++u) qsum[u] = 0.f;
#pragma unroll
    for (int x = 0; x < KS; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f0 = ldexpf(act_to_f32<DT>(q[x][j] & 0xffffu), 15 - e);
        const float f1 = ldexpf(act_to_f32<DT>(q[x][j] >> 16), 15 - e);
        qsum[x / 2] += f0 + f1;
        const float part = j & 1 ? 0x1p-4f : 1.f;
        q[x][j] = pack2<kF16>(f0 * part, f1 * part);
      }
#pragma unroll
    for (int u = 0; u < G; ++u) qsum[u] = sum_over_groups(qsum[u]) * 0x1p-24f;
    shift = 24 - 15 + e;
  }
  const int len = a.kv.length(slot);
  // equal parts of whole steps
  const int part = len <= kWhole ? kWhole
                                 : (int)((((int64_t)len + plan.splits - 1) / plan.splits + kUnit - 1) / kUnit * kUnit);
  const int parts = max(1, (len + part - 1) / part);
  if (split >= parts) return;
  const int begin = split * part, end = min(len, begin + part);

  State<DIM> st;
#pragma unroll
  for (int u = 0; u < G; ++u) {
    st.mids[u] = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) st.o[u][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  st.m = -INFINITY;
  st.l = 0.f;
  st.ev = kLeastExponent;
  const float scale2 = a.scale * 1.44269504088896340736f;
  if (begin + wave * kStep < end) {
    Pages<DIM> pg;
    pg.table = a.kv.table + (int64_t)slot * a.kv.max_pages;
    pg.page_bytes = a.kv.page_stride * 2;
    pg.head_offset = kvh * Kv4<DIM>::head_bytes(1 << a.kv.page_shift);
    pg.last = (len - 1) >> a.kv.page_shift;
    pg.num_pages = a.kv.num_pages;
    pg.shift = a.kv.page_shift;
    const char *k = (const char *)a.kv.k, *v = (const char *)a.kv.v;
    int pos = begin + wave * kStep;
    // two tiles in turn: one is worked on while the other is loaded
    Tile<DIM> t0, t1;
    load_tile<DIM>(t0, k, v, pg.at(pos), pg.at(pos + 16), lane);
    typename Pages<DIM>::At n0 = pg.at(pos + kUnit), n1 = pg.at(pos + kUnit + 16);
    while (true) {
      if (pos + kUnit < end) load_tile<DIM>(t1, k, v, n0, n1, lane);
      n0 = pg.at(pos + 2 * kUnit);
      n1 = pg.at(pos + 2 * kUnit + 16);
      step<DT, DIM>(st, t0, pairs[wave], q, qsum, scale2, shift, end - pos, lane);
      pos += kUnit;
      if (pos >= end) break;
      if (pos + kUnit < end) load_tile<DIM>(t0, k, v, n0, n1, lane);
      n0 = pg.at(pos + 2 * kUnit);
      n1 = pg.at(pos + 2 * kUnit + 16);
      step<DT, DIM>(st, t1, pairs[wave], q, qsum, scale2, shift, end - pos, lane);
      pos += kUnit;
      if (pos >= end) break;
    }
  }
  // ---- join the waves ----
  const float l = sum_over_groups(st.l);
  float mids[G];
#pragma unroll
  for (int u = 0; u < G; ++u) mids[u] = sum_over_groups(st.mids[u]);
  {
    const int h = lane & 15, g = lane >> 4;
    if (g == 0) {
      lds.m[wave][h] = st.m;
      lds.l[wave][h] = l;
    }
    if (h < heads) {
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f32x4 x;
#pragma unroll
          for (int n = 0; n < 4; ++n)
            x[n] = ldexpf(st.o[u][n][i], (n & 1 ? 20 : 24) - 15 + st.ev) + mids[u];
          *reinterpret_cast<f32x4 *>(&lds.o[wave][h][64 * u + 16 * g + 4 * i]) = x;
        }
    }
  }
  join_parts<DT, DIM>(a, plan, lds, counters, partials, row, kvh, tile, heads, split, parts, len);
}

}  // namespace

hipError_t launch_attention_decode4(const AttentionArgs &a, const DecodeAttentionPlan &p, uint32_t *counters,
                                    float *partials, hipStream_t st) {
  const dim3 grid((unsigned)(a.kv_heads * p.head_tiles), (unsigned)a.sequences, (unsigned)p.splits);
#define PARO_DECODE4(DT, DIM) \
  hipLaunchKernelGGL((decode4_attention_kernel<DT, DIM>), grid, dim3(256), 0, st, a, p, counters, partials)
  if (a.dt == kF16) {
    if (a.head_dim == 64) PARO_DECODE4(kF16, 64);
    else PARO_DECODE4(kF16, 128);
  } else {
    if (a.head_dim == 64) PARO_DECODE4(kBF16, 64);
    else PARO_DECODE4(kBF16, 128);
  }
#undef PARO_DECODE4
  return hipGetLastError();
}

}  // namespace paro
