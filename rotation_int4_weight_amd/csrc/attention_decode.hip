// attention_decode.hip - attention of one new token per sequence over the
// paged cache (paro_attention_decode).
//
// Every live K and V row is read once, so the time is that of reading the
// cache: 4 * head_dim * kv_heads bytes per position.  The work is arranged so
// that nothing but the loads takes part in the wait:
//   - A workgroup takes one row's key-value head with up to 16 of its query
//     heads (they read the same K and V), and one part of the length; its
//     four waves take 32 keys at a time in turn.
//   - S^T = K Q^T and O^T = V^T P^T run on v_mfma_f32_16x16x32.  A wave loads
//     K straight into A fragments (lane: key lane%16, 16 bytes of channels).
//     S^T leaves lane (head lane%16, group g = lane/16) with the keys 4g..4g+3
//     of two 16-key blocks: exactly the 8 keys that the lane feeds to the
//     second product if its keys are numbered that way, so the weights never
//     leave their lane.  V is loaded by rows (16 lanes cover one key's
//     channels) and turned into V^T fragments by v_perm in the lane.
//   - The head stays in lane%16 from S^T to O^T, so maxima and sums are per
//     lane; only the maximum crosses lanes (two permlane swaps per 32 keys).
//   - fp16 weights are exp2(s - m + 15) (inside the type; the quotient is the
//     same), so that those down to 2^-29 of the largest stay above its
//     subnormals: a long row may have many.
//   - 32 keys of K and V are in flight per wave while 32 are worked on.
// Parts are joined with their maxima (through LDS between the waves, through
// the workspace between workgroups, by the last one to arrive, in order).
// Measured (32 query heads over 8 of 128 channels, bf16, 16-position pages):
// 64 rows of 4096 187 us, 5.7 TB/s; 64 rows of 1 to 4096 104 us, 4.8 TB/s (all
// rows are resident at once, so the CUs with long rows end last; cutting them
// further gave 108 to 118 us); rows of 131072 and 100001 166 us, 5.7 TB/s; one
// row of 777 7.2 us, of 100 4.1 us.  A copy of 1 GiB moves 4.8 TB/s.
#include <math.h>

#include <algorithm>

#include "attention.hpp"
#include "attention_join.hpp"
#include "common.hpp"
#include "mfma.hpp"

namespace paro {
namespace {

constexpr int kWaves = kDecodeWaves;
constexpr int kStep = 32;           // keys per wave and step
constexpr int kUnit = kStep * kWaves;  // keys per workgroup and step
// Rows up to this length are not cut: joining parts costs 2 to 3 us (stores, a
// counter and loads through the coherent levels), one step about 1 us (whole
// and in parts: one row of 300 6.5 and 6.7 us, of 450 8.0 and 7.0; 16 rows of
// 300 6.7 and 8.7).
constexpr int kWhole = 3 * kUnit;
constexpr int64_t kCus = 256;

template <int DIM>
struct Tile {
  static constexpr int KS = DIM / 32;      // contraction steps of S^T
  static constexpr int E = DIM / 16;       // channels per lane of a V row
  u32x4 k[2][KS];                          // [16-key block][step]
  uint32_t v[8][E / 2];                    // [key of the lane][channel pair]
};

// First element of 16 consecutive positions (they lie in one page).
struct Pages {
  const int32_t *table;
  int64_t page_stride, head_offset;
  int last, num_pages, shift, dim;
  __device__ __forceinline__ int64_t at(int pos) const {
    const int j = min(pos >> shift, last);
    int page = table[j];
    page = page < 0 ? 0 : page >= num_pages ? num_pages - 1 : page;
    return (int64_t)page * page_stride + head_offset + (int64_t)(pos & ((1 << shift) - 1)) * dim;
  }
};

template <int DIM>
__device__ __forceinline__ void load_tile(Tile<DIM> &t, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
                                          int64_t a0, int64_t a1, int lane) {
  constexpr int E = Tile<DIM>::E;
  const int r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint16_t *kb = k + (b ? a1 : a0) + r * DIM + 8 * g;
#pragma unroll
    for (int s = 0; s < Tile<DIM>::KS; ++s) t.k[b][s] = *reinterpret_cast<const u32x4 *>(kb + 32 * s);
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const uint16_t *vb = v + (b ? a1 : a0) + 4 * g * DIM + r * E;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E == 8) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(vb + i * DIM);
#pragma unroll
        for (int c = 0; c < 4; ++c) t.v[4 * b + i][c] = x[c];
      } else {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(vb + i * DIM);
#pragma unroll
        for (int c = 0; c < 2; ++c) t.v[4 * b + i][c] = x[c];
      }
    }
  }
}

template <int DIM>
struct State {
  f32x4 o[DIM / 16];  // o[j][i]: channel (4 * group + i) * E + j of the lane's head
  float m, l;         // maximum (of scores * log2 e) and this lane's share of the sum
};

// One step: 32 keys, `live` of them in the sequence (>= 32 but at its end).
template <int DT, int DIM>
__device__ __forceinline__ void step(State<DIM> &st, Tile<DIM> &t, const u32x4 (&q)[DIM / 32], float scale2, int live,
                                     int lane) {
  constexpr int E = Tile<DIM>::E, KS = Tile<DIM>::KS;
  const int g = lane >> 4;
  float s[8];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < KS; ++x) c = mfma16x16x32<DT>(t.k[b][x], q[x], c);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[4 * b + i] = c[i] * scale2;
  }
  if (live < kStep) {
    // the end of the sequence: what the page holds behind it does not count,
    // and its V rows are cleared, since 0 * NaN is NaN
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (16 * (u >> 2) + 4 * g + (u & 3) >= live) {
        s[u] = -INFINITY;
#pragma unroll
        for (int c = 0; c < E / 2; ++c) t.v[u][c] = 0;
      }
    }
  }
  float top = s[0];
#pragma unroll
  for (int u = 1; u < 8; ++u) top = fmaxf(top, s[u]);
  const float m = fmaxf(st.m, max_over_groups(top));
  const float ref = m == -INFINITY ? 0.f : m;
  const float keep = __builtin_amdgcn_exp2f(st.m - ref);
  st.m = m;
  u32x4 p;
  float sum = 0.f;
  const float low = ref - (DT == kF16 ? 15.f : 0.f);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float e0 = __builtin_amdgcn_exp2f(s[2 * u] - low), e1 = __builtin_amdgcn_exp2f(s[2 * u + 1] - low);
    sum += e0 + e1;
    p[u] = pack2<DT>(e0, e1);
  }
  st.l = st.l * keep + sum;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    st.o[j] *= keep;
    u32x4 a;
#pragma unroll
    for (int x = 0; x < 4; ++x)  // keys 2x, 2x + 1 of channel j
      a[x] = __builtin_amdgcn_perm(t.v[2 * x + 1][j / 2], t.v[2 * x][j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
    st.o[j] = mfma16x16x32<DT>(a, p, st.o[j]);
  }
}

template <int DT, int DIM>
__global__ void __launch_bounds__(256, 2) decode_attention_kernel(AttentionArgs a, DecodeAttentionPlan plan,
                                                                  uint32_t *__restrict__ counters,
                                                                  float *__restrict__ partials) {
  constexpr int E = DIM / 16;
  __shared__ DecodeJoin<DIM> lds;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  // The part is the slowest index: workgroups go to the XCDs in turn, and with
  // it the fastest those that have work (short rows have one part) would sit on
  // few of them.
  const int split = blockIdx.z;
  const int tile = (int)(blockIdx.x % plan.head_tiles), kvh = (int)(blockIdx.x / plan.head_tiles);
  const int64_t row = blockIdx.y;
  const int heads = min(16, a.group - 16 * tile);  // query heads of this workgroup
  const int head0 = kvh * a.group + 16 * tile;
  const int slot = a.slots[row];
  // Q^T fragments: lane: head lane%16, channels 32 s + 8 g..; unused heads zero
  u32x4 q[DIM / 32];
  {
    const int h = lane & 15;
    const uint16_t *qp = a.q + row * a.q_token + (int64_t)(head0 + min(h, heads - 1)) * a.q_head + 8 * (lane >> 4);
#pragma unroll
    for (int s = 0; s < DIM / 32; ++s) {
      q[s] = *reinterpret_cast<const u32x4 *>(qp + 32 * s);
      if (h >= heads) q[s] = u32x4{0, 0, 0, 0};
    }
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
  for (int j = 0; j < E; ++j) st.o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  st.m = -INFINITY;
  st.l = 0.f;
  const float scale2 = a.scale * 1.44269504088896340736f;
  if (begin + wave * kStep < end) {
    Pages pg;
    pg.table = a.kv.table + (int64_t)slot * a.kv.max_pages;
    pg.page_stride = a.kv.page_stride;
    pg.head_offset = ((int64_t)kvh << a.kv.page_shift) * DIM;
    pg.last = (len - 1) >> a.kv.page_shift;
    pg.num_pages = a.kv.num_pages;
    pg.shift = a.kv.page_shift;
    pg.dim = DIM;
    int pos = begin + wave * kStep;
    // two tiles in turn: one is worked on while the other is loaded; the
    // addresses of the one after are looked up meanwhile
    Tile<DIM> t0, t1;
    load_tile<DIM>(t0, a.kv.k, a.kv.v, pg.at(pos), pg.at(pos + 16), lane);
    int64_t n0 = pg.at(pos + kUnit), n1 = pg.at(pos + kUnit + 16);
    while (true) {
      if (pos + kUnit < end) load_tile<DIM>(t1, a.kv.k, a.kv.v, n0, n1, lane);
      n0 = pg.at(pos + 2 * kUnit);
      n1 = pg.at(pos + 2 * kUnit + 16);
      step<DT, DIM>(st, t0, q, scale2, end - pos, lane);
      pos += kUnit;
      if (pos >= end) break;
      if (pos + kUnit < end) load_tile<DIM>(t0, a.kv.k, a.kv.v, n0, n1, lane);
      n0 = pg.at(pos + 2 * kUnit);
      n1 = pg.at(pos + 2 * kUnit + 16);
      step<DT, DIM>(st, t1, q, scale2, end - pos, lane);
      pos += kUnit;
      if (pos >= end) break;
    }
  }
  // ---- join the waves ----
  const float l = sum_over_groups(st.l);
  {
    const int h = lane & 15, g = lane >> 4;
    if (g == 0) {
      lds.m[wave][h] = st.m;
      lds.l[wave][h] = l;
    }
    if (h < heads) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          f32x4 x = {st.o[j][i], st.o[j + 1][i], st.o[j + 2][i], st.o[j + 3][i]};
          *reinterpret_cast<f32x4 *>(&lds.o[wave][h][(4 * g + i) * E + j]) = x;
        }
    }
  }
  const int64_t item = (row * a.kv_heads + kvh) * plan.head_tiles + tile;
  const int slots = plan.splits * part_floats(a.group, DIM);
  join_parts<DT, DIM, true>(a, lds, counters + item, raw_rsrc(partials + item * slots, (uint32_t)(slots * 4)),
                            PartsInOrder(), row, head0, heads, split, parts, len > 0);
}

}  // namespace

// One workgroup per CU streams the cache fastest: a second one adds only its
// own start and end (8 rows of 8192: 43.5 us with 256 workgroups, 45.1 with
// 512; one row of 32768: 27.2 and 30.4), so the parts fill the 256 CUs once.
// Between one and two workgroups per CU two parts even out the second round
// (40 rows of 4096: 124.6 us against 140.3); from two on, whole rows (64 rows
// of 4096: 187 us, 194 in two parts).  The rule looks at the number of rows, not
// at their lengths (they are on the device): 63 rows of 500 beside one of 131072
// take 1360 us, which eight workgroups spend on the long row, 667 MB that the
// whole card would read in 120; without the long row 23.5 us.
DecodeAttentionPlan plan_attention_decode(int64_t rows, int q_heads, int kv_heads, int64_t max_len) {
  DecodeAttentionPlan p;
  p.head_tiles = (q_heads / kv_heads + 15) / 16;
  const int64_t items = rows * kv_heads * p.head_tiles;
  const int64_t most = std::max<int64_t>(1, (max_len + kUnit - 1) / kUnit);
  p.splits = (int)std::min(most, items <= kCus ? kCus / items : items < 2 * kCus ? int64_t(2) : int64_t(1));
  return p;
}

size_t attention_decode_partial_bytes(const DecodeAttentionPlan &p, int64_t rows, int kv_heads, int head_dim) {
  if (p.splits == 1) return 0;
  return (size_t)rows * kv_heads * p.head_tiles * p.splits * 16 * (head_dim + 4) * 4;
}

hipError_t launch_attention_decode(const AttentionArgs &a, const DecodeAttentionPlan &p, uint32_t *counters,
                                   float *partials, hipStream_t st) {
  const dim3 grid((unsigned)(a.kv_heads * p.head_tiles), (unsigned)a.sequences, (unsigned)p.splits);
#define PARO_DECODE(DT, DIM) \
  hipLaunchKernelGGL((decode_attention_kernel<DT, DIM>), grid, dim3(256), 0, st, a, p, counters, partials)
  if (a.dt == kF16) {
    if (a.head_dim == 64) PARO_DECODE(kF16, 64);
    else PARO_DECODE(kF16, 128);
  } else {
    if (a.head_dim == 64) PARO_DECODE(kBF16, 64);
    else PARO_DECODE(kBF16, 128);
  }
#undef PARO_DECODE
  return hipGetLastError();
}

}  // namespace paro
