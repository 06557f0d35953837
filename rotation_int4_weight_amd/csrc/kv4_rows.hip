// kv4_rows.hip - rows into the pages of a cache in four bits (paro_kv_append)
// and out of the pages of either kind of cache (paro_kv_read).
//
// A wave takes one row, or a share of it where there are few rows; a lane takes
// eight channels, eight lanes a group of 64: lowest and greatest value by three
// exchanges inside eight lanes.  The rows' loads pass while the wave looks up
// entry, slot, length and page, which depend on one another.
// The format's code is decided exactly for any 16-bit inputs, in fp32 except
// where that leaves it open:
//   - scale = (greatest - low) / 15 is taken in 64 bits where fp32 leaves open to
//     which 16-bit number it rounds.
//   - With t = x - low, t / scale + 2^7 in fp32 keeps multiples of 2^-16 and is
//     off by less than 2^-17 before: half of a code comes out as that half, and
//     the next addition, of 2^23, rounds it to the even code.  What is nearer
//     than 2^-16 to a half without being one may come out wrong.
//   - d = t - code scale says so: a fused multiply-add has it exactly where it
//     is near half of the scale.  |d| under that half: the code is right.  Over
//     it, or equal to it with a t that fp32 rounded: the wave decides in 64 bits,
//     by the sign of t - (floor(t / scale) + 1/2) scale.
//   - So are groups whose scale is near the ends of fp32, moved to its middle by
//     a power of two first, or subnormal (there 15 may be the limit).
// What bounds it, in rows of 8 heads of 128 channels (a copy moves 4.8 to 5.0 TB/s):
//   - 64 rows are written in 4.1 us and read in 3.7, launch and look-ups.
//   - 4096 are written in 10.8 us (21.5 MB, 4.3 us at a copy's rate).  The waves,
//     four on a SIMD, wait half of their cycles, for entry, slot, length and page in
//     turn and then for pieces that are loaded one ahead; vector instructions take
//     27 % of the cycles.  V's 16-bit words reach memory as 7.3 MB for the 4.7 that
//     are held.
//   - 4096 are read as 16 bits in 7.8 us (21.5 MB; 9.7 with buffers in turn past the
//     last-level cache), as fp32 in 11.9 (38 MB).
//   - 95537 are read as 16 bits in 125 us: 501 MB, 4.0 TB/s, a quarter over a copy.
//     The waves wait 80 % of their cycles, and 147 MB are fetched for the 110 that
//     the rows hold: four waves read V's words of four positions, two bytes at a
//     time.  A cache in 16 bits (783 MB) is read in 145 us, 5.4 TB/s.

#include <math.h>

#include <algorithm>

#include "attention.hpp"
#include "common.hpp"
#include "kv4.hpp"
#include "kv_rows.hpp"

namespace paro {
namespace {

// The value of the lane that is 1, 2 (within four) or on the other half (of
// eight) away.
template <int CTRL>
__device__ __forceinline__ float from_lane(float x) {
  const int u = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(u, u, CTRL, 0xf, 0xf, false));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141;
__device__ __forceinline__ float min8(float x) {
  x = __builtin_elementwise_minimum(x, from_lane<kXor1>(x));
  x = __builtin_elementwise_minimum(x, from_lane<kXor2>(x));
  return __builtin_elementwise_minimum(x, from_lane<kMirror8>(x));
}
__device__ __forceinline__ float max8(float x) {
  x = __builtin_elementwise_maximum(x, from_lane<kXor1>(x));
  x = __builtin_elementwise_maximum(x, from_lane<kXor2>(x));
  return __builtin_elementwise_maximum(x, from_lane<kMirror8>(x));
}

// The codes where fp32 leaves one of them open (see the header).
template <int DT>
__device__ __forceinline__ void codes_in_64_bits(const float (&values)[8], float low, float scale, float (&code)[8]) {
  float unit = 1.f;
  if (scale > 0.f && !(scale > 0x1p-60f && scale < 0x1p60f)) {
    int e;
    (void)frexpf(scale, &e);
    unit = ldexpf(1.f, min(127, 1 - e));
  }
  const float mid = scale * unit, least_x = low * unit;
  const float inv = __builtin_amdgcn_rcpf(mid), half = 0.5f * mid, sure = inv * 0x1p30f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = values[i] * unit, t = x - least_x;
    const float f = floorf(t * inv);
    float d = __builtin_fmaf(-f, mid, t - half);
    const double d64 = ((double)x - (double)least_x) - ((double)f + 0.5) * (double)mid;
    // (its sign and zero are what counts)
    d = d == 0.f ? (d64 > 0.0 ? mid : d64 < 0.0 ? -mid : 0.f) : d;
    code[i] = __builtin_amdgcn_fmed3f(
        rintf(f + __builtin_amdgcn_fmed3f(__builtin_fmaf(d, sure, 0.5f), 0.25f, 0.75f)), 0.f, 15.f);
  }
}

// Eight channels of a group whose other channels the seven lanes beside have: the
// pair {scale, low}, and the codes as whole numbers; false: they are all 0.
template <int DT>
__device__ __forceinline__ bool quantise(u32x4 raw, uint32_t &pair, float (&code)[8]) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = act_to_f32<DT>(raw[i / 2] >> (16 * (i & 1)) & 0xffffu);
  float low = x[0], high = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    low = __builtin_elementwise_minimum(low, x[i]);  // (NaN stays NaN)
    high = __builtin_elementwise_maximum(high, x[i]);
  }
  low = min8(low);
  high = max8(high);
  const bool none = !(fabsf(low) < INFINITY && fabsf(high) < INFINITY);
  // The scale's type has so few bits that a fifteenth of the range from fp32
  // products, good to 2^-22, rounds as the exact one does, unless a border
  // between two of its numbers lies that near (or the range leaves fp32's middle).
  const float range = high - low, fifteenth = range * (1.f / 15.f);
  pair = pack2<DT>(fifteenth * (1.f - 0x1p-22f), fifteenth * (1.f + 0x1p-22f));
  if (__any((pair & 0xffffu) != pair >> 16 || !(range >= 0x1p-100f && range < INFINITY)))
    pair = pack2<DT>((float)(((double)high - (double)low) / 15.0), 0.f);
  const float scale = act_to_f32<DT>(pair & 0xffffu);
  // (a subnormal scale may be so far off a fifteenth that codes need the limit)
  constexpr float kLeast = DT == kF16 ? 0x1p-14f : 0x1p-60f, kMost = DT == kF16 ? 0x1p16f : 0x1p60f;
  const float inv = __builtin_amdgcn_rcpf(scale), half = 0.5f * scale;
  float d[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = x[i] - low;
    code[i] = (__builtin_fmaf(t, inv, 0x1p7f) + 0x1p23f) - (0x1p23f + 0x1p7f);
    d[i] = __builtin_fmaf(-code[i], scale, t);
    far = fmaxf(far, fabsf(d[i]));
  }
  bool open = scale > 0.f && !(scale >= kLeast && scale < kMost);
  if (__any(far >= half)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = x[i] - low;
      open |= fabsf(d[i]) > half || (fabsf(d[i]) == half && (x[i] - t != low || t + low != x[i]));
    }
  }
  if (__any(open)) codes_in_64_bits<DT>(x, low, scale, code);
  pair = none ? (DT == kF16 ? 0x7e007e00u : 0x7fc07fc0u) : pack2<DT>(scale, low);
  return scale > 0.f && !none;
}

// Four codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t four(float a, float b, float c, float d) {
  return (uint32_t)__builtin_fmaf(__builtin_fmaf(__builtin_fmaf(d, 16.f, c), 16.f, b), 16.f, a);
}

// Shares of a row: its pieces of 512 channels (of K, then of V, where they are
// quantised; of both where they are read) are taken by `shares` waves in turn.
// Few rows are cut so, as one wave's arithmetic takes longer than the look-ups
// that each of them then repeats: up to 4096 waves (written and read back, 64
// rows 14.7 us with a wave each, 12.4 cut; 4096 rows 22.0 either way, cut into
// four 24.4).
constexpr int kChannels = 512;
int shares_of(int64_t rows, int pieces) {
  int n = 1;
  while (n < pieces && rows * n < 4096) n *= 2;
  return n;
}
__device__ __forceinline__ int wave_of_grid() {
  return __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + wave_id()));
}

// K and V rows of the newest positions into the pages; where a row does not
// belong (see entry_of, named_before, newest_position, page_at) it is skipped.
template <int DT, int DIM>
__global__ void __launch_bounds__(256) append4_kernel(KvLayer kv, int kv_heads, int shares,
                                                      const uint16_t *__restrict__ k, int64_t k_token, int64_t k_head,
                                                      const uint16_t *__restrict__ v, int64_t v_token, int64_t v_head,
                                                      const int32_t *__restrict__ slots,
                                                      const int64_t *__restrict__ cu,
                                                      const int32_t *__restrict__ granted, int n, int64_t tokens) {
  typedef Kv4<DIM> L;
  const int wave = wave_of_grid(), share = wave % shares;
  const int64_t row = wave / shares;
  if (row >= tokens) return;
  const int lane = lane_id();
  const int width = kv_heads * DIM, chunks = (width + kChannels - 1) / kChannels;
  // piece p: channels c.. of K or V; whole groups of eight lanes have one or have none
  const auto fetch = [&](int p) {
    const int c = (p % chunks) * kChannels + lane * 8;
    if (c >= width) return u32x4{0, 0, 0, 0};
    const bool second = p >= chunks;
    return *reinterpret_cast<const u32x4 *>((second ? v : k) + row * (second ? v_token : k_token) +
                                            c / DIM * (second ? v_head : k_head) + c % DIM);
  };
  u32x4 raw = fetch(share);  // (passes while the position is looked up)
  Entry e;
  if (!entry_of(cu, n, row, tokens, lane, e)) return;
  const int s = slots[e.i];
  const bool refused = granted && granted[e.i] == 0;
  float code[8];
  uint32_t pair;
  bool some = quantise<DT>(raw, pair, code);
  if (s < 0 || s >= kv.slots || refused || named_before(slots, e.i, lane)) return;
  const int64_t pos = newest_position(kv, s, e, row);
  if (pos < 0) return;
  const int page = page_at(kv, s, pos);
  if (page < 0) return;
  const int size = 1 << kv.page_shift, at = (int)(pos & (size - 1));
  for (int p = share; p < 2 * chunks; p += shares) {
    if (p != share) some = quantise<DT>(raw, pair, code);
    if (p + shares < 2 * chunks) raw = fetch(p + shares);
    const int c = (p % chunks) * kChannels + lane * 8, d = c % DIM;
    if (c >= width) continue;
    const bool second = p >= chunks;
    char *to = (char *)((second ? kv.v : kv.k) + page * kv.page_stride) + c / DIM * L::head_bytes(size);
    if (second) {
      *reinterpret_cast<uint16_t *>(to + L::v_word(at, d / 4)) = (uint16_t)(some ? four(code[0], code[1], code[2], code[3]) : 0u);
      *reinterpret_cast<uint16_t *>(to + L::v_word(at, d / 4 + 1)) = (uint16_t)(some ? four(code[4], code[5], code[6], code[7]) : 0u);
    } else {
      *reinterpret_cast<uint32_t *>(to + L::k_word(at, d / 8)) =
          some ? four(code[0], code[2], code[4], code[6]) | four(code[1], code[3], code[5], code[7]) << 16 : 0u;
    }
    if ((lane & 7) == 0)
      *reinterpret_cast<uint32_t *>(to + L::pairs_at(size) + (at * L::kGroups + d / kKv4Group) * 4) = pair;
  }
}

// eight values of a row to out_dt
template <int OUT>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&x)[8]) {
  if constexpr (OUT == kF32) {
    f32x4 *q = reinterpret_cast<f32x4 *>((float *)p + at);
    q[0] = f32x4{x[0], x[1], x[2], x[3]};
    q[1] = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    *reinterpret_cast<u32x4 *>((uint16_t *)p + at) =
        u32x4{pack2<OUT>(x[0], x[1]), pack2<OUT>(x[2], x[3]), pack2<OUT>(x[4], x[5]), pack2<OUT>(x[6], x[7])};
  }
}

template <int DT, int OUT, int DIM, bool FOUR>
__global__ void __launch_bounds__(256) read_kernel(KvReadArgs a, int shares) {
  typedef Kv4<DIM> L;
  const int wave = wave_of_grid(), share = wave % shares;
  const int64_t row = wave / shares;
  if (row >= a.tokens) return;
  const int lane = lane_id();
  Entry e;
  if (!entry_of(a.cu, a.n, row, a.tokens, lane, e)) return;
  const int s = a.slots[e.i], len = a.kv.length(s);
  const int64_t pos = a.first ? a.first[e.i] + (row - e.low) : (int64_t)len - (e.high - row);
  const int page = pos >= 0 && pos < len ? page_at(a.kv, s, pos) : -1;
  const int size = 1 << a.kv.page_shift, at = (int)(pos & (size - 1));
  const int width = a.kv_heads * DIM;
  const uint16_t *kp = a.kv.k + (int64_t)max(page, 0) * a.kv.page_stride,
                 *vp = a.kv.v + (int64_t)max(page, 0) * a.kv.page_stride;
  for (int c = share * kChannels + lane * 8; c < width; c += shares * kChannels) {
    const int h = c / DIM, d = c % DIM;
    const int64_t ko = row * a.k_token + h * a.k_head + d, vo = row * a.v_token + h * a.v_head + d;
    if constexpr (FOUR) {
      const char *kf = (const char *)kp + h * L::head_bytes(size), *vf = (const char *)vp + h * L::head_bytes(size);
      const int pair = L::pairs_at(size) + (at * L::kGroups + d / kKv4Group) * 4;
      uint32_t kw = 0, k2 = 0, v0 = 0, v1 = 0, v2 = 0;
      if (page >= 0) {
        if (a.k) {
          kw = *reinterpret_cast<const uint32_t *>(kf + L::k_word(at, d / 8));
          k2 = *reinterpret_cast<const uint32_t *>(kf + pair);
        }
        if (a.v) {
          v0 = *reinterpret_cast<const uint16_t *>(vf + L::v_word(at, d / 4));
          v1 = *reinterpret_cast<const uint16_t *>(vf + L::v_word(at, d / 4 + 1));
          v2 = *reinterpret_cast<const uint32_t *>(vf + pair);
        }
      }
      float x[8];
      if (a.k) {
        const float scale = act_to_f32<DT>(k2 & 0xffffu), low = act_to_f32<DT>(k2 >> 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = __builtin_fmaf((float)(kw >> (4 * ((i >> 1) + 4 * (i & 1))) & 15u), scale, low);
        store8<OUT>(a.k, ko, x);
      }
      if (a.v) {
        const float scale = act_to_f32<DT>(v2 & 0xffffu), low = act_to_f32<DT>(v2 >> 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_fmaf((float)((i < 4 ? v0 : v1) >> (4 * (i & 3)) & 15u), scale, low);
        store8<OUT>(a.v, vo, x);
      }
    } else {
      const int64_t from = ((int64_t)h << a.kv.page_shift) * DIM + at * DIM + d;
      u32x4 kr = {0, 0, 0, 0}, vr = {0, 0, 0, 0};
      if (page >= 0) {
        if (a.k) kr = *reinterpret_cast<const u32x4 *>(kp + from);
        if (a.v) vr = *reinterpret_cast<const u32x4 *>(vp + from);
      }
      if constexpr (OUT == DT) {
        if (a.k) *reinterpret_cast<u32x4 *>((uint16_t *)a.k + ko) = kr;
        if (a.v) *reinterpret_cast<u32x4 *>((uint16_t *)a.v + vo) = vr;
      } else {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = act_to_f32<DT>(kr[i / 2] >> (16 * (i & 1)) & 0xffffu);
        if (a.k) store8<OUT>(a.k, ko, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = act_to_f32<DT>(vr[i / 2] >> (16 * (i & 1)) & 0xffffu);
        if (a.v) store8<OUT>(a.v, vo, x);
      }
    }
  }
}

template <int DT, int OUT, int DIM, bool FOUR>
void launch_read(const KvReadArgs &a, hipStream_t st) {
  const int shares = shares_of(a.tokens, (a.kv_heads * a.head_dim + kChannels - 1) / kChannels);
  const dim3 grid((unsigned)((a.tokens * shares + 3) / 4)), block(256);
  hipLaunchKernelGGL((read_kernel<DT, OUT, DIM, FOUR>), grid, block, 0, st, a, shares);
}
template <int DT, int OUT>
void launch_read(const KvReadArgs &a, hipStream_t st) {
  if (a.four) {
    if (a.head_dim == 64) launch_read<DT, OUT, 64, true>(a, st);
    else launch_read<DT, OUT, 128, true>(a, st);
  } else {
    if (a.head_dim == 64) launch_read<DT, OUT, 64, false>(a, st);
    else launch_read<DT, OUT, 128, false>(a, st);
  }
}

}  // namespace

hipError_t launch_kv_append4(const KvLayer &kv, int kv_heads, int head_dim, int dt, const uint16_t *k,
                             int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                             const int32_t *slots, const int64_t *cu, const int32_t *granted, int n, int64_t tokens,
                             hipStream_t st) {
  const int shares = shares_of(tokens, 2 * ((kv_heads * head_dim + kChannels - 1) / kChannels));
  const dim3 grid((unsigned)((tokens * shares + 3) / 4)), block(256);
#define PARO_APPEND4(DT, DIM)                                                                                    \
  hipLaunchKernelGGL((append4_kernel<DT, DIM>), grid, block, 0, st, kv, kv_heads, shares, k, k_token, k_head, v, \
                     v_token, v_head, slots, cu, granted, n, tokens)
  if (dt == kF16) {
    if (head_dim == 64) PARO_APPEND4(kF16, 64);
    else PARO_APPEND4(kF16, 128);
  } else {
    if (head_dim == 64) PARO_APPEND4(kBF16, 64);
    else PARO_APPEND4(kBF16, 128);
  }
#undef PARO_APPEND4
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs &a, hipStream_t st) {
  if (a.dt == kF16) {
    if (a.out_dt == kF32) launch_read<kF16, kF32>(a, st);
    else launch_read<kF16, kF16>(a, st);
  } else {
    if (a.out_dt == kF32) launch_read<kBF16, kF32>(a, st);
    else launch_read<kBF16, kBF16>(a, st);
  }
  return hipGetLastError();
}

}  // namespace paro
