// kv4_rows.hip - rows into the pages of a cache in four bits (paro_kv_append)
// and out of the pages of either kind of cache (paro_kv_read).
//
// A wave takes one row.  A lane takes eight channels, eight lanes a group of 64:
// lowest and greatest value by three exchanges inside eight lanes.
// The code is decided exactly, for any 16-bit inputs:
//   - scale = (greatest - low) / 15 is one division in 64 bits.
//   - q = (x - low) / scale is computed in fp32 with the scale's power of two
//     taken out (so that nothing overflows), which is within 2^-18 of the
//     quotient; f = floor(q) then says which half, f + 1/2, could be the border,
//     and x - low is compared with (f + 1/2) scale in 64 bits: above it the
//     code is f + 1, below f, on it the even one.  The three terms' sum is exact
//     for fp16; for bf16 where x and low are less than 2^45 apart in size.
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
  x = fminf(x, from_lane<kXor1>(x));
  x = fminf(x, from_lane<kXor2>(x));
  return fminf(x, from_lane<kMirror8>(x));
}
__device__ __forceinline__ float max8(float x) {
  x = fmaxf(x, from_lane<kXor1>(x));
  x = fmaxf(x, from_lane<kXor2>(x));
  return fmaxf(x, from_lane<kMirror8>(x));
}

struct Coded {
  uint32_t code[8];
  uint32_t pair;  // scale in the low half, low in the high one
};

// Eight channels of a group whose other channels the seven lanes beside have.
template <int DT>
__device__ __forceinline__ Coded quantise(u32x4 raw) {
  Coded out;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = act_to_f32<DT>(raw[i / 2] >> (16 * (i & 1)) & 0xffffu);
  float low = x[0], high = x[0], bad = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    low = fminf(low, x[i]);
    high = fmaxf(high, x[i]);
    bad = __builtin_fmaf(x[i], 0.f, bad);  // NaN if any is not finite
  }
  low = min8(low);
  high = max8(high);
  bad += from_lane<kXor1>(bad);
  bad += from_lane<kXor2>(bad);
  bad += from_lane<kMirror8>(bad);
  const float scale32 = (float)(((double)high - (double)low) / 15.0);
  const uint32_t sbits = pack2<DT>(scale32, 0.f);  // low half
  const float scale = act_to_f32<DT>(sbits & 0xffffu);
  if (bad != bad) {
    const uint32_t nan = DT == kF16 ? 0x7e007e00u : 0x7fc07fc0u;
    out.pair = nan;
#pragma unroll
    for (int i = 0; i < 8; ++i) out.code[i] = 0;
    return out;
  }
  out.pair = pack2<DT>(scale, low);
  // unit: a power of two that brings the scale near 1 (exact where 2^127 does)
  int e;
  (void)frexpf(scale, &e);
  const float unit = ldexpf(1.f, min(127, 1 - e));
  const float lowu = low * unit, inv = 1.f / (scale * unit);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = fminf(fmaxf(floorf(__builtin_fmaf(x[i], unit, -lowu) * inv), 0.f), 15.f);
    const double over = ((double)x[i] - (double)low) - ((double)f + 0.5) * (double)scale;
    const uint32_t c = (uint32_t)f;
    const uint32_t up = c + (over > 0.0 || (over == 0.0 && (c & 1u)) ? 1u : 0u);
    out.code[i] = scale > 0.f ? min(up, 15u) : 0u;
  }
  return out;
}

// K and V rows of the newest positions into the pages; where a row does not
// belong (see entry_of, named_before, newest_position, page_at) it is skipped.
template <int DT, int DIM>
__global__ void __launch_bounds__(256) append4_kernel(KvLayer kv, int kv_heads, const uint16_t *__restrict__ k,
                                                      int64_t k_token, int64_t k_head, const uint16_t *__restrict__ v,
                                                      int64_t v_token, int64_t v_head,
                                                      const int32_t *__restrict__ slots,
                                                      const int64_t *__restrict__ cu,
                                                      const int32_t *__restrict__ granted, int n, int64_t tokens) {
  typedef Kv4<DIM> L;
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
  const int size = 1 << kv.page_shift, p = (int)(pos & (size - 1));
  const int pairs = L::pairs_at(size) + p * L::kGroups * 4;
  // whole groups of eight lanes stay or leave
  for (int c = lane * 8; c < kv_heads * DIM; c += 512) {
    const int h = c / DIM, d = c % DIM;
    const Coded a = quantise<DT>(*reinterpret_cast<const u32x4 *>(k + row * k_token + h * k_head + d));
    const Coded b = quantise<DT>(*reinterpret_cast<const u32x4 *>(v + row * v_token + h * v_head + d));
    char *kb = (char *)(kv.k + page * kv.page_stride) + h * L::head_bytes(size);
    char *vb = (char *)(kv.v + page * kv.page_stride) + h * L::head_bytes(size);
    uint32_t w = 0, w0 = 0, w1 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w |= a.code[i] << (4 * ((i >> 1) + 4 * (i & 1)));
      (i < 4 ? w0 : w1) |= b.code[i] << (4 * (i & 3));
    }
    *reinterpret_cast<uint32_t *>(kb + L::k_word(p, d / 8)) = w;
    *reinterpret_cast<uint16_t *>(vb + L::v_word(p, d / 4)) = (uint16_t)w0;
    *reinterpret_cast<uint16_t *>(vb + L::v_word(p, d / 4 + 1)) = (uint16_t)w1;
    if ((lane & 7) == 0) {
      *reinterpret_cast<uint32_t *>(kb + pairs + (d / kKv4Group) * 4) = a.pair;
      *reinterpret_cast<uint32_t *>(vb + pairs + (d / kKv4Group) * 4) = b.pair;
    }
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
__global__ void __launch_bounds__(256) read_kernel(KvReadArgs a) {
  typedef Kv4<DIM> L;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave_id();
  if (row >= a.tokens) return;
  const int lane = lane_id();
  Entry e;
  if (!entry_of(a.cu, a.n, row, a.tokens, lane, e)) return;
  const int s = a.slots[e.i], len = a.kv.length(s);
  const int64_t pos = a.first ? a.first[e.i] + (row - e.low) : (int64_t)len - (e.high - row);
  const int page = pos >= 0 && pos < len ? page_at(a.kv, s, pos) : -1;
  const int size = 1 << a.kv.page_shift, p = (int)(pos & (size - 1));
  for (int c = lane * 8; c < a.kv_heads * DIM; c += 512) {
    const int h = c / DIM, d = c % DIM;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      void *to = w ? a.v : a.k;
      if (!to) continue;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (page >= 0) {
        const uint16_t *base = (w ? a.kv.v : a.kv.k) + page * a.kv.page_stride;
        if constexpr (FOUR) {
          const char *from = (const char *)base + h * L::head_bytes(size);
          const uint32_t pair =
              *reinterpret_cast<const uint32_t *>(from + L::pairs_at(size) + (p * L::kGroups + d / kKv4Group) * 4);
          const float scale = act_to_f32<DT>(pair & 0xffffu), low = act_to_f32<DT>(pair >> 16);
          const uint32_t word = w ? *reinterpret_cast<const uint16_t *>(from + L::v_word(p, d / 4)) |
                                        (uint32_t)*reinterpret_cast<const uint16_t *>(from + L::v_word(p, d / 4 + 1)) << 16
                                  : *reinterpret_cast<const uint32_t *>(from + L::k_word(p, d / 8));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = w ? i : (i >> 1) + 4 * (i & 1);
            x[i] = __builtin_fmaf((float)(word >> (4 * n) & 15u), scale, low);
          }
        } else {
          const u32x4 r = *reinterpret_cast<const u32x4 *>(base + ((int64_t)h << a.kv.page_shift) * DIM + p * DIM + d);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = act_to_f32<DT>(r[i / 2] >> (16 * (i & 1)) & 0xffffu);
        }
      }
      store8<OUT>(to, row * (w ? a.v_token : a.k_token) + h * (w ? a.v_head : a.k_head) + d, x);
    }
  }
}

template <int DT, int OUT>
void launch_read(const KvReadArgs &a, hipStream_t st) {
  const dim3 grid((unsigned)((a.tokens + 3) / 4)), block(256);
  if (a.four) {
    if (a.head_dim == 64) hipLaunchKernelGGL((read_kernel<DT, OUT, 64, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((read_kernel<DT, OUT, 128, true>), grid, block, 0, st, a);
  } else {
    if (a.head_dim == 64) hipLaunchKernelGGL((read_kernel<DT, OUT, 64, false>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((read_kernel<DT, OUT, 128, false>), grid, block, 0, st, a);
  }
}

}  // namespace

hipError_t launch_kv_append4(const KvLayer &kv, int kv_heads, int head_dim, int dt, const uint16_t *k,
                             int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token, int64_t v_head,
                             const int32_t *slots, const int64_t *cu, const int32_t *granted, int n, int64_t tokens,
                             hipStream_t st) {
  const dim3 grid((unsigned)((tokens + 3) / 4)), block(256);
#define PARO_APPEND4(DT, DIM)                                                                                    \
  hipLaunchKernelGGL((append4_kernel<DT, DIM>), grid, block, 0, st, kv, kv_heads, k, k_token, k_head, v, v_token, \
                     v_head, slots, cu, granted, n, tokens)
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
