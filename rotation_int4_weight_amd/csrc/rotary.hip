// rotary.hip - rotary positions of query and key heads (paro_rotary).
//
// Every element is read and written once; the angles depend on (token, pair)
// alone and are shared by all heads.  A workgroup takes as many tokens as have
// 256 pairs together (at least one): each thread takes one sine and cosine into
// LDS, then the threads go over the tokens' heads in units of 16 bytes.
//   - y is stored as the next kernel would have it, in the caches: stored past
//     them, 4096 tokens of 40 heads take 14.5 instead of 19.3 us, and a copy that
//     reads y afterwards 7.6 us more.
//   - The angle is reduced in 64 bits: position times frequency, less the
//     nearest whole number of quarter turns, leaves at most half of one, whose
//     fp32 value is off by 2^-26 of a quarter turn; the quarters are put back by
//     exchanging sine and cosine.  fp32 angles would be off by 2^-24 of the
//     angle itself, 0.06 radians at position 2^20.
// What bounds it: bytes, read and written once (counters: 42.2 and 41.9 MB of 41.9).
// 4096 tokens of 40 heads of 128 channels (84 MB in 16 bits) take 20.9 us with
// buffers in turn past the last-level cache, 4.0 TB/s, and 14.5 in the same ones
// again, 2048 tokens of 32 heads in fp32 (67 MB) 16.0 and 12.2; a copy of 1 GiB moves
// 4.8 to 5.0.  One token 2.6 us, a launch; 778 far ones of 14 heads of 64 channels
// 3.2.  Units are as wide as the pairs' number allows: 2000 tokens of 24 heads of 128
// channels (24.6 MB), 128, 124 and 126 of them turned, take 6.3, 9.1 and 11.4.
#include <math.h>

#include <algorithm>

#include "common.hpp"
#include "rotary.hpp"

namespace paro {
namespace {

constexpr int kThreads = 256;
constexpr int kWorkgroups = 2048;  // a launch has, if it can (4096 tokens of 40 heads: 512 20.9 us, 2048 19.3)
constexpr double k2OverPi = 0.63661977236758134308;
constexpr double kPiOver2 = 1.57079632679489661923, kPiOver2Low = 6.123233995736766e-17;  // pi / 2 in two parts

template <int BYTES>
struct Raw;
template <>
struct Raw<2> { typedef uint16_t type; };
template <>
struct Raw<4> { typedef uint32_t type; };
template <>
struct Raw<8> { typedef u32x2 type; };
template <>
struct Raw<16> { typedef u32x4 type; };

// V consecutive elements
template <int DT, int V>
struct Piece {
  static constexpr int kSize = DT == kF32 ? 4 : 2;
  typedef typename Raw<V * kSize>::type type;
  static __device__ __forceinline__ type load(const void *p, int64_t at) {
    return *reinterpret_cast<const type *>((const char *)p + at * kSize);
  }
  static __device__ __forceinline__ void store(void *p, int64_t at, type x) {
    *reinterpret_cast<type *>((char *)p + at * kSize) = x;
  }
  static __device__ __forceinline__ void open(type x, float (&f)[V]) {
    if constexpr (DT == kF32) {
      struct { float f[V]; } t = __builtin_bit_cast(decltype(t), x);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = t.f[i];
    } else {
      struct { uint16_t h[V]; } t = __builtin_bit_cast(decltype(t), x);
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = act_to_f32<DT>(t.h[i]);
    }
  }
  static __device__ __forceinline__ type close(const float (&f)[V]) {
    if constexpr (DT == kF32) {
      struct { float f[V]; } t;
#pragma unroll
      for (int i = 0; i < V; ++i) t.f[i] = f[i];
      return __builtin_bit_cast(type, t);
    } else if constexpr (V == 1) {
      return DT == kF16 ? f32_to_f16_bits(f[0]) : f32_to_bf16_bits(f[0]);
    } else {
      struct { uint32_t w[V / 2]; } t;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) t.w[i] = pack2<DT>(f[2 * i], f[2 * i + 1]);
      return __builtin_bit_cast(type, t);
    }
  }
};

// n / d for n * d < 2^32, with m = ceil(2^32 / d) (d > 1; d == 1: m = 0)
__device__ __forceinline__ int divide(int n, uint32_t m) { return m ? (int)__umulhi((uint32_t)n, m) : n; }

// Channels of a unit that is copied: the first of them is a multiple of twice the
// pairs' common divisor that V is.
template <int DT, int V, bool INTERLEAVED>
constexpr int rest_unit() {
  return INTERLEAVED || V == (DT == kF32 ? 4 : 8) ? V : 2 * V;
}

struct Split {
  int tokens, heads;         // of a workgroup
  int turned, units;         // units of a head: the turned ones, all
  uint32_t by_units, by_heads;  // for divide()
};

template <int DT, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a, Split w) {
  typedef Piece<DT, V> P;
  constexpr int kRest = rest_unit<DT, V, INTERLEAVED>();
  __shared__ float2 turn[kThreads];  // [token][pair]
  const int64_t token0 = (int64_t)blockIdx.x * w.tokens;
  const int head0 = blockIdx.y * w.heads;
  const int tokens = (int)min((int64_t)w.tokens, a.tokens - token0), heads = min(w.heads, a.heads - head0);
  const int items = tokens * w.heads * w.units;
  const bool in_place = a.x == a.y;
  // An item is a unit of a token's head: where it lies, and its loads (the second
  // one for the other half of the pairs)
  struct Item {
    int row, unit;
    int64_t from, to;  // element of the first load and store, negative: no item
    typename P::type x, y;
  };
  const auto fetch = [&](int n) {
    Item t;
    const int rh = divide(n, w.by_units);
    t.unit = n - rh * w.units;
    t.row = divide(rh, w.by_heads);
    const int h = rh - t.row * w.heads;
    t.from = -1;
    t.x = t.y = typename P::type{};
    const bool rest = t.unit >= w.turned;
    if (n >= items || h >= heads || (rest && in_place)) return t;
    const int c = rest ? 2 * a.pairs + (t.unit - w.turned) * kRest : t.unit * V;
    t.from = (token0 + t.row) * a.x_token + (head0 + h) * a.x_head + c;
    t.to = (token0 + t.row) * a.y_token + (head0 + h) * a.y_head + c;
    t.x = P::load(a.x, t.from);
    if (rest ? kRest > V : !INTERLEAVED) t.y = P::load(a.x, t.from + (rest ? V : a.pairs));
    return t;
  };
  Item next = fetch(threadIdx.x);  // (passes while the angles are taken)
  for (int t = threadIdx.x; t < tokens * a.pairs; t += kThreads) {
    const int row = t / a.pairs, i = t - row * a.pairs;
    const double angle = (double)a.positions[token0 + row] * a.freqs[i];
    const double whole = rint(angle * k2OverPi);
    const double rest = fma(-whole, kPiOver2Low, fma(-whole, kPiOver2, angle));
    float s, c;
    sincospif((float)(rest * k2OverPi) * 0.5f, &s, &c);
    const int q = (int)(whole - 4.0 * floor(whole * 0.25));
    float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
    if (q == 1 || q == 2) cs = -cs;
    if (q >= 2) sn = -sn;
    turn[t] = make_float2(cs * a.magnitude, (a.inverse ? -sn : sn) * a.magnitude);
  }
  __syncthreads();
#pragma unroll 2
  for (int n = threadIdx.x; n < items; n += kThreads) {
    const Item t = next;
    next = fetch(n + kThreads);
    if (t.from < 0) continue;
    if (t.unit >= w.turned) {
      P::store(a.y, t.to, t.x);
      if constexpr (kRest > V) P::store(a.y, t.to + V, t.y);
      continue;
    }
    const float2 *cs = turn + t.row * a.pairs;
    if constexpr (INTERLEAVED) {
      float f[V], g[V];
      P::open(t.x, f);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 r = cs[(t.unit * V + i) / 2];
        g[i] = __builtin_fmaf(f[i], r.x, -(f[i + 1] * r.y));
        g[i + 1] = __builtin_fmaf(f[i + 1], r.x, f[i] * r.y);
      }
      P::store(a.y, t.to, P::close(g));
    } else {
      float fa[V], fb[V], ga[V], gb[V];
      P::open(t.x, fa);
      P::open(t.y, fb);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 r = cs[t.unit * V + i];
        ga[i] = __builtin_fmaf(fa[i], r.x, -(fb[i] * r.y));
        gb[i] = __builtin_fmaf(fb[i], r.x, fa[i] * r.y);
      }
      P::store(a.y, t.to, P::close(ga));
      P::store(a.y, t.to + a.pairs, P::close(gb));
    }
  }
}

uint32_t magic(int d) { return d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d); }

template <int DT, int V, bool INTERLEAVED>
void launch(const RotaryArgs &a, hipStream_t st) {
  Split w;
  w.turned = INTERLEAVED ? 2 * a.pairs / V : a.pairs / V;
  w.units = w.turned + (a.head_dim - 2 * a.pairs) / rest_unit<DT, V, INTERLEAVED>();
  // as many tokens as share 256 angles, fewer and then fewer heads where that
  // leaves CUs idle (divide() needs items * divisor below 2^32)
  w.heads = a.heads;
  w.tokens = std::max(1, std::min(kThreads / a.pairs, 65536 / (w.heads * w.units)));
  const int64_t want = std::max<int64_t>(1, a.tokens / kWorkgroups);
  w.tokens = (int)std::min<int64_t>(w.tokens, want);
  while (w.heads > 1 && w.tokens * w.heads * w.units > kThreads &&
         (a.tokens + w.tokens - 1) / w.tokens * ((a.heads + w.heads - 1) / w.heads) < kWorkgroups)
    w.heads = (w.heads + 1) / 2;
  w.by_units = magic(w.units);
  w.by_heads = magic(w.heads);
  const dim3 grid((unsigned)((a.tokens + w.tokens - 1) / w.tokens), (unsigned)((a.heads + w.heads - 1) / w.heads));
  hipLaunchKernelGGL((rotary_kernel<DT, V, INTERLEAVED>), grid, dim3(kThreads), 0, st, a, w);
}

template <int DT>
void launch_typed(const RotaryArgs &a, hipStream_t st) {
  constexpr int V = DT == kF32 ? 4 : 8;  // 16 bytes
  // units as wide as the pairs allow
  if (a.interleaved) {
    if (2 * a.pairs % V == 0) launch<DT, V, true>(a, st);
    else if (V > 4 && a.pairs % 2 == 0) launch<DT, 4, true>(a, st);
    else launch<DT, 2, true>(a, st);
  } else {
    if (a.pairs % V == 0) launch<DT, V, false>(a, st);
    else if (V > 4 && a.pairs % 4 == 0) launch<DT, 4, false>(a, st);
    else if (a.pairs % 2 == 0) launch<DT, 2, false>(a, st);
    else launch<DT, 1, false>(a, st);
  }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
  if (a.dt == kF16) launch_typed<kF16>(a, st);
  else if (a.dt == kBF16) launch_typed<kBF16>(a, st);
  else launch_typed<kF32>(a, st);
  return hipGetLastError();
}

}  // namespace paro
