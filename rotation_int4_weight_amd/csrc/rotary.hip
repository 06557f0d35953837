// rotary.hip - rotary positions of query and key heads (paro_rotary).
//
// Every element is read and written once; the angles depend on (token, pair)
// alone and are shared by all heads.  A workgroup takes as many tokens as have
// 256 pairs together (at least one): each thread takes one sine and cosine into
// LDS, then the threads go over the tokens' heads in units of 16 bytes.
//   - The angle is reduced in 64 bits: position times frequency, less the
//     nearest whole number of quarter turns, leaves at most half of one, whose
//     fp32 value is off by 2^-26 of a quarter turn; the quarters are put back by
//     exchanging sine and cosine.  fp32 angles would be off by 2^-24 of the
//     angle itself, 0.06 radians at position 2^20.
#include <math.h>

#include <algorithm>

#include "common.hpp"
#include "rotary.hpp"

namespace paro {
namespace {

constexpr int kThreads = 256;
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

struct Split {
  int tokens, heads;         // of a workgroup
  int turned, units;         // units of a head: the turned ones, all
  uint32_t by_units, by_heads;  // for divide()
};

template <int DT, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a, Split w) {
  typedef Piece<DT, V> P;
  __shared__ float2 turn[kThreads];  // [token][pair]
  const int64_t token0 = (int64_t)blockIdx.x * w.tokens;
  const int head0 = blockIdx.y * w.heads;
  const int tokens = (int)min((int64_t)w.tokens, a.tokens - token0), heads = min(w.heads, a.heads - head0);
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
  const int items = tokens * w.heads * w.units;
  const bool in_place = a.x == a.y;
  for (int n = threadIdx.x; n < items; n += kThreads) {
    const int rh = divide(n, w.by_units), u = n - rh * w.units;
    const int row = divide(rh, w.by_heads), h = rh - row * w.heads;
    if (h >= heads) continue;
    const int64_t from = (token0 + row) * a.x_token + (head0 + h) * a.x_head;
    const int64_t to = (token0 + row) * a.y_token + (head0 + h) * a.y_head;
    if (u >= w.turned) {
      const int c = 2 * a.pairs + (u - w.turned) * V;
      if (!in_place) P::store(a.y, to + c, P::load(a.x, from + c));
      continue;
    }
    const float2 *cs = turn + row * a.pairs;
    if constexpr (INTERLEAVED) {
      const int c = u * V;
      float f[V], g[V];
      P::open(P::load(a.x, from + c), f);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 t = cs[(c + i) / 2];
        g[i] = __builtin_fmaf(f[i], t.x, -(f[i + 1] * t.y));
        g[i + 1] = __builtin_fmaf(f[i + 1], t.x, f[i] * t.y);
      }
      P::store(a.y, to + c, P::close(g));
    } else {
      const int c = u * V;
      float fa[V], fb[V], ga[V], gb[V];
      P::open(P::load(a.x, from + c), fa);
      P::open(P::load(a.x, from + a.pairs + c), fb);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 t = cs[c + i];
        ga[i] = __builtin_fmaf(fa[i], t.x, -(fb[i] * t.y));
        gb[i] = __builtin_fmaf(fb[i], t.x, fa[i] * t.y);
      }
      P::store(a.y, to + c, P::close(ga));
      P::store(a.y, to + a.pairs + c, P::close(gb));
    }
  }
}

uint32_t magic(int d) { return d == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + d - 1) / d); }

template <int DT, int V, bool INTERLEAVED>
void launch(const RotaryArgs &a, hipStream_t st) {
  Split w;
  w.turned = INTERLEAVED ? 2 * a.pairs / V : a.pairs / V;
  w.units = w.turned + (a.head_dim - 2 * a.pairs) / V;
  w.heads = a.heads;
  // (divide() needs items * divisor below 2^32)
  w.tokens = std::max(1, std::min(kThreads / a.pairs, 65536 / (w.heads * w.units)));
  w.by_units = magic(w.units);
  w.by_heads = magic(w.heads);
  const dim3 grid((unsigned)((a.tokens + w.tokens - 1) / w.tokens), (unsigned)((a.heads + w.heads - 1) / w.heads));
  hipLaunchKernelGGL((rotary_kernel<DT, V, INTERLEAVED>), grid, dim3(kThreads), 0, st, a, w);
}

template <int DT>
void launch_typed(const RotaryArgs &a, hipStream_t st) {
  constexpr int V = DT == kF32 ? 4 : 8;  // 16 bytes
  if (a.interleaved) {
    if (2 * a.pairs % V == 0) launch<DT, V, true>(a, st);
    else launch<DT, 2, true>(a, st);
  } else {
    if (a.pairs % V == 0) launch<DT, V, false>(a, st);
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
