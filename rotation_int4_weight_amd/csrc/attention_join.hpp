// attention_join.hpp - the end of a decode attention workgroup: its waves' sums
// are joined through LDS, and the parts of a row through the workspace by the
// last workgroup to arrive, in their order.  Shared by the kernels over the
// cache in 16 and in four bits.
#pragma once

#include <math.h>

#include <type_traits>

#include "attention.hpp"
#include "common.hpp"
#include "mfma.hpp"

namespace paro {

constexpr int kDecodeWaves = 4;  // of a decode workgroup
constexpr int kCoherent = 16;    // SC1: device-scope loads and stores of the parts
// Parts that a thread has in flight together.  Over 16 bits eight where it has more
// than kJoinFew, four otherwise; always four and always eight take, us: one row of
// 131072 keys with 16 heads on one key-value head 114 and 91 (by this rule 82), with
// 8 times 16 heads 108 and 105 (105), one of 8000 with 8 times 8 heads 17.1 and
// 15.6 (15.6), of 777 with 8 times 4 7.0 and 7.4 (7.1).  Over four bits always
// four: the code of both costs one row of 777 8.5 instead of 8.2 us, 40 rows of up
// to 1500 13.6 instead of 13.2, for 139 instead of 155 of one row of 131072 keys
// with 16 heads on one key-value head and 60.6 instead of 63 with 8 times 16.
// Sixteen in flight spill registers.
constexpr int kJoinBatch = 4, kJoinFew = 8;  // of a thread

// What the waves hand over: sums relative to 2^m, m the maximum of scores * log2 e.
template <int DIM>
struct DecodeJoin {
  static constexpr int RS = DIM + 4;  // the four words over keep rows on different banks
  __align__(16) float o[kDecodeWaves][16][RS];  // [wave][head][channel]
  float m[kDecodeWaves][16], l[kDecodeWaves][16];
  float jm[16], jl[16];
  int last;
};

__device__ __forceinline__ float max_over_groups(float x) {
  uint32_t u = __float_as_uint(x);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  u = __float_as_uint(x);
  auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_over_groups(float x) {
  uint32_t u = __float_as_uint(x);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  u = __float_as_uint(x);
  auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// (o, m, sum) joined with another part's, both relative to their maxima
__device__ __forceinline__ void add_part(f32x4 &o, float &m, float &sum, const f32x4 &po, float pm, float psum) {
  const float mn = fmaxf(m, pm), ref = mn == -INFINITY ? 0.f : mn;
  const float ka = __builtin_amdgcn_exp2f(m - ref), kb = __builtin_amdgcn_exp2f(pm - ref);
  o = o * ka + po * kb;
  sum = sum * ka + psum * kb;
  m = mn;
}

// four outputs in the type
template <int DT>
__device__ __forceinline__ u32x2 pack_row(const f32x4 &o, float inv) {
  constexpr bool F = DT == kF16;
  return u32x2{pack2<DT>(within_type<F>(o[0] * inv), within_type<F>(o[1] * inv)),
               pack2<DT>(within_type<F>(o[2] * inv), within_type<F>(o[3] * inv))};
}

// Where an output's parts lie in the workspace: part p in the place_of(p)-th
// slot of part_floats floats.
struct PartsInOrder {
  __device__ __forceinline__ int operator()(int p) const { return p; }
};
// floats of a part: per head DIM sums, maximum, sum, 2 unused
__host__ __device__ inline int part_floats(int group, int dim) { return (group < 16 ? group : 16) * (dim + 4); }

// Called by all threads once every wave has written its o, m and l (no barrier
// needed in between): part `part` of `parts` of the `heads` query heads from
// head0 of a row.  counter: this output's; rs: the slots (neither is used with
// one part).  some: the row has a key; without one it is zero.  MANY: outputs of
// many parts have more of them in flight.  Storing a part, counting and joining
// takes 2 to 3 us.
template <int DT, int DIM, bool MANY, class Place>
__device__ __forceinline__ void join_parts(const AttentionArgs &a, DecodeJoin<DIM> &lds, uint32_t *counter,
                                           __amdgpu_buffer_rsrc_t rs, Place place_of, int64_t row, int head0,
                                           int heads, int part, int parts, bool some) {
  constexpr int RS = DecodeJoin<DIM>::RS;
  __syncthreads();
  // thread: head t / (DIM / 4), four channels; heads in passes
  constexpr int kPerHead = DIM / 4, kHeadsPerPass = 256 / kPerHead;
  const int slot_floats = part_floats(a.group, DIM);
  const int ch = ((int)threadIdx.x % kPerHead) * 4;
  for (int h = (int)threadIdx.x / kPerHead; h < heads; h += kHeadsPerPass) {
    float m = lds.m[0][h];
#pragma unroll
    for (int w = 1; w < kDecodeWaves; ++w) m = fmaxf(m, lds.m[w][h]);
    const float ref = m == -INFINITY ? 0.f : m;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDecodeWaves; ++w) {
      const float k = __builtin_amdgcn_exp2f(lds.m[w][h] - ref);
      sum += k * lds.l[w][h];
      o += k * *reinterpret_cast<const f32x4 *>(&lds.o[w][h][ch]);
    }
    if (parts == 1) {
      const float inv = some ? 1.f / sum : 0.f;
      const u32x2 y = pack_row<DT>(o, inv);
      *reinterpret_cast<u32x2 *>(a.y + row * a.y_token + (int64_t)(head0 + h) * a.y_head + ch) =
          some ? y : u32x2{0, 0};
    } else {
      const uint32_t at = (uint32_t)(place_of(part) * slot_floats + h * (DIM + 4)) * 4u;
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), rs, at + ch * 4, 0, kCoherent);
      if (ch == 0) {
        const u32x2 ml = {__float_as_uint(m), __float_as_uint(sum)};
        __builtin_amdgcn_raw_buffer_store_b64(ml, rs, at + DIM * 4, 0, kCoherent);
      }
    }
  }
  if (parts == 1) return;
  // ---- join the parts: the last workgroup to arrive, in their order ----
  __builtin_amdgcn_s_waitcnt(0);  // this thread's part has been stored
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = old == (uint32_t)(parts - 1);
  }
  __syncthreads();
  if (!lds.last) return;
  // DIM / 4 threads per head leave room for `lanes` of them per output: each
  // takes every lanes-th part
  const int lanes = max(1, kHeadsPerPass / heads);
  const int sub = (int)threadIdx.x / kPerHead;
  float *const jo = &lds.o[0][0][0];  // [sub][RS], after the waves' use of o
  for (int h0 = 0; h0 < heads; h0 += kHeadsPerPass) {
    const int h = lanes > 1 ? sub / lanes : h0 + sub, first = lanes > 1 ? sub % lanes : 0;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    const auto gather = [&](auto batch) {
      constexpr int B = decltype(batch)::value;
      for (int p0 = first; p0 < parts; p0 += B * lanes) {
        f32x4 x[B];
        u32x2 ml[B];
#pragma unroll
        for (int u = 0; u < B; ++u) {
          const uint32_t at = (uint32_t)(place_of(min(p0 + u * lanes, parts - 1)) * slot_floats + h * (DIM + 4)) * 4u;
          x[u] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at + ch * 4, 0, kCoherent));
          ml[u] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, at + DIM * 4, 0, kCoherent));
        }
#pragma unroll
        for (int u = 0; u < B; ++u)
          if (p0 + u * lanes < parts) add_part(o, m, sum, x[u], __uint_as_float(ml[u][0]), __uint_as_float(ml[u][1]));
      }
    };
    if (h < heads) {
      if (MANY && parts > kJoinFew * lanes) gather(std::integral_constant<int, MANY ? 2 * kJoinBatch : kJoinBatch>());
      else gather(std::integral_constant<int, kJoinBatch>());
    }
    if (lanes > 1) {  // then heads <= kHeadsPerPass / 2: this loop runs once
      __syncthreads();
      if (h < heads) {
        *reinterpret_cast<f32x4 *>(jo + sub * RS + ch) = o;
        if (ch == 0) {
          lds.jm[sub] = m;
          lds.jl[sub] = sum;
        }
      }
      __syncthreads();
      if (first != 0) continue;
      for (int u = 1; u < lanes && h < heads; ++u)
        add_part(o, m, sum, *reinterpret_cast<const f32x4 *>(jo + (sub + u) * RS + ch), lds.jm[sub + u], lds.jl[sub + u]);
    }
    if (h >= heads) continue;
    const float inv = 1.f / sum;
    const u32x2 y = pack_row<DT>(o, inv);
    *reinterpret_cast<u32x2 *>(a.y + row * a.y_token + (int64_t)(head0 + h) * a.y_head + ch) = y;
  }
  if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace paro
