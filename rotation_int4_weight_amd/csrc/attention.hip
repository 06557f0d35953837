// attention.hip - attention over packed prompts and over the paged cache
// (paro_attention_prompt, _prompt_cached, _decode).
//
// One wave per (row, head).  Keys in steps of 64: lane j holds key j's score,
// the running maximum and sum join the steps (a step's weights are
// exp(s - m) with the new maximum m, and what was summed before is scaled by
// exp(m_old - m)), and the output's channels lie over the lanes.
#include <math.h>

#include "attention.hpp"
#include "common.hpp"

namespace paro {
namespace {

template <int DT, int DIM, bool CACHED>
__global__ void __launch_bounds__(256) row_attention_kernel(AttentionArgs a) {
  __shared__ float qs[4][DIM];
  const int lane = lane_id(), wave = wave_id();
  const int64_t item = (int64_t)blockIdx.x * 4 + wave;
  const int64_t row = item / a.q_heads;
  const int head = (int)(item % a.q_heads), kvh = head / a.group;
  if (row >= a.q_tokens) return;
  int s = (int)row;
  int64_t q0 = row, q1 = row + 1;
  if (a.cu_q) {
    s = -1;
    for (int j = 0; j < a.sequences; ++j) {
      q0 = a.cu_q[j] < 0 ? 0 : a.cu_q[j];
      q1 = a.cu_q[j + 1] > a.q_tokens ? a.q_tokens : a.cu_q[j + 1];
      if (row >= q0 && row < q1) {
        s = j;
        break;
      }
    }
    if (s < 0) return;
  }
  int64_t k0 = 0, keys = 0;
  const int32_t *table = nullptr;
  if constexpr (CACHED) {
    const int slot = a.slots[s];
    if (slot >= 0 && slot < a.kv.slots) {
      const int most = a.kv.max_pages << a.kv.page_shift, len = a.kv.lengths[slot];
      keys = len < 0 ? 0 : len > most ? most : len;
      table = a.kv.table + (int64_t)slot * a.kv.max_pages;
    }
  } else {
    k0 = a.cu_k[s] < 0 ? 0 : a.cu_k[s];
    const int64_t k1 = a.cu_k[s + 1] > a.k_tokens ? a.k_tokens : a.cu_k[s + 1];
    keys = k1 > k0 ? k1 - k0 : 0;
  }
  int64_t seen = keys;  // keys this row may see
  if (a.causal) seen = min(keys, row - q0 + 1 + keys - (q1 - q0));

  auto row_of = [&](const uint16_t *packed, const uint16_t *paged, int64_t token, int64_t hs, int64_t j) {
    if constexpr (CACHED) {
      int page = table[j >> a.kv.page_shift];
      page = page < 0 ? 0 : page >= a.kv.num_pages ? a.kv.num_pages - 1 : page;
      return paged + (int64_t)page * a.kv.page_stride + ((int64_t)kvh << a.kv.page_shift) * DIM +
             (j & ((1 << a.kv.page_shift) - 1)) * DIM;
    } else {
      return packed + (k0 + j) * token + kvh * hs;
    }
  };
  const uint16_t *q = a.q + row * a.q_token + head * a.q_head;
  for (int d = lane; d < DIM; d += 64) qs[wave][d] = act_to_f32<DT>(q[d]) * a.scale;
  wave_lds_sync();
  float m = -INFINITY, l = 0.f, acc[DIM / 64] = {};
  for (int64_t j0 = 0; j0 < seen; j0 += 64) {
    const int64_t j = j0 + lane;
    float sc = -INFINITY;
    if (j < seen) {
      const uint16_t *k = row_of(a.k, a.kv.k, a.k_token, a.k_head, j);
      sc = 0.f;
      for (int d = 0; d < DIM; ++d) sc = fmaf(qs[wave][d], act_to_f32<DT>(k[d]), sc);
    }
    float top = sc;
    for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float mn = fmaxf(m, top);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float p = act_to_f32<DT>(pack2<DT>(j < seen ? expf(sc - ref) : 0.f, 0.f) & 0xffffu);
    const float keep = expf(m - ref);
    l = l * keep + p;  // lane j sums its own keys
    m = mn;
    for (int c = 0; c < DIM / 64; ++c) acc[c] *= keep;
    const int n = (int)min((int64_t)64, seen - j0);
    for (int jj = 0; jj < n; ++jj) {
      const float w = __shfl(p, jj, 64);
      const uint16_t *v = row_of(a.v, a.kv.v, a.v_token, a.v_head, j0 + jj);
      for (int c = 0; c < DIM / 64; ++c) acc[c] = fmaf(w, act_to_f32<DT>(v[c * 64 + lane]), acc[c]);
    }
  }
  for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, 64);
  uint16_t *y = a.y + row * a.y_token + head * a.y_head;
  for (int c = 0; c < DIM / 64; ++c)
    y[c * 64 + lane] = (uint16_t)(pack2<DT>(seen > 0 ? acc[c] / l : 0.f, 0.f) & 0xffffu);
}

template <bool CACHED>
hipError_t launch_rows(const AttentionArgs &a, hipStream_t st) {
  const int64_t items = a.q_tokens * a.q_heads;
  const dim3 grid((unsigned)((items + 3) / 4));
#define PARO_ROWS(DT, DIM) hipLaunchKernelGGL((row_attention_kernel<DT, DIM, CACHED>), grid, dim3(256), 0, st, a)
  if (a.dt == kF16) {
    if (a.head_dim == 64) PARO_ROWS(kF16, 64);
    else PARO_ROWS(kF16, 128);
  } else {
    if (a.head_dim == 64) PARO_ROWS(kBF16, 64);
    else PARO_ROWS(kBF16, 128);
  }
#undef PARO_ROWS
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_prompt(const AttentionArgs &a, bool cached, hipStream_t st) {
  return cached ? launch_rows<true>(a, st) : launch_rows<false>(a, st);
}

}  // namespace paro
