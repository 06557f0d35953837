// rotary_abi.cpp - C-ABI of the rotary positions: argument validation, the
// frequencies (on the host) and launch-error mapping.  The contract is in
// include/paro.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "abi.hpp"
#include "paro.h"
#include "rotary.hpp"

namespace {

using paro::aligned;
using paro::fail;
using paro::hip_fail;
using paro::ok;
using paro::overlap;
using paro::strided_overlap;

constexpr int64_t kMaxRows = int64_t(1) << 21;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kMaxHeads = 256, kMaxDim = 512;
constexpr double kTurn = 6.283185307179586476925;

int check_stride(int64_t s, const char *what) {
  if (s < 0 || s >= kMaxStride || s % 8)
    return fail(PARO_ERR_SHAPE, "%s=%lld must be a multiple of 8 elements in 0..2^40", what, (long long)s);
  return PARO_OK;
}

size_t extent(const paro_rotary_shape *s, int64_t tokens, int64_t token, int64_t head, size_t size) {
  return (size_t)((tokens - 1) * token + (s->heads - 1) * head + s->head_dim) * size;
}

// y's rows and heads lie apart from each other.
bool apart(const paro_rotary_shape *s, int64_t rows) {
  const int64_t d = s->head_dim, t = s->y_token, h = s->y_head;
  return ((s->heads == 1 || h >= d) && (rows <= 1 || t >= (s->heads - 1) * h + d)) ||
         ((rows <= 1 || t >= d) && (s->heads == 1 || h >= (rows - 1) * t + d));
}

}  // namespace

extern "C" {

int paro_rotary(const paro_rotary_shape *s, const void *x, paro_dtype dt, const int32_t *positions,
                const double *freqs, int64_t tokens, void *y, void *stream) {
  if (!s) return fail(PARO_ERR_NULL, "shape is NULL");
  if (s->heads < 1 || s->heads > kMaxHeads)
    return fail(PARO_ERR_SHAPE, "heads=%d must be in 1..%d", s->heads, kMaxHeads);
  if (s->head_dim < 8 || s->head_dim > kMaxDim || s->head_dim % 8)
    return fail(PARO_ERR_UNSUPPORTED, "head_dim=%d must be a multiple of 8 in 8..%d", s->head_dim, kMaxDim);
  if (s->rot_dim < 2 || s->rot_dim > s->head_dim || s->rot_dim % 2)
    return fail(PARO_ERR_SHAPE, "rot_dim=%d must be even and in 2..head_dim=%d", s->rot_dim, s->head_dim);
  if (!std::isfinite(s->magnitude)) return fail(PARO_ERR_SHAPE, "magnitude must be finite");
  if (tokens < 0) return fail(PARO_ERR_SHAPE, "tokens=%lld is negative", (long long)tokens);
  if (tokens > kMaxRows)
    return fail(PARO_ERR_UNSUPPORTED, "tokens=%lld exceeds %lld", (long long)tokens, (long long)kMaxRows);
  if (dt != PARO_F16 && dt != PARO_BF16 && dt != PARO_F32)
    return fail(PARO_ERR_DTYPE, "dtype %d must be F16, BF16 or F32", (int)dt);
  int rc;
  if ((rc = check_stride(s->x_token, "x_token")) || (rc = check_stride(s->x_head, "x_head")) ||
      (rc = check_stride(s->y_token, "y_token")) || (rc = check_stride(s->y_head, "y_head")))
    return rc;
  if (tokens == 0) return ok();
  if (!apart(s, tokens))
    return fail(PARO_ERR_SHAPE, "y strides (token %lld, head %lld) make rows or heads overlap", (long long)s->y_token,
                (long long)s->y_head);
  if (!x || !y || !positions || !freqs) return fail(PARO_ERR_NULL, "x, y, positions and freqs are required");
  if (!aligned(x, 16) || !aligned(y, 16)) return fail(PARO_ERR_ALIGN, "x and y must be 16-byte aligned");
  if (!aligned(positions, 4) || !aligned(freqs, 8))
    return fail(PARO_ERR_ALIGN, "positions must be 4-byte aligned, freqs 8-byte aligned");
  const size_t size = dt == PARO_F32 ? 4 : 2;
  const size_t xb = extent(s, tokens, s->x_token, s->x_head, size), yb = extent(s, tokens, s->y_token, s->y_head, size);
  const bool alike = (tokens == 1 || s->x_token == s->y_token) && (s->heads == 1 || s->x_head == s->y_head);
  if (!(alike && x == y) && overlap(x, xb, y, yb) &&
      !(alike && !strided_overlap(x, y, tokens, s->heads, s->head_dim * size, s->y_token * size, s->y_head * size)))
    return fail(PARO_ERR_SHAPE, "y overlaps x: only the same tensor, or views apart of one, with the same strides");
  if (overlap(y, yb, positions, (size_t)tokens * 4) || overlap(y, yb, freqs, (size_t)s->rot_dim * 4))
    return fail(PARO_ERR_SHAPE, "y overlaps positions or freqs");
  paro::RotaryArgs a = {};
  a.x = x;
  a.y = y;
  a.positions = positions;
  a.freqs = freqs;
  a.x_token = s->x_token;
  a.x_head = s->x_head;
  a.y_token = s->y_token;
  a.y_head = s->y_head;
  a.tokens = tokens;
  a.heads = s->heads;
  a.head_dim = s->head_dim;
  a.pairs = s->rot_dim / 2;
  a.interleaved = s->interleaved != 0;
  a.inverse = s->inverse != 0;
  a.dt = (int)dt;
  a.magnitude = s->magnitude;
  const hipError_t e = paro::launch_rotary(a, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "rotary launch");
  return ok();
}

int paro_rotary_frequencies(const paro_rotary_scaling *s, int rot_dim, double *freqs, float *magnitude) {
  if (!s || !freqs) return fail(PARO_ERR_NULL, "scaling and freqs are required");
  if (s->kind < PARO_ROTARY_NONE || s->kind > PARO_ROTARY_RAMP)
    return fail(PARO_ERR_UNSUPPORTED, "kind=%d is not a paro_rotary_kind", s->kind);
  if (rot_dim < 2 || rot_dim > kMaxDim || rot_dim % 2 || (s->kind == PARO_ROTARY_BASE && rot_dim < 4))
    return fail(PARO_ERR_SHAPE, "rot_dim=%d must be even and in 2..%d (from 4 with a scaled base)", rot_dim, kMaxDim);
  if (!(s->base > 1) || !std::isfinite(s->base)) return fail(PARO_ERR_SHAPE, "base must be over 1 and finite");
  const bool scaled = s->kind != PARO_ROTARY_NONE, ends = s->kind == PARO_ROTARY_BANDS || s->kind == PARO_ROTARY_RAMP;
  if (scaled && (!(s->factor >= 1) || !std::isfinite(s->factor)))
    return fail(PARO_ERR_SHAPE, "factor must be at least 1 and finite");
  if (ends && (!(s->context > 0) || !std::isfinite(s->context) || !(s->low > 0) || !(s->high > s->low) ||
               !std::isfinite(s->high)))
    return fail(PARO_ERR_SHAPE, "context must be over 0 and 0 < low < high, all finite");
  const int n = rot_dim / 2;
  // the pair that makes `turns` turns over the context, as a real number
  const auto index = [&](double turns) {
    return rot_dim * std::log(s->context / (turns * kTurn)) / (2 * std::log(s->base));
  };
  double first = 0, last = 0;
  if (s->kind == PARO_ROTARY_RAMP) {
    first = std::max(std::floor(index(s->high)), 0.0);
    last = std::min(std::ceil(index(s->low)), rot_dim - 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(s->base, -2.0 * i / rot_dim);
    if (s->kind == PARO_ROTARY_BASE) {
      // (base * factor^(rot_dim / (rot_dim - 2)))^(-2i / rot_dim), whose base may be no 64-bit number
      f *= std::pow(s->factor, -2.0 * i / (rot_dim - 2));
    } else if (s->kind == PARO_ROTARY_LINEAR) {
      f /= s->factor;
    } else if (ends) {
      // kept: 1 as it is, 0 divided by factor
      const double kept = s->kind == PARO_ROTARY_BANDS ? (s->context * f / kTurn - s->low) / (s->high - s->low)
                                                       : 1 - (i - first) / std::max(last - first, 0.001);
      const double k = std::min(1.0, std::max(0.0, kept));
      f = f * k + f / s->factor * (1 - k);
    }
    freqs[i] = f;
  }
  if (magnitude) *magnitude = s->kind == PARO_ROTARY_RAMP ? (float)(0.1 * std::log(s->factor) + 1.0) : 1.f;
  return ok();
}

}  // extern "C"
