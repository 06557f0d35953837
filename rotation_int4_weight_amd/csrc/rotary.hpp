// rotary.hpp - internal host launcher of the rotary position kernel.
// rotary_abi.cpp validates every argument before calling it; all pointers are
// device pointers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace paro {

struct RotaryArgs {
  const void *x;
  void *y;
  const int32_t *positions;
  const double *freqs;
  int64_t x_token, x_head, y_token, y_head;  // elements
  int64_t tokens;
  int heads, head_dim, pairs;  // pairs = rot_dim / 2
  int interleaved, inverse, dt;
  float magnitude;
};
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st);

}  // namespace paro
