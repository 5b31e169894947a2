// Launcher of rotary positions (sage_attn_rotary of include/sage_attn.h).
#pragma once

#include <cuda_runtime.h>

#include "../../include/sage_attn.h"

namespace sage {

struct RotaryParams {
  sage_rotary r;
  sage_heads in[2], out[2];  // queries and keys
  int heads[2];              // (keys: 0, none)
  const int *positions, *start, *cu;
  int B, N, S;
  int inverse;
};

int launch_rotary(const RotaryParams& p, int D, cudaStream_t st);

}  // namespace sage
