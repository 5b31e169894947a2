// Launchers of attention over packed sequences (the sage_attn_packed_* calls of include/sage_attn.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include "../../include/sage_attn.h"

namespace sage {

// Most sequences and tokens of one call, and most query heads of a key/value head (their rows share a tile).
constexpr int kPackedMaxSeqs = 65536;
constexpr int kPackedMaxTokens = 1 << 24;
constexpr int kPackedMaxGroup = 128;
// Least sm_scale of the backward, which divides LSE by it: the log of 2^24 keys over 2^-120 is still below 2^125.
constexpr float kPackedLeastScale = 0x1p-120f;

struct PackedWs {
  size_t part, stats, total;  // (the status word and the counters come first)
};
PackedWs packed_ws_layout(int T, int S, int H, int Hkv, int D, bool backward);

int launch_packed_fwd(const sage_rows& Q, const sage_rows& K, const sage_rows& V, const int* cu, const sage_rows& O,
                      float* LSE, void* ws, int T, int S, int H, int Hkv, int D, int causal, float sm_scale,
                      cudaStream_t st);
int launch_packed_bwd(const sage_rows& Q, const sage_rows& K, const sage_rows& V, const sage_rows& O, const float* LSE,
                      const sage_rows& dO, const int* cu, const sage_rows& dQ, const sage_rows& dK, const sage_rows& dV,
                      void* ws, int T, int S, int H, int Hkv, int D, int causal, float sm_scale, cudaStream_t st);

}  // namespace sage
