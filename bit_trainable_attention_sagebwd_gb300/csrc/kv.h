// Launchers and shared device code of the 8-bit paged key/value cache (the sage_attn_kv_*
// calls of include/sage_attn.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sage_attn.h"

namespace sage {

// device status codes of the cache calls (beside those of ptx.cuh); the largest one is kept
enum : int { kDevPages = 6, kDevIndex = 7 };

// Most slots of a cache, and most batch rows of one attention call: the kernels keep one number
// for each in shared memory.
constexpr int kKvMaxSlots = 8192;
constexpr int kKvMaxBatch = 4096;

struct KvAttnWs {
  size_t info, part, total;
  int rows;    // query rows of a unit
  int tiles;   // units of one (batch row, key/value head)
};
KvAttnWs kv_attn_ws_layout(int B, int H, int Hkv, int D, int Nq);
size_t kv_compact_ws_bytes(int n_pages);

int launch_kv_append(const sage_kv_cache& c, const void* K, const void* V, const float* k_shift, const int* slots,
                     const int* pos, const int* n_new, int B, int Nn, cudaStream_t st);
int launch_kv_attention(const sage_kv_cache& c, const void* Q, const int* slots, const int* q_len, void* O,
                        float* LSE, void* ws, int B, int H, int Nq, int causal, float sm_scale, cudaStream_t st);
// the join of an attention call alone (sage_attn_selftest_kv_join)
int launch_kv_join(const sage_kv_cache& c, void* O, float* LSE, void* ws, int B, int H, int Nq, cudaStream_t st);
int launch_kv_fork(const sage_kv_cache& c, const int* src, cudaStream_t st);
int launch_kv_extend(const sage_kv_cache& c, const int* n_new, int* pos, int* cow, cudaStream_t st);
int launch_kv_truncate(const sage_kv_cache& c, const int* keep, cudaStream_t st);
int launch_kv_compact(const sage_kv_cache& c, const sage_kv_cache& to, void* ws, cudaStream_t st);

}  // namespace sage
