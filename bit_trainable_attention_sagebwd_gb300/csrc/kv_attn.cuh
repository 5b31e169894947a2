// What the two attention kernels over the paged cache share: parameters, the line of work that
// is cut over the grid, and the codes' way into fp16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"
#include "line.cuh"
#include "ptx.cuh"

namespace sage {

struct AttnParams {
  sage_kv_cache c;
  const __nv_bfloat16* Q;
  const int *slots, *q_len;
  __nv_bfloat16* O;
  float* LSE;
  int2* info;      // first and last worker of each unit; not written where a wait ran out
  float* part;     // two partial results of each worker: [R][D] sums, then [R] maxima and [R] row sums
  int B, H, G, Nq, tiles, causal;
  int most_parts;  // CTAs of the grid: the parts of the line at most (the joins: those that the workspace holds)
  float alpha;     // sm_scale log2 e
};

namespace {  // internal linkage: each translation unit keeps its own copy

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 16 bytes from src, or zeros (src is then not read)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four codes of a word as fp16: bytes (0, 2) and bytes (1, 3), the pairing that takes the fewest
// instructions; who contracts over the channels or writes them out puts up with the order.
// int8: byte ^ 0x80 under the exponent 0x64 is the fp16 1024 + c + 128.  e4m3: sign, exponent and
// fraction moved to fp16's places give the value times 2^-8 (subnormal codes too), which kCodeUnit
// takes back; every byte is finite.
template <int KIND>
constexpr float kCodeUnit = KIND == SAGE_KV_INT8 ? 1.f : 256.f;

template <int KIND>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (KIND == SAGE_KV_INT8) {
    even = hsub2((w & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
    odd = hsub2(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u, 0x64806480u);
  } else {
    even = ((w << 7) & 0x3f803f80u) | ((w << 8) & 0x80008000u);
    odd = ((w >> 1) & 0x3f803f80u) | (w & 0x80008000u);
  }
}

// P and the V scales.  s_v of a page goes into the exponent: with t_j the logit of key j in powers of
// two and u_j = t_j + log2 s_v(j), P_j = 2^(u_j - m), m a running reference of the u that keeps the
// largest P of a row between 2^7 and 2^15, so fp16 holds P whatever the pages' scales are (11 bits
// down to 2^-21 of the largest, 2^-32 of it absolute below); the row sum takes P_j / s_v(j).  m moves
// only when a row's maximum passes 2^15, so accumulators are seldom rescaled.  A page of zeros
// (s_v = 0) takes the largest scale met so far (`ref`) instead; scales below 2^-80 (values below 2^-71)
// are read as 2^-80, so that the row sums stay in fp32's range.
constexpr float kRaise = 15.f, kBelow = 7.f;
__device__ __forceinline__ float value_scale(float vs, float ref) {
  constexpr float kLeast = 0x1p-80f;
  return vs > 0.f ? fmaxf(vs, kLeast) : ref > 0.f ? fmaxf(ref, kLeast) : 1.f;
}

// The power of two that brings a query row's largest element `top` to [2^8, 2^9), where fp16 holds
// every bf16 down to 2^-25 of it exactly, and its inverse.
__device__ __forceinline__ void row_power(float top, float& up, float& down) {
  const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -110), 126);
  up = __uint_as_float((uint32_t)(127 + 8 - ex) << 23);
  down = __uint_as_float((uint32_t)(127 - 8 + ex) << 23);
}

// The slot of batch row b and its length; what is out of range is reported and counts as empty.
__device__ __forceinline__ int row_length(const AttnParams& p, int b, int& slot) {
  slot = p.slots ? p.slots[b] : b;
  int len = 0;
  bool bad = (unsigned)slot >= (unsigned)p.c.n_slots;
  if (!bad) {
    len = p.c.lengths[slot];
    bad = len < 0 || (long long)len > (long long)p.c.max_pages * p.c.page;
  }
  if (bad) {
    atomicMax(p.c.status, kDevIndex);
    slot = 0, len = 0;
  }
  return len;
}
__device__ __forceinline__ int row_queries(const AttnParams& p, int b) {
  return p.q_len ? max(0, min(p.Nq, p.q_len[b])) : p.Nq;
}
// keys that query i of q_len sees
__device__ __forceinline__ int row_end(const AttnParams& p, int len, int q_len, int i) {
  return p.causal ? max(0, min(len, len - q_len + i + 1)) : len;
}

// Whether a unit's first and last part are such as a join may read: two at least, and in the workspace.  After a
// wait that ran out they are whatever the workspace held, and the unit's rows are left.
__device__ __forceinline__ bool was_cut(const AttnParams& p, int2 w) {
  return w.x >= 0 && w.x < w.y && w.y < p.most_parts;
}

// the most parts
constexpr int kMaxParts = 512;         // few query rows
constexpr int kMaxChunkParts = 160;    // many (one CTA an SM)
constexpr int kChunkRows = 256;        // query rows of a unit, many

}  // namespace

// the kernel of up to 16 query rows a unit (up to 32 of a shared head, in two units), and the one of kChunkRows
int launch_kv_few(const AttnParams& p, int kind, int rows, int sms, cudaStream_t st);
int launch_kv_chunk(const AttnParams& p, int kind, int sms, cudaStream_t st);

}  // namespace sage
