// A line of work cut over a grid: prefix sums of costs, and the places where the parts begin.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sage {

namespace {  // internal linkage: each translation unit keeps its own copy

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// pre[b] = sum of cost(b') over b' < b, pre[B] = the total (all threads of the CTA, which must
// synchronise before they read it); wsum: one word for each warp
template <int NT, class Cost>
__device__ __forceinline__ void prefix_of(int B, long long* pre, long long* wsum, Cost&& cost) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = (B + NT - 1) / NT, b0 = min(B, tid * n), b1 = min(B, b0 + n);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    pre[b] = sum;
    sum += cost(b);
  }
  long long s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += x;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  long long base = s - sum;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  for (int b = b0; b < b1; ++b) pre[b] += base;
  if (tid == NT - 1) pre[B] = base + sum;
}
// the batch row that holds place `at` of the line
__device__ __forceinline__ int row_at(const long long* pre, int B, long long at) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= at) lo = mid;
    else hi = mid;
  }
  return lo;
}

// a b / c; the 32-bit division where it serves (a 64-bit one costs a microsecond of a part's start)
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
  const unsigned long long x = (unsigned long long)a * (unsigned)b;
  return (x | (unsigned long long)c) >> 32 ? (long long)(x / (unsigned long long)c) : (long long)((uint32_t)x / (uint32_t)c);
}
// The line of work, `total` places, cut into equal parts for the CTAs of a grid in order.
struct Line {
  long long total;
  int parts;
  // where part v begins
  __device__ long long start(int v) const { return mul_div(total, v, parts); }
  // the part that holds place x
  __device__ int holder(long long x) const {
    int v = (int)mul_div(x, parts, total);
    while (start(v + 1) <= x) ++v;
    while (start(v) > x) --v;
    return v;
  }
};

}  // namespace

}  // namespace sage
