// The 8-bit paged key/value cache: the quantizing write and the bookkeeping of its pages
// (sage_attn_kv_append, _fork, _extend, _truncate, _compact in include/sage_attn.h).
//
// Every decision that numbers depend on (which page is taken, who copies a shared page, where a
// live page goes) follows the order of slots and pages, never the order in which threads arrive:
// the same state and arguments give the same tables.  The only atomics are integer additions
// into `refs` and the maximum of the status word, whose results do not depend on their order.
//
// All of it is bound by memory or, in small calls, by the launches.  Measured: kv_append of two prompts of
// 20k to 32k tokens (8 heads, D = 128, e4m3, 0.32 GB) 52 us, 6.2 TB/s, 92 % of the rate of a plain
// copy; of one token for each of 64 sequences 6.3 us from Python, a launch and its three dependent loads.  fork, extend
// and truncate of 32 prompts into 256 sequences (67 MB of copied pages) 20 us, of which extend's one CTA
// and the copies are 8 us and 9 us.  kv_compact of 2.7 GB of reads and writes 415 us, 6.5 TB/s, 95 %.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kv.h"
#include "launch.h"
#include "ptx.cuh"
#include "timer.h"

namespace sage {

namespace {

__device__ __forceinline__ void kv_error(int* status, int code) { atomicMax(status, code); }

// ------------------------------------------------------------------------------ append

// Threads of a page and head: 64 values each, at 64 registers (1024 threads an SM with 128 KB of new
// tokens on their way), a warp at least.  A CTA is a page's threads, two pages' where they are a warp: with
// a CTA of two warps for a 16-token page two prompts of 20k-32k tokens took 70 us, so 54 us; two
// pages of two warps each (32 tokens of D = 128) take 65 us against 54 us, whatever barrier joins them.
__host__ __device__ constexpr int append_threads(int D, int P) { return D * P / 64 < 32 ? 32 : D * P / 64; }
__host__ __device__ constexpr int append_pages(int D, int P) { return append_threads(D, P) < 64 ? 2 : 1; }

// What a block's scale s brings to its codes.  RN(x / s) by Markstein's correction (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990): inv = RN(1 / s),
// q = RN(x inv), r = x - q s (exact), RN(q + r inv) is the rounded quotient unless s's fraction is all
// ones; r is exact for every x that matters (|x / s| >= 2^-10, below it the code is 0) where
// s >= 2^-110.  Other scales divide.  With z = -x for x and -r for r a zero keeps its sign: q is RN(z ninv)
// and the quotient RN(q + (q s + z) ninv), ninv = -inv.
struct Quant {
  float s;
  bool fast;
  uint64_t ninv2, s2;
};
__device__ __forceinline__ Quant quant_of(float s) {
  Quant q;
  q.s = s;
  q.fast = s >= 0x1p-110f && s <= 0x1p110f && (__float_as_uint(s) & 0x7fffffu) != 0x7fffffu;
  const float inv = q.fast ? __frcp_rn(s) : 0.f;
  q.ninv2 = f2(-inv, -inv), q.s2 = f2(s, s);
  return q;
}
// Codes of four values x = -z: the int8 code is the low byte of RN(x / s) + 1.5 2^23.  Of a FAST scale |x / s| is at
// most 127 (1 + 2^-22): nothing to saturate.  A subnormal scale is rounded to so few bits (fp32 keys less a shift
// reach them) that the quotient may be half as much again.
template <int KIND, bool FAST>
__device__ __forceinline__ uint32_t codes4(float z0, float z1, float z2, float z3, const Quant& q) {
  float y[4];
  if (FAST) {
    const uint64_t a = f2(z0, z1), b = f2(z2, z3);
    const uint64_t qa = fmul2(a, q.ninv2), qb = fmul2(b, q.ninv2);
    f2split(ffma2(ffma2(qa, q.s2, a), q.ninv2, qa), y[0], y[1]);
    f2split(ffma2(ffma2(qb, q.s2, b), q.ninv2, qb), y[2], y[3]);
  } else if (q.s > 0.f) {
    y[0] = __fdiv_rn(-z0, q.s), y[1] = __fdiv_rn(-z1, q.s), y[2] = __fdiv_rn(-z2, q.s), y[3] = __fdiv_rn(-z3, q.s);
    if (KIND == SAGE_KV_INT8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fminf(fmaxf(y[i], -127.f), 127.f);
    }
  } else {
    return 0u;
  }
  if (KIND == SAGE_KV_INT8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
template <int KIND, bool FAST>
__device__ __forceinline__ uint2 codes8(const float (&z)[8], const Quant& q) {
  return make_uint2(codes4<KIND, FAST>(z[0], z[1], z[2], z[3], q), codes4<KIND, FAST>(z[4], z[5], z[6], z[7], q));
}
// the negated values of eight codes
template <int KIND>
__device__ __forceinline__ void negated8(uint2 c, float s, float (&z)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xffu;
    const float v = KIND == SAGE_KV_INT8 ? (float)(int)(int8_t)b
                                         : __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
    z[i] = -__fmul_rn(v, s);
  }
}

struct AppendParams {
  sage_kv_cache c;
  const __nv_bfloat16 *K, *V;
  const float* shift;
  const int *slots, *pos, *n_new;
  int B, Nn;
};

// One group of threads per (page that the new tokens of a batch row can touch, key/value head, K or V).  A
// thread holds its eight channels of up to eight tokens in registers between the maximum and the
// codes, so the new tokens are read once.  SHIFT: k_shift is given.
template <int D, int P, int KIND, bool SHIFT>
__global__ void __launch_bounds__(append_threads(D, P) * append_pages(D, P), 1024 / (append_threads(D, P) * append_pages(D, P)))
    kv_append_kernel(const AppendParams p) {
  constexpr int kThreads = append_threads(D, P), kPages = append_pages(D, P);
  constexpr int TPR = D / 8, RPP = kThreads / TPR, NP = P / RPP;  // threads a token, tokens a pass, passes
  static_assert(P % RPP == 0, "a page is a whole number of passes");
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, hk = blockIdx.y >> 1, group = threadIdx.x / kThreads, tid = threadIdx.x % kThreads;
  const bool is_v = blockIdx.y & 1;
  const int slot = p.slots ? p.slots[b] : b;
  if ((unsigned)slot >= (unsigned)p.c.n_slots) {
    if (threadIdx.x == 0) kv_error(p.c.status, kDevIndex);
    return;
  }
  const int pos = p.pos[slot], n = p.n_new[slot], len = p.c.lengths[slot];
  if (pos < 0 || n <= 0) return;  // nothing new, or refused by sage_attn_kv_extend
  const int j = pos / P + blockIdx.x * kPages + group;
  const long long t0 = (long long)j * P;
  // the new tokens are on their way while the table is read
  const int off = (int)max(0ll, pos - t0);       // tokens of the page that are there already
  const int end = (int)max(0ll, min((long long)P, pos - t0 + n));  // 0: the page is behind them
  // token 0 of the page is token t0 - pos of the new ones
  const __nv_bfloat16* src =
      (is_v ? p.V : p.K) + (((size_t)b * p.c.Hkv + hk) * p.Nn) * D + (t0 - pos) * D;
  const int g = tid % TPR, r0 = tid / TPR;
  uint4 u[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = r0 + i * RPP;
    if (r >= off && r < end && n <= p.Nn) u[i] = reinterpret_cast<const uint4*>(src + (size_t)r * D)[g];
  }
  // a batch row that names a slot again is left out
  if (p.slots) {
    bool again = false;
    for (int i = threadIdx.x; i < b; i += kThreads * kPages) again |= p.slots[i] == slot;
    if (__syncthreads_or(again)) {
      if (threadIdx.x == 0) kv_error(p.c.status, kDevIndex);
      return;
    }
  }
  if (end == 0) return;
  const int page = n <= p.Nn && j < p.c.max_pages ? p.c.table[(size_t)slot * p.c.max_pages + j] : -1;
  // Tokens past the slot's length, a page that is not there, or that another slot lists too: not written.  Behind the
  // length the table says nothing: what it lists there may be another slot's page.
  const bool room = n <= len && pos <= len - n;
  if (!room || (unsigned)page >= (unsigned)p.c.n_pages || p.c.refs[page] != 1) {
    if (tid == 0) kv_error(p.c.status, kDevIndex);
    return;
  }
  const size_t block = (size_t)page * p.c.Hkv + hk;
  float* scale = (is_v ? p.c.v_scale : p.c.k_scale) + block;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + block * P * D;
  const float was = off > 0 ? *scale : 0.f;
  const bool shifted = SHIFT && !is_v;
  float sh[8] = {};
  if (shifted) {
    const float4* s4 = reinterpret_cast<const float4*>(p.shift + hk * D + g * 8);
    const float4 a = s4[0], c = s4[1];
    sh[0] = a.x, sh[1] = a.y, sh[2] = a.z, sh[3] = a.w, sh[4] = c.x, sh[5] = c.y, sh[6] = c.z, sh[7] = c.w;
  }
  auto negated = [&](const uint4& w, float (&z)[8]) {
    const uint32_t flip = shifted ? 0u : 0x80008000u;
    const uint32_t v[4] = {w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip};
#pragma unroll
    for (int e = 0; e < 4; ++e) z[2 * e] = __uint_as_float(v[e] << 16), z[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    if (shifted) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = -__fsub_rn(z[e], sh[e]);
    }
  };
  float top = 0.f;
  if (shifted) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = r0 + i * RPP;
      if (r >= off && r < end) {
        float z[8];
        negated(u[i], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(z[e]));
      }
    }
  } else {  // two values at a time
    __nv_bfloat162 top2 = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = r0 + i * RPP;
      if (r >= off && r < end) {
        const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&u[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) top2 = __hmax2(top2, __habs2(x[e]));
      }
    }
    top = fmaxf(__low2float(top2), __high2float(top2));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (kThreads > 32) {
    static_assert(kThreads == 32 || kPages == 1, "a page's threads are a warp or the CTA");
    __shared__ float wtop[kThreads / 32];
    if ((tid & 31) == 0) wtop[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, wtop[i]);
  }
  const float fresh = __fmul_rn(top, KIND == SAGE_KV_INT8 ? 1.f / 127.f : 1.f / 448.f);
  const float now = fmaxf(was, fresh);
  const Quant q = quant_of(now);
  uint2* dst = reinterpret_cast<uint2*>(codes) + g;  // of token 0; a token is TPR of them
  float z[8];
  if (q.fast) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = r0 + i * RPP;
      if (r >= off && r < end) {
        negated(u[i], z);
        dst[r * TPR] = codes8<KIND, true>(z, q);
      }
    }
  } else {  // (kept apart and short: the instructions of a page's one pass are fetched, not found)
#pragma unroll 1
    for (int r = r0; r < end; r += RPP) {
      if (r < off) continue;
      negated(reinterpret_cast<const uint4*>(src + (ptrdiff_t)r * D)[g], z);
      dst[r * TPR] = codes8<KIND, false>(z, q);
    }
  }
  if (now != was) {  // the page's scale grew: what the old codes stand for, under the new one
#pragma unroll 1
    for (int r = r0; r < off; r += RPP) {
      negated8<KIND>(dst[r * TPR], was, z);
      dst[r * TPR] = q.fast ? codes8<KIND, true>(z, q) : codes8<KIND, false>(z, q);
    }
  }
  if (tid == 0) *scale = now;
}

template <int D, int P>
auto append_kernel_for(int kind, bool shift) {
  return kind == SAGE_KV_INT8
             ? (shift ? kv_append_kernel<D, P, SAGE_KV_INT8, true> : kv_append_kernel<D, P, SAGE_KV_INT8, false>)
             : (shift ? kv_append_kernel<D, P, SAGE_KV_E4M3, true> : kv_append_kernel<D, P, SAGE_KV_E4M3, false>);
}
template <int D>
auto append_kernel_for(int page, int kind, bool shift) {
  return page == 16   ? append_kernel_for<D, 16>(kind, shift)
         : page == 32 ? append_kernel_for<D, 32>(kind, shift)
         : page == 64 ? append_kernel_for<D, 64>(kind, shift)
                      : append_kernel_for<D, 128>(kind, shift);
}

// ------------------------------------------------------------------------------ pages

constexpr int kScanThreads = 1024;

// sum of v over the threads before this one, and over all (whole CTA of kScanThreads)
template <class T>
__device__ __forceinline__ T block_exclusive(T v, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  T x = warp_sums[lane];  // (every warp for itself: one barrier less)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  *total = __shfl_sync(0xffffffffu, x, 31);
  const T before = __shfl_sync(0xffffffffu, x, w ? w - 1 : 0);
  return s - v + (w ? before : 0);
}

// One CTA per slot that takes over another slot's pages.
__global__ void __launch_bounds__(256) kv_fork_kernel(const sage_kv_cache c, const int* __restrict__ src) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, from = src[s];
  if (from < 0) return;
  // only an empty slot takes over, and from a slot that does not take over itself
  const int n = from < c.n_slots ? c.lengths[from] : -1;
  const bool ok = from < c.n_slots && src[from] < 0 && c.lengths[s] == 0 && n >= 0 &&
                  (long long)n <= (long long)c.max_pages * c.page;
  if (!ok) {
    if (threadIdx.x == 0) kv_error(c.status, kDevIndex);
    return;
  }
  const int np = (n + c.page - 1) / c.page;
  const int* row = c.table + (size_t)from * c.max_pages;
  int* to = c.table + (size_t)s * c.max_pages;
  for (int j = threadIdx.x; j < np; j += blockDim.x) {
    const int page = row[j];
    to[j] = page;
    if ((unsigned)page < (unsigned)c.n_pages)
      atomicAdd(c.refs + page, 1);
    else
      kv_error(c.status, kDevIndex);
  }
  __syncthreads();  // every thread has read this slot's length
  if (threadIdx.x == 0) c.lengths[s] = n;
}

__global__ void __launch_bounds__(128) kv_truncate_kernel(const sage_kv_cache c, const int* __restrict__ keep) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, want = keep[s];
  if (want < 0) return;
  const int len = c.lengths[s];
  const long long cap = (long long)c.max_pages * c.page;
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) kv_error(c.status, kDevIndex);
    return;
  }
  const int now = min(want, len);
  const int* row = c.table + (size_t)s * c.max_pages;
  for (int j = (int)(((long long)now + c.page - 1) / c.page) + threadIdx.x; (long long)j * c.page < len; j += blockDim.x) {
    const int page = row[j];
    if ((unsigned)page < (unsigned)c.n_pages)
      atomicSub(c.refs + page, 1);
    else
      kv_error(c.status, kDevIndex);
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) c.lengths[s] = now;
}

// What a slot needs: `have` pages now, `want` after, one more if its last page is shared and
// partly filled (it is copied first; `last` is that page, else -1).
struct Need {
  int len, n, have, want, last;
  bool bad;
  __device__ int count() const { return want - have + (last >= 0); }
};
__device__ __forceinline__ Need slot_need(const sage_kv_cache& c, const int* n_new, int s) {
  Need q;
  q.len = c.lengths[s];
  q.n = n_new[s];
  q.last = -1;
  const long long cap = (long long)c.max_pages * c.page, end = (long long)q.len + q.n;
  q.bad = q.len < 0 || q.n < 0 || end > cap;
  q.have = q.bad ? 0 : (q.len + c.page - 1) / c.page;
  q.want = q.bad ? 0 : (int)((end + c.page - 1) / c.page);
  if (!q.bad && q.n > 0 && q.len % c.page) {
    const int page = c.table[(size_t)s * c.max_pages + q.have - 1];
    if ((unsigned)page >= (unsigned)c.n_pages)
      q.bad = true, q.have = q.want = 0;
    else if (c.refs[page] > 1)
      q.last = page;
  }
  return q;
}

// One CTA: the slots' needs are summed in slot order, then refs is scanned for free pages and
// the r-th free page goes to the slot whose range of needs holds r.  Shared memory keeps the sums
// (so finding the slot is a binary search) and the place in its table where a slot's pages begin.
__global__ void __launch_bounds__(kScanThreads) kv_extend_kernel(const sage_kv_cache c, const int* __restrict__ n_new,
                                                                 int* __restrict__ pos, int* __restrict__ cow) {
  extern __shared__ int excl[];        // [n_slots + 1]
  int* first_page = excl + c.n_slots + 1;  // [n_slots]; -1: refused
  __shared__ int warp_sums[32];
  __shared__ long long need_sums[32];
  constexpr int kPer = 16;  // pages a thread looks at in one step
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  // refs of the thread's pages of a step, on their way a step ahead (a step changes only its own pages)
  int4 ahead[kPer / 4];
  auto fetch = [&](int p0) {
    const long long first = (long long)p0 + tid * kPer;
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const long long at = first + 4 * i;
      ahead[i] = make_int4(1, 1, 1, 1);
      if (at + 4 <= c.n_pages) {
        ahead[i] = *reinterpret_cast<const int4*>(c.refs + at);
      } else {
        if (at < c.n_pages) ahead[i].x = c.refs[at];
        if (at + 1 < c.n_pages) ahead[i].y = c.refs[at + 1];
        if (at + 2 < c.n_pages) ahead[i].z = c.refs[at + 2];
      }
    }
  };
  fetch(0);
  int carry = 0;
  int len0 = 0, n0 = 0, from0 = -1;  // of slot tid
  for (int s0 = 0; s0 < c.n_slots; s0 += kScanThreads) {
    const int s = s0 + tid;
    int need = 0;
    if (s < c.n_slots) {
      const Need q = slot_need(c, n_new, s);
      need = q.count();
      if (s0 == 0) len0 = q.len, n0 = q.n, from0 = q.last;
      cow[s] = q.last;
      first_page[s] = q.bad ? -1 : q.have - (q.last >= 0);
      if (q.bad) kv_error(c.status, kDevIndex);
    }
    long long total;
    const long long e = block_exclusive((long long)need, need_sums, &total);
    // a pool has at most 2^28 pages: past 2^30 in all nothing can be served any more
    const int at = (int)min(carry + e, 1ll << 30);
    if (s < c.n_slots) excl[s] = at;
    carry = (int)min(carry + total, 1ll << 30);
  }
  if (tid == 0) excl[c.n_slots] = carry;
  __syncthreads();
  int found = 0;
  for (int p0 = 0; p0 < c.n_pages && found < carry; p0 += kScanThreads * kPer) {
    const int first = p0 + tid * kPer;
    unsigned free = 0;
#pragma unroll
    for (int i = 0; i < kPer / 4; ++i) {
      const int4 r = ahead[i];
      free |= (unsigned)(r.x == 0) << (4 * i) | (unsigned)(r.y == 0) << (4 * i + 1) |
              (unsigned)(r.z == 0) << (4 * i + 2) | (unsigned)(r.w == 0) << (4 * i + 3);
    }
    fetch(p0 + kScanThreads * kPer);
    int total;
    int r = found + block_exclusive(__popc(free), warp_sums, &total);
    int lo = 0;
    for (; free && r < carry; free &= free - 1, ++r) {
      const int page = first + __ffs(free) - 1;
      // the slot with excl[lo] <= r < excl[lo + 1]: often that of the page before or the next one
      if (excl[lo + 1] <= r && excl[++lo + 1] <= r) {
        int hi = c.n_slots;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (excl[mid] <= r) lo = mid;
          else hi = mid;
        }
      }
      c.table[(size_t)lo * c.max_pages + first_page[lo] + r - excl[lo]] = page;
      c.refs[page] = 1;
    }
    found += total;
  }
  __syncthreads();
  for (int s = tid; s < c.n_slots; s += kScanThreads) {
    const bool kept = s == tid;
    const int n = kept ? n0 : n_new[s], len = kept ? len0 : c.lengths[s], from = kept ? from0 : cow[s];
    const int need = excl[s + 1] - excl[s], begin = first_page[s];  // (need: 0 where the sums stand at 2^30)
    const bool nothing = ((long long)len + n + c.page - 1) / c.page == begin && from < 0;
    if (begin >= 0 && (nothing || excl[s + 1] <= found)) {
      pos[s] = len;
      if (n > 0) c.lengths[s] = len + n;
      if (from >= 0) atomicSub(c.refs + from, 1);
    } else {
      pos[s] = -1;
      cow[s] = -1;
      if (begin >= 0) {
        // too few pages: what this slot has been given goes back
        int* row = c.table + (size_t)s * c.max_pages + begin;
        for (int i = 0; i < need && excl[s] + i < found; ++i) c.refs[row[i]] = 0;
        if (from >= 0) row[0] = from;
        kv_error(c.status, kDevPages);
      }
    }
  }
}

// copy of `bytes` (a multiple of 16) with `n` threads, the t-th of them
__device__ __forceinline__ void copy16(void* dst, const void* src, size_t bytes, size_t t, size_t n) {
  const uint4* s = static_cast<const uint4*>(src);
  uint4* d = static_cast<uint4*>(dst);
  const size_t m = bytes / 16;
  size_t i = t;
  for (; i + 3 * n < m; i += 4 * n) {
    const uint4 a = s[i], b = s[i + n], e = s[i + 2 * n], f = s[i + 3 * n];
    d[i] = a, d[i + n] = b, d[i + 2 * n] = e, d[i + 3 * n] = f;
  }
  for (; i < m; i += n) d[i] = s[i];
}

// The pages that kv_extend_kernel moved from a shared page to one of the slot's own.
constexpr int kCowParts = 8;
__global__ void __launch_bounds__(256) kv_cow_kernel(const sage_kv_cache c, const int* __restrict__ pos,
                                                     const int* __restrict__ cow) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, from = cow[s];
  if (from < 0) return;
  const int to = c.table[(size_t)s * c.max_pages + pos[s] / c.page];
  const size_t bytes = (size_t)c.Hkv * c.page * c.D;
  const size_t t = blockIdx.y * 256 + threadIdx.x, n = kCowParts * 256, m = bytes / 16;
  const uint4 *kf = static_cast<const uint4*>(c.k) + from * m, *vf = static_cast<const uint4*>(c.v) + from * m;
  uint4 *kt = static_cast<uint4*>(c.k) + to * m, *vt = static_cast<uint4*>(c.v) + to * m;
  for (size_t i = t; i < m; i += 2 * n) {
    const bool two = i + n < m;
    const uint4 a = kf[i], b = vf[i];
    uint4 x, y;
    if (two) x = kf[i + n], y = vf[i + n];
    kt[i] = a, vt[i] = b;
    if (two) kt[i + n] = x, vt[i + n] = y;
  }
  for (size_t h = t; h < (size_t)c.Hkv; h += n) {
    c.k_scale[(size_t)to * c.Hkv + h] = c.k_scale[(size_t)from * c.Hkv + h];
    c.v_scale[(size_t)to * c.Hkv + h] = c.v_scale[(size_t)from * c.Hkv + h];
  }
}

// ------------------------------------------------------------------------------ compact

// ws: int count, then (256-byte aligned) int number[n_pages] (the new number of a live page, -1
// of a free one) and int live[n_pages] (the live pages in order).  One CTA: 16 pages a thread and step, an
// int at a time.  For pools of 10^5 pages and more the steps, one behind the other, would count.
__global__ void __launch_bounds__(kScanThreads) kv_rank_kernel(const sage_kv_cache c, int to_pages,
                                                               int* __restrict__ count, int* __restrict__ number,
                                                               int* __restrict__ live) {
  __shared__ int warp_sums[32];
  constexpr int kPer = 16;
  pdl_wait();
  pdl_trigger();
  int done = 0;
  for (int p0 = 0; p0 < c.n_pages; p0 += kScanThreads * kPer) {
    const int first = p0 + threadIdx.x * kPer;
    unsigned used = 0;
    for (int i = 0; i < kPer; ++i)
      if (first + i < c.n_pages && c.refs[first + i] > 0) used |= 1u << i;
    int total;
    int r = done + block_exclusive(__popc(used), warp_sums, &total);
    for (int i = 0; i < kPer && first + i < c.n_pages; ++i) {
      const bool u = used >> i & 1;
      number[first + i] = u ? r : -1;
      if (u) live[r++] = first + i;
    }
    done += total;
  }
  if (threadIdx.x == 0) {
    const bool fits = done <= to_pages;
    *count = fits ? done : -1;
    if (!fits) kv_error(c.status, kDevPages);
  }
}

// Persistent CTAs: first the tables, lengths and refs, then the live pages, a piece at a time.
__global__ void __launch_bounds__(256) kv_move_kernel(const sage_kv_cache c, const sage_kv_cache to,
                                                      const int* __restrict__ count, const int* __restrict__ number,
                                                      const int* __restrict__ live) {
  pdl_wait();
  pdl_trigger();
  const int n = *count;
  if (n < 0) return;
  const size_t t = (size_t)blockIdx.x * 256 + threadIdx.x, nt = (size_t)gridDim.x * 256;
  for (size_t i = t; i < (size_t)to.n_pages; i += nt) to.refs[i] = i < (size_t)n ? c.refs[live[i]] : 0;
  for (size_t i = t; i < (size_t)n * c.Hkv; i += nt) {
    const size_t from = (size_t)live[i / c.Hkv] * c.Hkv + i % c.Hkv;
    to.k_scale[i] = c.k_scale[from];
    to.v_scale[i] = c.v_scale[from];
  }
  for (size_t i = t; i < (size_t)c.n_slots * c.max_pages; i += nt) {
    const size_t s = i / c.max_pages, j = i % c.max_pages;
    if ((long long)j * c.page < c.lengths[s]) {
      const int page = c.table[i];
      const int now = (unsigned)page < (unsigned)c.n_pages ? number[page] : -1;
      to.table[i] = now;
      if (now < 0) kv_error(c.status, kDevIndex);  // out of range, or free and not moved
    }
  }
  for (size_t i = t; i < (size_t)c.n_slots; i += nt) to.lengths[i] = c.lengths[i];
  const size_t bytes = (size_t)c.Hkv * c.page * c.D;
  for (size_t i = blockIdx.x; i < 2 * (size_t)n; i += gridDim.x) {
    const bool v = i & 1;
    const size_t k = i >> 1;
    copy16(static_cast<uint8_t*>(v ? to.v : to.k) + k * bytes,
           static_cast<const uint8_t*>(v ? c.v : c.k) + (size_t)live[k] * bytes, bytes, threadIdx.x, 256);
  }
}

}  // namespace

size_t kv_compact_ws_bytes(int n_pages) { return 256 + 2 * (((size_t)n_pages * 4 + 255) & ~(size_t)255); }

int launch_kv_append(const sage_kv_cache& c, const void* K, const void* V, const float* k_shift, const int* slots,
                     const int* pos, const int* n_new, int B, int Nn, cudaStream_t st) {
  AppendParams p{c, static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V), k_shift, slots, pos,
                 n_new, B, Nn};
  const bool shift = k_shift != nullptr;
  auto kern = c.D == 128 ? append_kernel_for<128>(c.page, c.kind, shift) : append_kernel_for<64>(c.page, c.kind, shift);
  const unsigned pages = (unsigned)(((long long)Nn + c.page - 2) / c.page + 1);  // that Nn tokens can touch
  const int threads = append_threads(c.D, c.page), group = append_pages(c.D, c.page);
  ScopedTimer timer("kv_append", st);
  if (launch_pdl(kern, dim3((pages + group - 1) / group, 2 * c.Hkv, B), dim3(threads * group), 0, st, p) != cudaSuccess) return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

int launch_kv_fork(const sage_kv_cache& c, const int* src, cudaStream_t st) {
  ScopedTimer timer("kv_pages", st);
  if (launch_pdl(kv_fork_kernel, dim3(c.n_slots), dim3(256), 0, st, c, src) != cudaSuccess) return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

int launch_kv_truncate(const sage_kv_cache& c, const int* keep, cudaStream_t st) {
  ScopedTimer timer("kv_pages", st);
  if (launch_pdl(kv_truncate_kernel, dim3(c.n_slots), dim3(128), 0, st, c, keep) != cudaSuccess) return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

int launch_kv_extend(const sage_kv_cache& c, const int* n_new, int* pos, int* cow, cudaStream_t st) {
  ScopedTimer timer("kv_pages", st);
  const size_t smem = (2 * (size_t)c.n_slots + 1) * 4;
  // (48 KB with the static part need no leave; the limit is the process's, so it is the same in every call)
  constexpr size_t kMost = (2 * (size_t)kKvMaxSlots + 1) * 4;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(kv_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost) != cudaSuccess)
    return 3;
  if (launch_pdl(kv_extend_kernel, dim3(1), dim3(kScanThreads), smem, st, c, n_new, pos, cow) != cudaSuccess ||
      launch_pdl(kv_cow_kernel, dim3(c.n_slots, kCowParts), dim3(256), 0, st, c, (const int*)pos, (const int*)cow) !=
          cudaSuccess)
    return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

int launch_kv_compact(const sage_kv_cache& c, const sage_kv_cache& to, void* ws, cudaStream_t st) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  int* count = reinterpret_cast<int*>(w);
  int* number = reinterpret_cast<int*>(w + 256);
  int* live = reinterpret_cast<int*>(w + 256 + (((size_t)c.n_pages * 4 + 255) & ~(size_t)255));
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 3;
  ScopedTimer timer("kv_compact", st);
  if (launch_pdl(kv_rank_kernel, dim3(1), dim3(kScanThreads), 0, st, c, to.n_pages, count, number, live) !=
          cudaSuccess ||
      launch_pdl(kv_move_kernel, dim3(sms * 8), dim3(256), 0, st, c, to, (const int*)count, (const int*)number,
                 (const int*)live) != cudaSuccess)
    return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

}  // namespace sage
