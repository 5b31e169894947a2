// Rotary positions: the pairs of channels of every query and key turned by the angle of the token's position
// (sage_attn_rotary).
//
// HBM-bound: each value is read and written once.  A thread takes 16 channels of a token (two pieces of 16 bytes, whose
// pairs it holds whole in either layout) in up to kHeads heads, so that eight sines and cosines serve kHeads times 16
// values; all its loads are in flight before the first product.  32768 tokens of 32 and 8 heads: 98 us, 6.8 TB/s, what a
// copy reaches; 64 tokens: 2.4 us, a launch.
//
// The angle of pair c at position n is n times a frequency, of which only the part of a turn counts.  Frequencies come
// as 64-bit fractions of a turn, so n f modulo a turn is an integer product that wraps by itself: off by 2^-65 n turns at
// most (and by what the caller's frequency is off n times: n f 2^-53 for a double's rounding), where an fp32 product would
// lose the angle at 2^20.
#include <cuda_bf16.h>

#include "launch.h"
#include "ptx.cuh"
#include "rotary.h"
#include "timer.h"

namespace sage {

namespace {

constexpr int kThreads = 256;

// the position of token t of batch row b; false: it belongs to no sequence
__device__ __forceinline__ bool position_of(const RotaryParams& p, int b, int t, long long& pos) {
  if (p.positions) {
    pos = p.positions[(long long)b * p.N + t];
    return true;
  }
  if (!p.cu) {
    pos = (long long)t + (p.start ? p.start[b] : 0);
    return true;
  }
  // the last sequence that begins at or before t
  int lo = -1, hi = p.S + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  if (lo < 0 || lo >= p.S) return false;
  pos = (long long)t - p.cu[lo] + (p.start ? p.start[lo] : 0);
  return true;
}

// two channels of a word
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Threads: piece of the row, group of heads, token.  Thread (piece, g) takes heads g, g + groups, ...
template <int D, int kHeads>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p, int groups) {
  constexpr int kPieces = D / 16;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int piece = (int)(id % kPieces);
  const long long rest = id / kPieces;
  const int g = (int)(rest % groups);
  const long long token = rest / groups;
  pdl_wait();
  pdl_trigger();
  if (token >= (long long)p.B * p.N) return;
  const int b = (int)(token / p.N), t = (int)(token - (long long)b * p.N);
  long long pos;
  if (!position_of(p, b, t, pos)) return;
  const int turned = p.r.rot / 16;                // pieces that are
  const bool turns = piece < turned;
  // the two 16-byte vectors: the pairs' first and second channels, or (interleaved) four pairs each
  const int v0 = turns ? piece : 2 * piece, v1 = turns ? piece + turned : 2 * piece + 1;
  const int heads = p.heads[0] + p.heads[1];
  auto at = [&](const sage_heads* x, int h) {
    const bool k = h >= p.heads[0];
    const sage_heads& y = x[k];
    return static_cast<__nv_bfloat16*>(y.p) + b * y.batch + t * y.token + (k ? h - p.heads[0] : h) * y.head;
  };
  uint4 w[kHeads][2];
#pragma unroll
  for (int x = 0; x < kHeads; ++x) {
    const int h = g + x * groups;
    if (h >= heads) break;
    const uint4* row = reinterpret_cast<const uint4*>(at(p.in, h));
    w[x][0] = row[v0], w[x][1] = row[v1];
  }
  float c[8], s[8];
  if (turns) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int pair = p.r.interleaved ? 4 * (e < 4 ? v0 : v1) + (e & 3) : 8 * piece + e;
      const unsigned long long turn = (unsigned long long)pos * p.r.turns[pair];
      // the part of a turn in [-1/2, 1/2), to 32 bits
      sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s[e], &c[e]);
      c[e] *= p.r.gain;
      s[e] *= p.inverse ? -p.r.gain : p.r.gain;
    }
  }
#pragma unroll
  for (int x = 0; x < kHeads; ++x) {
    const int h = g + x * groups;
    if (h >= heads) break;
    if (turns) {
      uint32_t* u = reinterpret_cast<uint32_t*>(w[x]);  // eight words
      if (p.r.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = lo_of(u[e]), z = hi_of(u[e]);
          u[e] = pack(fmaf(a, c[e], -z * s[e]), fmaf(a, s[e], z * c[e]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = lo_of(u[e]), a1 = hi_of(u[e]), z0 = lo_of(u[4 + e]), z1 = hi_of(u[4 + e]);
          u[e] = pack(fmaf(a0, c[2 * e], -z0 * s[2 * e]), fmaf(a1, c[2 * e + 1], -z1 * s[2 * e + 1]));
          u[4 + e] = pack(fmaf(a0, s[2 * e], z0 * c[2 * e]), fmaf(a1, s[2 * e + 1], z1 * c[2 * e + 1]));
        }
      }
    }
    uint4* row = reinterpret_cast<uint4*>(at(p.out, h));
    row[v0] = w[x][0], row[v1] = w[x][1];
  }
}

template <int D, int kHeads>
int launch(const RotaryParams& p, cudaStream_t st) {
  const int heads = p.heads[0] + p.heads[1], groups = (heads + kHeads - 1) / kHeads;
  const long long blocks = ((long long)p.B * p.N * groups * (D / 16) + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return SAGE_ERR_UNSUPPORTED;
  const cudaError_t e = launch_pdl(rotary_kernel<D, kHeads>, dim3((unsigned)blocks), dim3(kThreads), 0, st, p, groups);
  return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA;
}

}  // namespace

int launch_rotary(const RotaryParams& p, int D, cudaStream_t st) {
  ScopedTimer timer("rotary", st);
  // four heads a thread where there are 152 x 2048 threads of them, else one.  With one and with four, 40 heads: 64 tokens
  // 2.3 and 2.8 us, 250 3.7 and 3.5, 1000 7.8 and 6.5, 2000 12.9 and 10.2, 4000 24.2 and 16.3, 32000 174 and 96.  They cross
  // near 200 tokens, well below the switch, which lies at 3900: up to there the one that is taken is the slower.
  const long long threads = (long long)p.B * p.N * ((p.heads[0] + p.heads[1] + 3) / 4) * (D / 16);
  if (threads >= 152 * 2048) return D == 128 ? launch<128, 4>(p, st) : launch<64, 4>(p, st);
  return D == 128 ? launch<128, 1>(p, st) : launch<64, 1>(p, st);
}

}  // namespace sage
