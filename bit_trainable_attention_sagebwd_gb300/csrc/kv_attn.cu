// Attention of new queries over the 8-bit paged cache (sage_attn_kv_attention).
//
// Row (b, h, i) sees keys j < end: O = sum_j p_j s_v(j) v_j / sum_j p_j, p_j = 2^(t_j - m),
// t_j = (q . k_j) s_k(j) sm_scale log2 e, with the codes k_j, v_j and one scale per (page, head).
//
// A token is answered at the rate at which the codes come from HBM: 2 Hkv D bytes per cached token
// against 4 H D operations, far below what the tensor cores could do.  So the kernel is built
// around the loads:
//  - The keys of all (batch row, key/value head) units form one line of 16-token chunks, cut into
//    equal parts for a grid that fills the GPU once; a unit that is cut leaves partial results,
//    joined by kv_join_kernel in the order of the parts.  Ragged batches and single long
//    sequences load every SM alike.
//  - A warp walks its own chunks and keeps kStages of them in flight with cp.async into a ring
//    that only the same lane reads: no barrier and no bank conflict, registers left for the
//    arithmetic.
//  - S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16, fp16): the codes are the 16-row operand, the
//    (at most 8 RT) query rows of the shared head the 8-column one, so a group of 8 query heads
//    wastes nothing.  A lane's registers are read from whole 16-byte pieces of a token's row; the
//    order of the contracted channels (K) and of the output channels (V) is permuted to fit.
//  - int8 and e4m3 codes are exact in fp16.  q is bf16: scaled by a power of two per row it is
//    exact in fp16 for every element within 2^-25 of the row's largest.  P is rounded to fp16
//    (2^-12 relative, p <= 1): bf16, the output's type, would lose more than the output's own
//    rounding.  Statistics, scales and sums are fp32.
#include "kv_attn.cuh"
#include "launch.h"
#include "timer.h"

namespace sage {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kChunk = 16;        // tokens of one step of a warp; a page is a whole number of them
constexpr int kStages = 4;        // chunks of a warp in flight
constexpr int kCtasPerSm = 3;     // the ring (4 warps x 4 chunks x 2 x 16 D bytes) of D = 128 is 64 KB

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 block of 16-bit values held one row pair per lane
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <int D>
struct Ring {
  static constexpr int kPieces = D / 32;                  // 16-byte K pieces of a lane and chunk
  static constexpr int kBytes = 2 * kChunk * D;           // K and V of a chunk
  static constexpr int kWarpBytes = kStages * kBytes;
};

// Cross-warp exchange at the end of a unit's part, in the ring's place: [warp][row][D + 4] sums,
// then maxima, row sums
template <int D, int RT>
struct Exchange {
  static constexpr int R = 8 * RT, kRow = D + 4;
  static constexpr int kFloats = kWarps * R * (kRow + 2);
  static_assert(kFloats * 4 <= kWarps * Ring<D>::kWarpBytes, "the exchange fits in the ring");
};

struct Unit {
  int b, slot, hk, tile, len, q_len, chunks;
};

template <int D, int KIND, int RT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv_attn_kernel(const AttnParams p) {
  constexpr int R = 8 * RT, NK = D / 16, NJ = D / 16;     // k-steps of S^T, 16-channel tiles of O^T
  constexpr int VB = D / 8;                               // bytes of a V piece (8 lanes cover a row)
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring = smem;
  float* xch = reinterpret_cast<float*>(smem);
  long long* pre = reinterpret_cast<long long*>(smem + kWarps * Ring<D>::kWarpBytes);  // [B + 1] chunks before a batch row
  __shared__ long long wsum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const sage_kv_cache& c = p.c;
  pdl_wait();
  pdl_trigger();

  // a unit without keys still has one (empty) chunk: its rows are written like any other's
  const int per_b = c.Hkv * p.tiles;
  prefix_of<kThreads>(p.B, pre, wsum, [&](int b) {
    int slot;
    return (long long)max(1, (row_length(p, b, slot) + kChunk - 1) / kChunk) * per_b;
  });
  __syncthreads();
  const long long total = pre[p.B];
  // a worker takes at least one chunk for each of its warps
  const int workers = (int)min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
  const int w0 = blockIdx.x;
  if (w0 >= workers) return;
  auto start_of = [&](int w) { return total * w / workers; };
  long long at = start_of(w0);
  const long long stop = start_of(w0 + 1);
  int b = row_at(pre, p.B, at);

  const uint32_t my_ring = smem_u32(ring) + warp * Ring<D>::kWarpBytes;
  const uint8_t* my_ring_p = ring + warp * Ring<D>::kWarpBytes;
  const int per_page = c.page / kChunk;
  const int page_shift = 31 - __clz(per_page);
  const size_t page_bytes = (size_t)c.page * D;

  while (at < stop) {
    while (pre[b + 1] <= at) ++b;
    Unit u;
    u.b = b;
    u.len = row_length(p, b, u.slot);
    u.chunks = max(1, (u.len + kChunk - 1) / kChunk);
    const int in_b = (int)((at - pre[b]) / u.chunks);
    const long long unit_at = pre[b] + (long long)in_b * u.chunks;
    u.tile = in_b / c.Hkv;
    u.hk = in_b % c.Hkv;
    u.q_len = row_queries(p, b);
    const int c0 = (int)(at - unit_at);
    const int c1 = (int)min((long long)u.chunks, stop - unit_at);
    const long long unit_id = (long long)b * per_b + in_b;
    if (c0 == 0 && tid == 0) {
      // the workers that hold the unit's first and last chunk
      int last = w0;
      while (start_of(last + 1) < unit_at + u.chunks) ++last;
      p.info[unit_id] = make_int2(w0, last);
    }
    at = unit_at + c1;

    // rows of this lane as B columns (row g of each 8-row tile) and as accumulator columns
    uint32_t qf[RT][NK][2];
    float ar[RT][2];   // alpha of accumulator columns 2 tig, 2 tig + 1, powers of two of q and codes taken back
    int lim[RT][2];    // keys that those rows see
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = u.tile * R + t * 8 + g, i = row / p.G;
      const bool live = i < u.q_len;
      const __nv_bfloat16* q =
          p.Q + (((size_t)b * p.H + (size_t)u.hk * p.G + row % p.G) * p.Nq + (live ? i : 0)) * D;
      float x[NK][4];
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        // channels of k-step s: 64 (s / 4) + 16 tig + 4 (s % 4) + 0..3
        uint2 w = make_uint2(0u, 0u);
        if (live) w = *reinterpret_cast<const uint2*>(q + (s >> 2) * 64 + tig * 16 + (s & 3) * 4);
        x[s][0] = __uint_as_float(w.x << 16), x[s][1] = __uint_as_float(w.x & 0xffff0000u);
        x[s][2] = __uint_as_float(w.y << 16), x[s][3] = __uint_as_float(w.y & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[s][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float up, down;
      row_power(top, up, down);
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        qf[t][s][0] = h2bits(__floats2half2_rn(x[s][0] * up, x[s][1] * up));
        qf[t][s][1] = h2bits(__floats2half2_rn(x[s][2] * up, x[s][3] * up));
      }
      const float a = p.alpha * down * kCodeUnit<KIND>;
      // (a row that is not there holds q = 0 and masks nothing; it is not stored)
      const int end = live ? row_end(p, u.len, u.q_len, i) : u.len;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ar[t][e] = __shfl_sync(0xffffffffu, a, (2 * tig + e) * 4);
        lim[t][e] = __shfl_sync(0xffffffffu, end, (2 * tig + e) * 4);
      }
    }
    int lim_min = lim[0][0];
#pragma unroll
    for (int t = 0; t < RT; ++t) lim_min = min(lim_min, min(lim[t][0], lim[t][1]));

    float acc[RT][NJ][4];
    float m[RT][2], l[RT][2];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][j][e] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }

    // chunk k of this warp is c0 + warp + kWarps k; a lane looks up one of 32 pages at a time
    const int mine = c1 > c0 + warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
    const int* row = c.table + (size_t)u.slot * c.max_pages;
    int id_next = -1, id_now = -1;
    float ks_now = 0.f, vs_now = 0.f, ks_next = 0.f, vs_next = 0.f;
    auto look_up = [&](int k, int& id, float& ks, float& vs) {
      id = -1, ks = vs = 0.f;
      const int ch = c0 + warp + kWarps * k;
      if (k < mine && ch * kChunk < u.len) {
        const int page = row[ch >> page_shift];
        if ((unsigned)page < (unsigned)c.n_pages) {
          id = page;
          ks = c.k_scale[(size_t)page * c.Hkv + u.hk];
          vs = c.v_scale[(size_t)page * c.Hkv + u.hk] * kCodeUnit<KIND>;
        } else {
          atomicMax(c.status, kDevIndex);
        }
      }
    };
    auto issue = [&](int k) {
      if (k < mine) {
        const int id = __shfl_sync(0xffffffffu, (k >> 5) & 1 ? id_next : id_now, k & 31);
        if (id >= 0) {
          const int ch = c0 + warp + kWarps * k;
          const size_t off = ((size_t)id * c.Hkv + u.hk) * page_bytes + (size_t)((ch & (per_page - 1)) * kChunk) * D;
          const uint8_t* kp = static_cast<const uint8_t*>(c.k) + off;
          const uint8_t* vp = static_cast<const uint8_t*>(c.v) + off;
          const uint32_t dst = my_ring + (k % kStages) * Ring<D>::kBytes;
#pragma unroll
          for (int i = 0; i < Ring<D>::kPieces; ++i) {
            // D = 128: pieces 0, 1 of token g, 2, 3 of token g + 8; D = 64: one piece of each
            const int tok = g + (D == 128 ? 8 * (i >> 1) : 8 * i), byte = tig * 16 + (D == 128 ? 64 * (i & 1) : 0);
            cp_async16(dst + (i * 32 + lane) * 16, kp + tok * D + byte);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 2 * tig + (i & 1) + 8 * (i >> 1);
            if (D == 128)
              cp_async16(dst + kChunk * D + (i * 32 + lane) * 16, vp + tok * D + g * VB);
            else
              cp_async8(dst + kChunk * D + (i * 32 + lane) * 8, vp + tok * D + g * VB);
          }
        }
      }
      cp_commit();
    };
    look_up(lane, id_now, ks_now, vs_now);
    look_up(lane + 32, id_next, ks_next, vs_next);
#pragma unroll 1
    for (int k = 0; k < kStages - 1; ++k) issue(k);

#pragma unroll 1
    for (int k = 0; k < mine; ++k) {
      cp_wait<kStages - 2>();
      issue(k + kStages - 1);
      const bool odd = (k >> 5) & 1;
      const int id = __shfl_sync(0xffffffffu, odd ? id_next : id_now, k & 31);
      const float ks = __shfl_sync(0xffffffffu, odd ? ks_next : ks_now, k & 31);
      const float vs = __shfl_sync(0xffffffffu, odd ? vs_next : vs_now, k & 31);
      if ((k & 31) == 31) {
        // the 32 pages just finished make room for those 64 ahead
        if (odd) look_up(k + 33 + lane, id_next, ks_next, vs_next);
        else look_up(k + 33 + lane, id_now, ks_now, vs_now);
      }
      if (id < 0) continue;
      const uint8_t* src = my_ring_p + (k % kStages) * Ring<D>::kBytes;
      // S^T
      float s[RT][4];
#pragma unroll
      for (int t = 0; t < RT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
      constexpr int HP = Ring<D>::kPieces / 2;  // pieces of one token
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        const uint4 ka = reinterpret_cast<const uint4*>(src)[h * 32 + lane];
        const uint4 kb = reinterpret_cast<const uint4*>(src)[(HP + h) * 32 + lane];
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          codes_to_half<KIND>(wa[w], a0, a2);
          codes_to_half<KIND>(wb[w], a1, a3);
#pragma unroll
          for (int t = 0; t < RT; ++t) mma16816(s[t], a0, a1, a2, a3, qf[t][h * 4 + w][0], qf[t][h * 4 + w][1]);
        }
      }
      // softmax of the lane's tokens g, g + 8 in rows 2 tig, 2 tig + 1
      const int j0 = (c0 + warp + kWarps * k) * kChunk + g;
      const bool edge = (c0 + warp + kWarps * k) * kChunk + kChunk > lim_min;
      uint32_t pb[RT][2];
      float corr[RT][2];
      bool moved = false;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = ar[t][e] * ks;
          s[t][e] *= f;
          s[t][2 + e] *= f;
          if (edge) {
            if (j0 >= lim[t][e]) s[t][e] = -INFINITY;
            if (j0 + 8 >= lim[t][e]) s[t][2 + e] = -INFINITY;
          }
          float mx = fmaxf(s[t][e], s[t][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[t][e], mx);
          const float sub = mn == -INFINITY ? 0.f : mn;
          corr[t][e] = ex2(m[t][e] - sub);
          moved |= mn != m[t][e];
          m[t][e] = mn;
          s[t][e] = ex2(s[t][e] - sub);
          s[t][2 + e] = ex2(s[t][2 + e] - sub);
          l[t][e] = l[t][e] * corr[t][e] + (s[t][e] + s[t][2 + e]);
        }
        pb[t][0] = movmatrix(h2bits(__floats2half2_rn(s[t][0], s[t][1])));
        pb[t][1] = movmatrix(h2bits(__floats2half2_rn(s[t][2], s[t][3])));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][j][e] *= corr[t][e & 1];
      }
      // O^T: tokens 2 tig, 2 tig + 1 (pair 0) and + 8 (pair 1), channels g VB + 2 j, + 1 of tile j
      const uint8_t* vsrc = src + kChunk * D;
      uint32_t v[4][VB / 4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (D == 128) {
          const uint4 x = reinterpret_cast<const uint4*>(vsrc)[i * 32 + lane];
          v[i][0] = x.x, v[i][1] = x.y, v[i][VB / 4 - 2] = x.z, v[i][VB / 4 - 1] = x.w;
        } else {
          const uint2 x = reinterpret_cast<const uint2*>(vsrc)[i * 32 + lane];
          v[i][0] = x.x, v[i][1] = x.y;
        }
      }
#pragma unroll
      for (int w = 0; w < VB / 4; ++w) {
        uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
        codes_to_half<KIND>(__byte_perm(v[0][w], v[1][w], 0x5140), a0, a1);
        codes_to_half<KIND>(__byte_perm(v[2][w], v[3][w], 0x5140), a2, a3);
        codes_to_half<KIND>(__byte_perm(v[0][w], v[1][w], 0x7362), b0, b1);
        codes_to_half<KIND>(__byte_perm(v[2][w], v[3][w], 0x7362), b2, b3);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816(d0, a0, a1, a2, a3, pb[t][0], pb[t][1]);
          mma16816(d1, b0, b1, b2, b3, pb[t][0], pb[t][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[t][2 * w][e] = fmaf(vs, d0[e], acc[t][2 * w][e]);
            acc[t][2 * w + 1][e] = fmaf(vs, d1[e], acc[t][2 * w + 1][e]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // ---- the warps' results of this part
    constexpr int kRow = Exchange<D, RT>::kRow;
    float* xm = xch + kWarps * R * kRow;  // [warp][R] maxima
    float* xl = xm + kWarps * R;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[t][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int r = t * 8 + 2 * tig + e;
        if (g == 0) xm[warp * R + r] = m[t][e], xl[warp * R + r] = s;
        float* dst = xch + (size_t)(warp * R + r) * kRow + g * VB;
#pragma unroll
        for (int j = 0; j < NJ; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) =
              make_float4(acc[t][j][e], acc[t][j][2 + e], acc[t][j + 1][e], acc[t][j + 1][2 + e]);
      }
    }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == u.chunks;
    float* part = p.part + (size_t)(2 * w0 + (c0 == 0 ? 1 : 0)) * R * (D + 2);
    for (int x = tid; x < R * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      const int rw = u.tile * R + r, i = rw / p.G;
      if (i >= u.q_len) continue;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, xm[w * R + r]);
      const float sub = mt == -INFINITY ? 0.f : mt;
      float ls = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(xm[w * R + r] - sub);
        ls = fmaf(f, xl[w * R + r], ls);
        const float4 y = *reinterpret_cast<const float4*>(xch + (size_t)(w * R + r) * kRow + d);
        o[0] = fmaf(f, y.x, o[0]), o[1] = fmaf(f, y.y, o[1]), o[2] = fmaf(f, y.z, o[2]), o[3] = fmaf(f, y.w, o[3]);
      }
      if (whole) {
        const float inv = ls > 0.f ? 1.f / ls : 0.f;
        const size_t orow = ((size_t)b * p.H + (size_t)u.hk * p.G + rw % p.G) * p.Nq + i;
        uint2 out;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&out);
        h[0] = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
        h[1] = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(p.O + orow * D + d) = out;
        if (d == 0) p.LSE[orow] = ls > 0.f ? (mt + log2f(ls)) * 0.69314718055994531f : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = make_float4(o[0], o[1], o[2], o[3]);
        if (d == 0) part[R * D + r] = mt, part[R * D + R + r] = ls;
      }
    }
    __syncthreads();  // the exchange is read before the next part fills it
  }
}

// Joins the parts of the units that were cut, in their order.  WARPS = 4: one CTA per (unit, row),
// a quarter of the parts to each warp (few units, many parts).  WARPS = 1: four rows to a CTA, one
// to each warp.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) kv_join_kernel(const AttnParams p, int R) {
  constexpr int E = D / 32;  // channels of a lane
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = blockIdx.x;
  const int r = WARPS == 4 ? blockIdx.y : blockIdx.y * 4 + warp;
  const int per_b = p.c.Hkv * p.tiles, b = (int)(unit / per_b), in_b = (int)(unit % per_b);
  const int hk = in_b % p.c.Hkv, row = in_b / p.c.Hkv * R + r, i = row / p.G;
  if (i >= row_queries(p, b)) return;
  const int2 w = p.info[unit];
  if (w.x == w.y) return;
  const size_t stride = (size_t)R * (D + 2);
  auto part_of = [&](int k) { return p.part + (size_t)(k == w.x ? 2 * k + 1 : 2 * k) * stride; };
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int k0 = w.x + (WARPS == 4 ? warp : 0); k0 <= w.y; k0 += 4 * WARPS) {
    // four parts at a time, their loads in flight together
    float mm[4], ll[4], oo[4][E];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + WARPS * q;
      mm[q] = -INFINITY, ll[q] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) oo[q][e] = 0.f;
      if (k <= w.y) {
        const float* s = part_of(k);
        mm[q] = s[R * D + r], ll[q] = s[R * D + R + r];
#pragma unroll
        for (int e = 0; e < E; ++e) oo[q][e] = s[r * D + e * 32 + lane];
      }
    }
    float mn = m;
#pragma unroll
    for (int q = 0; q < 4; ++q) mn = fmaxf(mn, mm[q]);
    const float sub = mn == -INFINITY ? 0.f : mn;
    const float f0 = ex2(m - sub);
    l *= f0;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float f = ex2(mm[q] - sub);
      l = fmaf(f, ll[q], l);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, oo[q][e], o[e]);
    }
    m = mn;
  }
  const size_t orow = ((size_t)b * p.H + (size_t)hk * p.G + row % p.G) * p.Nq + i;
  if (WARPS == 1) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) p.O[orow * D + e * 32 + lane] = __float2bfloat16_rn(o[e] * inv);
    if (lane == 0) p.LSE[orow] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    return;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  const float mt = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float sub = mt == -INFINITY ? 0.f : mt;
  float ls = 0.f, x = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = ex2(sm[k] - sub);
    ls = fmaf(f, sl[k], ls);
    x = fmaf(f, so[k][d], x);
  }
  p.O[orow * D + d] = __float2bfloat16_rn(ls > 0.f ? x / ls : 0.f);
  if (d == 0) p.LSE[orow] = ls > 0.f ? (mt + log2f(ls)) * 0.69314718055994531f : -INFINITY;
}

template <int D, int KIND, int RT>
int launch_few(const AttnParams& p, int sms, cudaStream_t st) {
  auto kern = kv_attn_kernel<D, KIND, RT>;
  const size_t smem = (size_t)kWarps * Ring<D>::kWarpBytes + ((size_t)p.B + 1) * 8;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 3;
  const int grid = sms * kCtasPerSm < kMaxWorkers ? sms * kCtasPerSm : kMaxWorkers;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, p) == cudaSuccess ? 0 : 3;
}
template <int D, int KIND>
int launch_few(const AttnParams& p, int rows, int sms, cudaStream_t st) {
  return rows == 8 ? launch_few<D, KIND, 1>(p, sms, st) : launch_few<D, KIND, 2>(p, sms, st);
}

// Query rows of a unit: 8 where all rows of a shared head fit in one, 16 up to kFewRows rows, then
// the tensor-core kernel's 256.
constexpr long long kFewRows = 32;

}  // namespace

int launch_kv_few(const AttnParams& p, int kind, int rows, int sms, cudaStream_t st) {
  if (p.c.D == 128)
    return kind == SAGE_KV_INT8 ? launch_few<128, SAGE_KV_INT8>(p, rows, sms, st)
                                : launch_few<128, SAGE_KV_E4M3>(p, rows, sms, st);
  return kind == SAGE_KV_INT8 ? launch_few<64, SAGE_KV_INT8>(p, rows, sms, st)
                              : launch_few<64, SAGE_KV_E4M3>(p, rows, sms, st);
}

KvAttnWs kv_attn_ws_layout(int B, int H, int Hkv, int D, int Nq) {
  KvAttnWs L{};
  const long long rows = (long long)(H / Hkv) * Nq;
  L.rows = rows <= 8 ? 8 : rows <= kFewRows ? 16 : kChunkRows;
  L.tiles = (int)((rows + L.rows - 1) / L.rows);
  L.info = 0;
  L.part = ((size_t)B * Hkv * L.tiles * 8 + 255) & ~(size_t)255;
  const size_t workers = L.rows == kChunkRows ? kMaxChunkWorkers : kMaxWorkers;
  L.total = L.part + workers * 2 * L.rows * (D + 2) * 4;
  return L;
}

int launch_kv_attention(const sage_kv_cache& c, const void* Q, const int* slots, const int* q_len, void* O,
                        float* LSE, void* ws, int B, int H, int Nq, int causal, float sm_scale, cudaStream_t st) {
  const KvAttnWs L = kv_attn_ws_layout(B, H, c.Hkv, c.D, Nq);
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnParams p;
  p.c = c;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.slots = slots;
  p.q_len = q_len;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.LSE = LSE;
  p.info = reinterpret_cast<int2*>(w + L.info);
  p.part = reinterpret_cast<float*>(w + L.part);
  p.B = B;
  p.H = H;
  p.G = H / c.Hkv;
  p.Nq = Nq;
  p.tiles = L.tiles;
  p.causal = causal;
  p.alpha = (float)((double)sm_scale * 1.4426950408889634074);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 3;
  ScopedTimer timer("kv_attention", st);
  const bool many = L.rows == kChunkRows;
  if (int rc = many ? launch_kv_chunk(p, c.kind, sms, st) : launch_kv_few(p, c.kind, L.rows, sms, st)) return rc;
  const unsigned units = (unsigned)((long long)B * c.Hkv * L.tiles);
  auto join = many ? (c.D == 128 ? kv_join_kernel<128, 1> : kv_join_kernel<64, 1>)
                   : (c.D == 128 ? kv_join_kernel<128, 4> : kv_join_kernel<64, 4>);
  if (launch_pdl(join, dim3(units, many ? L.rows / 4 : L.rows), dim3(128), 0, st, p, L.rows) != cudaSuccess) return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

}  // namespace sage
