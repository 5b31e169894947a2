// Attention of new queries over the 8-bit paged cache (sage_attn_kv_attention).
//
// Row (b, h, i) sees keys j < end: O = sum_j p_j s_v(j) v_j / sum_j p_j, p_j = 2^(t_j - m),
// t_j = (q . k_j) s_k(j) sm_scale log2 e, with the codes k_j, v_j and one scale per (page, head).
//
// A token is answered at the rate at which the codes come from HBM: 2 Hkv D bytes per cached token
// against 4 H D operations, far below what the tensor cores could do.  So the kernel is built
// around the loads:
//  - The keys of all (batch row, key/value head) units form one line of 32-token chunks, cut into
//    equal parts for a grid that fills the GPU once; a unit that is cut leaves partial results,
//    joined by kv_join_kernel in the order of the parts.  Ragged batches and single long
//    sequences load every SM alike.  Every unit begins with kPad places without a chunk, for the time
//    that its start takes; on a line too short to fill the GPU some parts are padding alone.
//  - A warp walks its own chunks and keeps kStages - 1 of them in flight with TMA, across the ends of
//    units, in a ring of its own: a chunk of K or V is one box of a page's [head, token] rows (two with
//    pages of 16 tokens).  (Copies of 16 bytes a thread, cp.async, read the same bytes at 5.6 TB/s against 6.7.)
//  - S^T = K Q^T and O^T = V^T P^T (mma.sync m16n8k16, fp16): the codes are the 16-row operand, the
//    (at most 8 RT) query rows of the shared head the 8-column one, so a group of 8 query heads
//    wastes nothing.  A lane's registers are read from whole 16-byte pieces of a token's row; the
//    order of the contracted channels (K) and of the output channels (V) is permuted to fit.
//  - int8 and e4m3 codes are exact in fp16.  q is bf16: scaled by a power of two per row it is
//    exact in fp16 for every element within 2^-25 of the row's largest.  P is rounded to fp16
//    (2^-11 relative at most): bf16, the output's type, would lose as much as the output's own
//    rounding.  Statistics, scales and sums are fp32.
//
// Measured, 32 query heads over 8 of D = 128, the join included: one token for each of 64 sequences of 500 to
// 8192 tokens (int8, 0.57 GB) in 95 us, of 4 of 100k to 131k (e4m3, 0.95 GB) in 159 us: 5.9 TB/s, 87 % of
// the rate of a plain copy.  What is left is the start of the units and the join.  With one to four queries each
// (16 rows, 16 sequences of 900 to 16k tokens, 0.28 GB) 62 us, 4.6 TB/s: eight warps of 255 registers issue
// in half of the cycles, the ALU (codes into fp16) at 51 %, and neither more warps nor fewer
// registers helped (three CTAs with Q in shared memory: 75 us).  D = 64, e4m3, 24 heads of their own, 12
// sequences of 300 to 16k (0.31 GB): 57 us, 5.5 TB/s, the ALU at 54 %.
#include "kv_attn.cuh"
#include "launch.h"
#include "timer.h"
#include "tmap.h"

namespace sage {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kSub = 2;           // 16-token MMA row tiles of a chunk
constexpr int kChunk = 16 * kSub; // tokens of one step of a warp
// Chunks of a warp in flight or at work, and CTAs an SM.  D = 64 with 8 query rows: three CTAs of 168
// registers a thread and two chunks (12 sequences of 0.3-16k tokens: 57 us, 63 us the other way).  Else two
// CTAs of 255 and three chunks: D = 128 gains 3 % by it (4 of 100-131k tokens: 159 us, 164 us the other
// way), and 16 rows at 168 registers spill (75 us against 62 us).
template <int D, int RT>
constexpr bool kThreeCtas = D == 64 && RT == 1;
template <int D, int RT>
constexpr int kStages = kThreeCtas<D, RT> ? 2 : 3;
template <int D, int RT>
constexpr int kCtasPerSm = kThreeCtas<D, RT> ? 3 : 2;
// What the start of a unit costs a CTA, in chunks of the line.  64 sequences of 500 to 8192 tokens took
// 109 us without, 101 us with 4, 99 us with 8 to 16; 256 of 100 to 1000 110, 93, 83 and 82 us.  Lines that do
// not fill the GPU are cut with it too, at a cost: one sequence of 700 tokens on 8 heads is 48 parts, two of each
// head's six without a chunk.
constexpr int kPad = 12;

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four codes of a word as fp16, in two pairs.  e4m3: the conversion instruction (bytes 0, 1 and 2, 3), true
// values, NaN for a NaN code; faster here than codes_to_half by a tenth at D = 64 (there it is slower: the
// packing of P takes the same unit).  int8: bytes 0, 2 and 1, 3.
template <int KIND>
__device__ __forceinline__ void pairs(uint32_t w, uint32_t& first, uint32_t& second) {
  if (KIND == SAGE_KV_INT8)
    codes_to_half<KIND>(w, first, second);
  else
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(first), "=r"(second)
        : "r"(w));
}
// A maximum above this one raises the reference m.  Rounded down, no fp32 lies between it and m + kRaise; to nearest
// it would pass m + kRaise from 2^25 on, and P 2^15.  (Known before the maximum is: its difference from m is not.)
__device__ __forceinline__ float raise_past(float m) { return __fadd_rd(m, kRaise); }
// transpose of an 8 x 8 block of 16-bit values held one row pair per lane
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <int D, int RT>
struct Ring {
  static constexpr int kBytes = 2 * kChunk * D;  // K and V of a chunk; also 16 rows of D fp32
  static constexpr int kWarpBytes = kStages<D, RT> * kBytes;
};

// A part of a unit: chunks [c0, c1) of a row tile of (batch row b, key/value head hk); `next`: where
// on the line it ends, `unit_at`: where the unit's first chunk is.
struct FewSeg {
  int b, slot, len, hk, tile, chunks, c0, c1;
  long long unit_at, next;
};

template <int D, int KIND, int RT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D, RT>)
    kv_attn_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  constexpr int R = 8 * RT, NK = D / 16, NJ = D / 16;     // k-steps of S^T, 16-channel tiles of O^T
  constexpr int VB = D / 8;                               // bytes of a V piece (8 lanes cover a row)
  constexpr int kPlaces = kStages<D, RT>;
  constexpr bool kNan = KIND == SAGE_KV_E4M3;             // a byte may be NaN (what pairs() makes of int8 is finite)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  long long* pre = reinterpret_cast<long long*>(ring + kWarps * Ring<D, RT>::kWarpBytes);  // [B + 1] chunks before a batch row
  int2* rows = reinterpret_cast<int2*>(pre + p.B + 1);                                // [B] slot, length
  __shared__ long long wsum[kWarps];
  __shared__ uint64_t bars[kWarps][kPlaces];  // a ring place's copies have landed
  __shared__ float4 meta[kWarps][kPlaces][kSub];  // K scale, log2 of V's scale (-inf: no keys there) and its inverse
  __shared__ int abort;
  __shared__ float xm[kWarps][R], xl[kWarps][R];
  __shared__ int left_place[kWarps];
  __shared__ __align__(16) __nv_bfloat16 q_buf[2][R * D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const sage_kv_cache& c = p.c;
  if (tid < kWarps * kPlaces) mbar_init(&bars[0][0] + tid, 1);
  if (tid == 0) abort = 0;
  fence_mbar_init();
  tma_prefetch_desc(&tm_k);
  tma_prefetch_desc(&tm_v);
  pdl_wait();
  pdl_trigger();

  // a unit without keys still has one (empty) chunk: its rows are written like any other's
  const int per_b = c.Hkv * p.tiles;
  prefix_of<kThreads>(p.B, pre, wsum, [&](int b) {
    int slot;
    const int len = row_length(p, b, slot);
    rows[b] = make_int2(slot, len);
    return (long long)(kPad + max(1, (len + kChunk - 1) / kChunk)) * per_b;
  });
  __syncthreads();
  const long long total = pre[p.B];
  // As many parts as give each warp a chunk where the units allow it (counted without the padding, which then
  // takes parts of its own: see kPad).  A line that does not fill the GPU, or is one sequence's, is cut so that the
  // parts of units of one length end with them: a part that goes on into another unit costs its CTA another start.
  const long long units = (long long)p.B * per_b;
  int parts = (int)min((long long)p.most_parts, max(units, (total - kPad * units + kWarps - 1) / kWarps));
  if (parts < p.most_parts || p.B == 1) {
    const long long up = (parts + units - 1) / units * units;
    parts = up <= p.most_parts ? (int)up : parts >= units ? parts - (int)(parts % units) : parts;
  }
  const Line line{total, parts};
  const int w0 = blockIdx.x;
  if (w0 >= parts) return;
  const long long begin = line.start(w0), stop = line.start(w0 + 1);
  if (begin >= stop) return;
  // the part of a unit that begins at `at`, in batch row b or behind it
  auto seg_at = [&](long long at, int b) {
    FewSeg s;
    while (pre[b + 1] <= at) ++b;
    s.b = b;
    s.slot = rows[b].x, s.len = rows[b].y;
    s.chunks = max(1, (s.len + kChunk - 1) / kChunk);
    const long long in = at - pre[b];
    const int size = kPad + s.chunks;
    const int in_b = in <= 0xffffffffll ? (int)((uint32_t)in / (uint32_t)size) : (int)(in / size);
    s.tile = in_b / c.Hkv;
    s.hk = in_b % c.Hkv;
    s.unit_at = pre[b] + (long long)in_b * size + kPad;
    s.next = min(s.unit_at + s.chunks, stop);
    s.c0 = (int)max(0ll, at - s.unit_at);
    s.c1 = (int)max(0ll, s.next - s.unit_at);
    return s;
  };
  // chunk k of this warp in a part is c0 + warp + kWarps k
  auto chunks_of = [&](const FewSeg& s) { return max(0, (s.c1 - s.c0 - warp + kWarps - 1) / kWarps); };

  // ---- copies.  They run ahead of the products, across parts, in windows of up to 32 chunks: a
  // lane looks after one chunk, its page a window ahead.
  uint8_t* my_ring = ring + warp * Ring<D, RT>::kWarpBytes;
  const int page_shift = 31 - __clz(c.page);
  const bool halves = c.page < kChunk;  // a chunk is two pages of 16 tokens
  int b = row_at(pre, p.B, begin);
  FewSeg ns = seg_at(begin, b);    // the next window: window nw of part ns, nn chunks of this warp in it
  int nw = 0, nn = chunks_of(ns), next_page = -1, next_half = -1, next_keys = 0;  // (keys from the lane's chunk on)
  bool have_next = true;
  int left = 0, at_i = 0;          // chunks of the window that are still to be copied, and the next one's lane
  int w_page = -1, w_half = -1, w_row = 0;  // the lane's chunk: page (-1: no keys), that of its second half, row
  float ref = 0.f;
  float4 w_meta[kSub] = {};
  auto load_window = [&]() {
    const int k = nw * 32 + lane, token = (ns.c0 + warp + kWarps * k) * kChunk;
    const int* row = c.table + (size_t)ns.slot * c.max_pages + (token >> page_shift);
    next_keys = k < nn ? ns.len - token : 0;
    next_page = next_keys > 0 ? row[0] : -1;
    next_half = halves && next_keys > 16 ? row[1] : -1;
  };
  auto next_window = [&]() {
    if (++nw * 32 >= nn) {
      nw = 0;
      do {
        if (ns.next >= stop) {
          have_next = false;
          return;
        }
        ns = seg_at(ns.next, ns.b);
        nn = chunks_of(ns);
      } while (nn == 0);
    }
    load_window();
  };
  int place = 0, flight = 0;       // ring place of the next copy; chunks copied or on their way, not yet used
  auto issue = [&]() {
    float ks[kSub] = {}, vs[kSub] = {};
    const bool enter = left == 0 && have_next;
    if (enter) {
      w_page = (unsigned)next_page < (unsigned)c.n_pages ? next_page : -1;
      w_half = (unsigned)next_half < (unsigned)c.n_pages ? next_half : -1;
      // (by the keys that are there, not by next_page: a table may say -1 among them)
      if ((next_keys > 0 && w_page < 0) || (halves && next_keys > 16 && w_half < 0)) atomicMax(c.status, kDevIndex);
      w_row = ns.hk * c.page + (((ns.c0 + warp + kWarps * (nw * 32 + lane)) * kChunk) & (c.page - 1));
      const int second = halves ? w_half : w_page;
      if (w_page >= 0) {
        ks[0] = c.k_scale[(size_t)w_page * c.Hkv + ns.hk];
        vs[0] = c.v_scale[(size_t)w_page * c.Hkv + ns.hk];
      }
      if (second >= 0) {
        ks[1] = c.k_scale[(size_t)second * c.Hkv + ns.hk];
        vs[1] = c.v_scale[(size_t)second * c.Hkv + ns.hk];
      }
      left = min(32, nn - nw * 32);
      at_i = 0;
      next_window();
    }
    if (left == 0) return;
    const int page = __shfl_sync(0xffffffffu, w_page, at_i), row = __shfl_sync(0xffffffffu, w_row, at_i);
    const int half = halves ? __shfl_sync(0xffffffffu, w_half, at_i) : -1;
    uint64_t* bar = &bars[warp][place];
    if (lane == 0) {
      uint8_t* dst = my_ring + place * Ring<D, RT>::kBytes;
      const uint32_t box = Ring<D, RT>::kBytes >> (halves ? 1 : 0);
      const uint32_t bytes = (page >= 0 ? box : 0) + (half >= 0 ? box : 0);
      if (bytes)
        mbar_arrive_expect_tx(bar, bytes);
      else
        mbar_arrive(bar);
      if (page >= 0) {
        tma_load_3d(dst, &tm_k, 0, row, page, bar);
        tma_load_3d(dst + kChunk * D, &tm_v, 0, row, page, bar);
      }
      if (half >= 0) {
        tma_load_3d(dst + 16 * D, &tm_k, 0, row, half, bar);
        tma_load_3d(dst + (kChunk + 16) * D, &tm_v, 0, row, half, bar);
      }
    }
    if (enter) {  // (the scales have been on their way)
      float big = fmaxf(vs[0], vs[1]);
#pragma unroll
      for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      ref = fmaxf(ref, big);
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        const float ve = value_scale(vs[h], ref);
        const bool none = (h && halves ? w_half : w_page) < 0;
        w_meta[h] = make_float4(ks[h], none ? -INFINITY : lg2(ve), __frcp_rn(ve), 0.f);
      }
    }
    if (lane == at_i) {
#pragma unroll
      for (int h = 0; h < kSub; ++h) meta[warp][place][h] = w_meta[h];
    }
    ++at_i, --left, ++flight;
    place = place + 1 == kPlaces ? 0 : place + 1;
  };
  // where a lane reads in a 128-byte (D = 64: 64-byte) swizzled box.  MMA row g stands for token
  // tk = g, odd g for g ^ 4: the eight lanes of a load then meet in no bank.  K token tk, unit tig (and
  // tig + 4); V tokens 2 tig, (2 tig + 1) ^ 4 (and + 8), channels g VB ..
  const int tk = g ^ (g & 1) << 2, tv = (2 * tig + 1) ^ 4;
  const uint32_t at_k = D == 128 ? tk * 128 + ((tig ^ tk) << 4) : tk * 64 + ((tig ^ (tk >> 1)) << 4);
  const uint32_t at_v0 = D == 128 ? tig * 256 + ((g ^ 2 * tig) << 4) : tig * 128 + (((g >> 1) ^ tig) << 4) + (g & 1) * 8;
  const uint32_t at_v1 = D == 128 ? tv * 128 + ((g ^ tv) << 4) : tv * 64 + (((g >> 1) ^ (tv >> 1)) << 4) + (g & 1) * 8;
  if (nn) load_window();
  else next_window();

  uint32_t phase = 0;
  int here = 0;                    // ring place of the next products
  // Q of a part's rows, a part ahead
  auto fetch_q = [&](const FewSeg& u, int to) {
    const int q_len = row_queries(p, u.b);
    for (int x = tid; x < R * (D / 8); x += kThreads) {
      const int r = x / (D / 8), row = u.tile * R + r, i = row / p.G;
      const bool live = i < q_len;
      const __nv_bfloat16* q =
          p.Q + (((size_t)u.b * p.H + (size_t)u.hk * p.G + row % p.G) * p.Nq + (live ? i : 0)) * D + x % (D / 8) * 8;
      cp_async16_or_zero(smem_u32(&q_buf[to][0]) + x * 16, q, live);
    }
    cp_commit();
  };
  FewSeg u = seg_at(begin, b);
  fetch_q(u, 0);
#pragma unroll 1
  for (int k = 0; k < kPlaces - 1; ++k) issue();
  cp_wait<0>();
  __syncthreads();
  for (int q_at = 0;; q_at ^= 1) {
    b = u.b;
    const int q_len = row_queries(p, b);
    FewSeg after = u;
    if (u.next < stop) {
      after = seg_at(u.next, b);
      fetch_q(after, q_at ^ 1);
    }
    if (u.c0 == 0 && u.c1 > 0 && tid == 0)  // the parts that hold the unit's first and last chunk
      p.info[(long long)b * per_b + u.tile * c.Hkv + u.hk] = make_int2(w0, line.holder(u.unit_at + u.chunks - 1));

    // rows of this lane as B columns (row g of each 8-row tile) and as accumulator columns
    uint32_t qf[RT][NK][2];
    float ar[RT][2];   // alpha of accumulator columns 2 tig, 2 tig + 1, powers of two of q and codes taken back
    int lim[RT][2];    // keys that those rows see
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int row = u.tile * R + t * 8 + g, i = row / p.G;
      const bool live = i < q_len;
      float x[NK][4];
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        // channels of k-step s: 64 (s / 4) + 16 tig + 4 (s % 4) + 0..3
        const uint2 w = *reinterpret_cast<const uint2*>(&q_buf[q_at][(t * 8 + g) * D + (s >> 2) * 64 + tig * 16 + (s & 3) * 4]);
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
        constexpr int k1 = KIND == SAGE_KV_INT8 ? 2 : 1, k2 = 3 - k1;  // (as pairs() gives the codes)
        qf[t][s][0] = h2bits(__floats2half2_rn(x[s][0] * up, x[s][k1] * up));
        qf[t][s][1] = h2bits(__floats2half2_rn(x[s][k2] * up, x[s][3] * up));
      }
      const float a = p.alpha * down;
      // (a row that is not there holds q = 0 and masks nothing; it is not stored)
      const int end = live ? row_end(p, u.len, q_len, i) : u.len;
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

#pragma unroll 1
    for (int k = chunks_of(u), ch = u.c0 + warp; k > 0; --k, ch += kWarps) {
      issue();
      if (!mbar_wait_warp(&bars[warp][here], phase, &abort)) break;
      __syncwarp();  // (meta)
      --flight;
      const uint8_t* src = my_ring + here * Ring<D, RT>::kBytes;
      float4 sc[kSub];
#pragma unroll
      for (int h = 0; h < kSub; ++h) sc[h] = meta[warp][here][h];
      if (++here == kPlaces) here = 0, phase ^= 1;
      // S^T
      float s[kSub][RT][4];
#pragma unroll
      for (int h = 0; h < kSub; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) s[h][t][0] = s[h][t][1] = s[h][t][2] = s[h][t][3] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
#pragma unroll
        for (int h = 0; h < kSub; ++h) {
          const uint4 ka = *reinterpret_cast<const uint4*>(src + h * 16 * D + (at_k ^ x * 64));
          const uint4 kb = *reinterpret_cast<const uint4*>(src + h * 16 * D + (at_k ^ x * 64) + 8 * D);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            pairs<KIND>(wa[w], a0, a2);
            pairs<KIND>(wb[w], a1, a3);
#pragma unroll
            for (int t = 0; t < RT; ++t)
              mma16816(s[h][t], a0, a1, a2, a3, qf[t][x * 4 + w][0], qf[t][x * 4 + w][1]);
          }
        }
      }
      // softmax of the lane's tokens tk, tk + 8 of each row tile in rows 2 tig, 2 tig + 1
      bool edge = (ch + 1) * kChunk > lim_min;
#pragma unroll
      for (int h = 0; h < kSub; ++h) edge |= kNan && sc[h].y == -INFINITY;
      bool raise = false;
      float mx[RT][2];
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[t][e] = -INFINITY;
#pragma unroll
          for (int h = 0; h < kSub; ++h) {
            const float f = ar[t][e] * sc[h].x;
            s[h][t][e] = fmaf(s[h][t][e], f, sc[h].y);
            s[h][t][2 + e] = fmaf(s[h][t][2 + e], f, sc[h].y);
            if (edge) {
              const int j = ch * kChunk + h * 16 + tk;
              if (j >= lim[t][e] || (kNan && sc[h].y == -INFINITY)) s[h][t][e] = -INFINITY;
              if (j + 8 >= lim[t][e] || (kNan && sc[h].y == -INFINITY)) s[h][t][2 + e] = -INFINITY;
            }
            mx[t][e] = max3(mx[t][e], s[h][t][e], s[h][t][2 + e]);
          }
          raise |= mx[t][e] > raise_past(m[t][e]);
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[t][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float to = x > raise_past(m[t][e]) ? x - kBelow : m[t][e];
            corr[e] = to == m[t][e] ? 1.f : ex2(m[t][e] - to);
            m[t][e] = to;
            l[t][e] *= corr[e];
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[t][j][e] *= corr[e & 1];
        }
      }
      uint32_t pb[kSub][RT][2];
#pragma unroll
      for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float sub = m[t][e] == -INFINITY ? 0.f : m[t][e];
#pragma unroll
          for (int h = 0; h < kSub; ++h) {
            s[h][t][e] = ex2(s[h][t][e] - sub);
            s[h][t][2 + e] = ex2(s[h][t][2 + e] - sub);
            l[t][e] = fmaf(s[h][t][e] + s[h][t][2 + e], sc[h].z, l[t][e]);
          }
        }
#pragma unroll
        for (int h = 0; h < kSub; ++h) {
          pb[h][t][0] = movmatrix(h2bits(__floats2half2_rn(s[h][t][0], s[h][t][1])));
          pb[h][t][1] = movmatrix(h2bits(__floats2half2_rn(s[h][t][2], s[h][t][3])));
        }
      }
      // O^T: the lane's tokens (pair 0) and those + 8 (pair 1); of the bytes 4 w + 0..3 of the
      // lane's channels g VB .., tile 2 w takes 0 and 1, tile 2 w + 1 takes 2 and 3
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        const uint8_t* vsrc = src + (kChunk + h * 16) * D;
        uint32_t v[4][VB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* y = vsrc + (i & 1 ? at_v1 : at_v0) + (i >> 1) * 8 * D;
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(y);
            v[i][0] = x.x, v[i][1] = x.y, v[i][VB / 4 - 2] = x.z, v[i][VB / 4 - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(y);
            v[i][0] = x.x, v[i][1] = x.y;
          }
        }
        if (kNan && edge) {  // what lies behind the keys may be anything, NaN among it: 0 x NaN must not enter
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = ch * kChunk + h * 16 + (i & 1 ? tv : 2 * tig) + (i >> 1) * 8;
            if (j >= u.len || sc[h].y == -INFINITY) {
#pragma unroll
              for (int w = 0; w < VB / 4; ++w) v[i][w] = 0u;
            }
          }
        }
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
          uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
          // the lane's two tokens at channels 4 w, 4 w + 1, then 4 w + 2, 4 w + 3
          constexpr uint32_t k01 = KIND == SAGE_KV_INT8 ? 0x5410 : 0x5140, k23 = KIND == SAGE_KV_INT8 ? 0x7632 : 0x7362;
          pairs<KIND>(__byte_perm(v[0][w], v[1][w], k01), a0, a1);
          pairs<KIND>(__byte_perm(v[2][w], v[3][w], k01), a2, a3);
          pairs<KIND>(__byte_perm(v[0][w], v[1][w], k23), b0, b1);
          pairs<KIND>(__byte_perm(v[2][w], v[3][w], k23), b2, b3);
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            mma16816(acc[t][2 * w], a0, a1, a2, a3, pb[h][t][0], pb[h][t][1]);
            mma16816(acc[t][2 * w + 1], b0, b1, b2, b3, pb[h][t][0], pb[h][t][1]);
          }
        }
      }
    }

    // ---- the warps' results of this part, through the ring place that each warp has just left (the
    // copies into the others go on).  16-byte unit x of row r lies at x ^ (r / 2 % 4), against bank
    // conflicts.
    const bool whole = u.c0 == 0 && u.c1 == u.chunks, any = u.c1 > u.c0;
    float* part = p.part + (size_t)(2 * w0 + (u.c0 == 0 ? 1 : 0)) * R * (D + 2);
    const int left_at = here == 0 ? kPlaces - 1 : here - 1;
    float4* mine = reinterpret_cast<float4*>(my_ring + left_at * Ring<D, RT>::kBytes);
    if (lane == 0) left_place[warp] = left_at;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float s = l[t][e];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int r = t * 8 + 2 * tig + e;
        if (g == 0) xm[warp][r] = m[t][e], xl[warp][r] = s;
#pragma unroll
        for (int j = 0; j < NJ; j += 2)
          mine[r * (D / 4) + ((g * (VB / 4) + j / 2) ^ (r >> 1 & 3))] =
              make_float4(acc[t][j][e], acc[t][j][2 + e], acc[t][j + 1][e], acc[t][j + 1][2 + e]);
      }
    __syncthreads();
    for (int x = tid; x < R * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = x % (D / 4);
      const int rw = u.tile * R + r, i = rw / p.G;
      if (!any || i >= q_len) continue;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, xm[w][r]);
      const float sub = mt == -INFINITY ? 0.f : mt;
      float ls = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(xm[w][r] - sub);
        ls = fmaf(f, xl[w][r], ls);
        const float4 y = reinterpret_cast<const float4*>(ring + w * Ring<D, RT>::kWarpBytes +
                                                         left_place[w] * Ring<D, RT>::kBytes)[r * (D / 4) + (d ^ (r >> 1 & 3))];
        o[0] = fmaf(f, y.x, o[0]), o[1] = fmaf(f, y.y, o[1]), o[2] = fmaf(f, y.z, o[2]), o[3] = fmaf(f, y.w, o[3]);
      }
      if (whole) {
        const float inv = ls != 0.f ? 1.f / ls : 0.f;
        const size_t orow = ((size_t)b * p.H + (size_t)u.hk * p.G + rw % p.G) * p.Nq + i;
        uint2 out;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&out);
        h[0] = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
        h[1] = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(p.O + orow * D + d * 4) = out;
        if (d == 0) p.LSE[orow] = ls != 0.f ? (mt + log2f(ls)) * 0.69314718055994531f : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(part + r * D + d * 4) = make_float4(o[0], o[1], o[2], o[3]);
        if (d == 0) part[R * D + r] = mt, part[R * D + R + r] = ls;
      }
    }
    fence_proxy_async_smem();  // the places are read before they are filled again
    cp_wait<0>();
    if (__syncthreads_or(abort) || u.next >= stop || after.c1 == 0) break;
    u = after;
  }
  if (abort) {  // a wait ran out: the copies that are still in flight
    if (tid == 0) atomicMax(c.status, (int)kDevTimeout);
    for (; flight > 0; --flight) {
      int give_up = 0;
      mbar_wait(&bars[warp][here], phase, &give_up);
      if (++here == kPlaces) here = 0, phase ^= 1;
    }
  }
}

// Joins the parts of the units that were cut, in their order: one CTA for each (unit, row), a quarter of
// the parts to each warp (few units, which may have many parts).
template <int D>
__global__ void __launch_bounds__(128) kv_join_kernel(const AttnParams p, int R) {
  constexpr int E = D / 32;  // channels of a lane
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = blockIdx.x;
  const int r = blockIdx.y;
  const int per_b = p.c.Hkv * p.tiles, b = (int)(unit / per_b), in_b = (int)(unit % per_b);
  const int hk = in_b % p.c.Hkv, row = in_b / p.c.Hkv * R + r, i = row / p.G;
  if (i >= row_queries(p, b)) return;
  const int2 w = p.info[unit];
  if (!was_cut(p, w)) return;
  const size_t stride = (size_t)R * (D + 2);
  auto part_of = [&](int k) { return p.part + (size_t)(k == w.x ? 2 * k + 1 : 2 * k) * stride; };
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int k0 = w.x + warp; k0 <= w.y; k0 += 16) {
    // four parts at a time, their loads in flight together
    float mm[4], ll[4], oo[4][E];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = k0 + 4 * q;
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
  p.O[orow * D + d] = __float2bfloat16_rn(ls != 0.f ? x / ls : 0.f);
  if (d == 0) p.LSE[orow] = ls != 0.f ? (mt + log2f(ls)) * 0.69314718055994531f : -INFINITY;
}

// The same for many units: a warp takes JR rows of a unit, PF parts at a time.
template <int D, int JR>
__global__ void __launch_bounds__(128) kv_join_rows_kernel(const AttnParams p, int R) {
  constexpr int E = D / 32;           // channels of a lane, side by side
  constexpr int PF = JR == 1 ? 4 : 2;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = blockIdx.x;
  const int r0 = (blockIdx.y * (blockDim.x >> 5) + warp) * JR;  // (R is a multiple of JR)
  const int per_b = p.c.Hkv * p.tiles, b = (int)(unit / per_b), in_b = (int)(unit % per_b);
  const int hk = in_b % p.c.Hkv, row0 = in_b / p.c.Hkv * R + r0, q_len = row_queries(p, b);
  if (row0 / p.G >= q_len) return;
  const int2 w = p.info[unit];
  if (!was_cut(p, w)) return;
  const size_t stride = (size_t)R * (D + 2);
  float m[JR], l[JR], o[JR][E];
#pragma unroll
  for (int x = 0; x < JR; ++x) {
    m[x] = -INFINITY, l[x] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[x][e] = 0.f;
  }
  for (int k0 = w.x; k0 <= w.y; k0 += PF) {
    float mm[PF][JR], ll[PF][JR], oo[PF][JR][E];
    // (a row that is not there: whatever the workspace holds, and not stored)
#pragma unroll
    for (int q = 0; q < PF; ++q) {
      const int k = k0 + q;
      const float* s = p.part + (size_t)(k == w.x ? 2 * k + 1 : 2 * k) * stride;
#pragma unroll
      for (int x = 0; x < JR; ++x) {
        mm[q][x] = -INFINITY, ll[q][x] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) oo[q][x][e] = 0.f;
        if (k > w.y) continue;
        const int r = r0 + x;
        mm[q][x] = s[R * D + r], ll[q][x] = s[R * D + R + r];
        if (D == 128) {
          const float4 y = *reinterpret_cast<const float4*>(s + r * D + lane * 4);
          oo[q][x][0] = y.x, oo[q][x][1] = y.y, oo[q][x][E - 2] = y.z, oo[q][x][E - 1] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(s + r * D + lane * 2);
          oo[q][x][0] = y.x, oo[q][x][1] = y.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < JR; ++x) {
      float mn = m[x];
#pragma unroll
      for (int q = 0; q < PF; ++q) mn = fmaxf(mn, mm[q][x]);
      const float sub = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2(m[x] - sub);
      l[x] *= f0;
#pragma unroll
      for (int e = 0; e < E; ++e) o[x][e] *= f0;
#pragma unroll
      for (int q = 0; q < PF; ++q) {
        const float f = ex2(mm[q][x] - sub);
        l[x] = fmaf(f, ll[q][x], l[x]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[x][e] = fmaf(f, oo[q][x][e], o[x][e]);
      }
      m[x] = mn;
    }
  }
#pragma unroll
  for (int x = 0; x < JR; ++x) {
    const int row = row0 + x, i = row / p.G;
    if (i >= q_len) return;
    const size_t orow = ((size_t)b * p.H + (size_t)hk * p.G + row % p.G) * p.Nq + i;
    const float inv = l[x] != 0.f ? 1.f / l[x] : 0.f;
    uint32_t y[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(o[x][e] * inv, o[x][e + 1] * inv);
      y[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (D == 128)
      *reinterpret_cast<uint2*>(p.O + orow * D + lane * 4) = make_uint2(y[0], y[E / 2 - 1]);
    else
      *reinterpret_cast<uint32_t*>(p.O + orow * D + lane * 2) = y[0];
    if (lane == 0) p.LSE[orow] = l[x] != 0.f ? (m[x] + log2f(l[x])) * 0.69314718055994531f : -INFINITY;
  }
}

// As many CTAs as run at once, fewer where the line cannot be long enough for them.
void few_grid(AttnParams& p, int ctas) {
  const long long units = (long long)p.B * p.c.Hkv * p.tiles;
  const long long chunks = units * (((long long)p.c.max_pages * p.c.page + kChunk - 1) / kChunk);
  const long long need = (chunks + kWarps - 1) / kWarps > units ? (chunks + kWarps - 1) / kWarps : units;
  p.most_parts = ctas < kMaxParts ? ctas : kMaxParts;
  if (need < p.most_parts) p.most_parts = (int)need;
}

template <int D, int KIND, int RT>
int launch_few(AttnParams p, int sms, cudaStream_t st) {
  few_grid(p, sms * kCtasPerSm<D, RT>);
  auto kern = kv_attn_kernel<D, KIND, RT>;
  // a page's rows [head, token]: boxes of a chunk's tokens
  const int box = p.c.page < kChunk ? p.c.page : kChunk;
  const CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tk, tv;
  if (!make_tmap_3d(&tk, p.c.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, (uint64_t)p.c.Hkv * p.c.page, p.c.n_pages, D,
                    box, swizzle) ||
      !make_tmap_3d(&tv, p.c.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, (uint64_t)p.c.Hkv * p.c.page, p.c.n_pages, D,
                    box, swizzle))
    return 3;
  // The kernel's limit is the process's: always the same one, for the most batch rows, or a call of another
  // thread could lower it before this launch.
  // (16 bytes for each batch row: at D = 128 two CTAs of the grid share an SM up to 701 rows at 8 query rows, 445 at
  // 16; beyond, the line goes over the GPU in two turns.)
  const size_t ring = 1024 + (size_t)kWarps * Ring<D, RT>::kWarpBytes, most = ring + ((size_t)kKvMaxBatch + 1) * 16;
  const size_t smem = ring + ((size_t)p.B + 1) * 16;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) return 3;
  return launch_pdl(kern, dim3(p.most_parts), dim3(kThreads), smem, st, p, tk, tv) == cudaSuccess ? 0 : 3;
}
template <int D, int KIND>
int launch_few(const AttnParams& p, int rows, int sms, cudaStream_t st) {
  return rows == 8 ? launch_few<D, KIND, 1>(p, sms, st) : launch_few<D, KIND, 2>(p, sms, st);
}

// Query rows of a unit: 8 where all rows of a shared head fit in one, 16 up to kFewRows rows, then the
// tensor-core kernel's 256.  16 sequences of 900 to 16k tokens, 4 query heads to each of 8, D = 128, this
// kernel against that one: 16 rows 62 us against 130 us, 32 rows 112 against 130, 48 rows 162 against 129;
// D = 64: 32 rows 77 against 94, 48 rows 110 against 95.
constexpr long long kFewRows = 32;
// The join takes a CTA for each row below so many units (each may be cut into many parts: 16 units with 16
// rows 12.1 us in all against 12.9 us), a warp for each row from there (64 units 11.0 us against 12.0 us, 512
// units 15.0 us against 15.7 us).
constexpr unsigned kFewUnits = 64;
// Of many query rows a warp takes four at once from so many units (2048 queries of 32 heads over 8: on 4096 keys
// 161 us against 167 us, on 32k 900 us against 910 us); with fewer units and more parts that is too few
// warps (16 units of 210 queries: 44 us against 26 us).
constexpr unsigned kManyUnits = 128;

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
  const size_t workers = L.rows == kChunkRows ? kMaxChunkParts : kMaxParts;
  L.total = L.part + workers * 2 * L.rows * (D + 2) * 4;
  return L;
}

namespace {

// what the kernels of a call share (scales and sizes of the queries left to the caller)
AttnParams attn_params(const sage_kv_cache& c, const KvAttnWs& L, const int* q_len, void* O, float* LSE, void* ws, int B,
                       int H, int Nq) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnParams p{};
  p.c = c;
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
  p.most_parts = L.rows == kChunkRows ? kMaxChunkParts : kMaxParts;
  return p;
}

int launch_join(const AttnParams& p, int R, cudaStream_t st) {
  const bool many = R == kChunkRows;
  const long long rows = (long long)p.G * p.Nq;
  const unsigned unit_rows = (unsigned)(rows < R ? rows : R);
  const unsigned units = (unsigned)((long long)p.B * p.c.Hkv * p.tiles);
  auto join = p.c.D == 128 ? kv_join_kernel<128> : kv_join_kernel<64>;
  dim3 join_grid(units, unit_rows), join_block(128);
  if (many || units >= kFewUnits) {
    const int rows_each = many && units >= kManyUnits ? 4 : 1;
    join = rows_each == 4 ? (p.c.D == 128 ? kv_join_rows_kernel<128, 4> : kv_join_rows_kernel<64, 4>)
                          : (p.c.D == 128 ? kv_join_rows_kernel<128, 1> : kv_join_rows_kernel<64, 1>);
    const unsigned turns = (unit_rows + rows_each - 1) / rows_each, warps = turns < 4 ? turns : 4;
    join_grid.y = (turns + warps - 1) / warps, join_block.x = 32 * warps;
  }
  if (launch_pdl(join, join_grid, join_block, 0, st, p, R) != cudaSuccess) return 3;
  return cudaGetLastError() == cudaSuccess ? 0 : 3;
}

}  // namespace

int launch_kv_attention(const sage_kv_cache& c, const void* Q, const int* slots, const int* q_len, void* O,
                        float* LSE, void* ws, int B, int H, int Nq, int causal, float sm_scale, cudaStream_t st) {
  const KvAttnWs L = kv_attn_ws_layout(B, H, c.Hkv, c.D, Nq);
  AttnParams p = attn_params(c, L, q_len, O, LSE, ws, B, H, Nq);
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.slots = slots;
  p.causal = causal;
  p.alpha = (float)((double)sm_scale * 1.4426950408889634074);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 3;
  ScopedTimer timer("kv_attention", st);
  if (int rc = L.rows == kChunkRows ? launch_kv_chunk(p, c.kind, sms, st) : launch_kv_few(p, c.kind, L.rows, sms, st))
    return rc;
  return launch_join(p, L.rows, st);
}

int launch_kv_join(const sage_kv_cache& c, void* O, float* LSE, void* ws, int B, int H, int Nq, cudaStream_t st) {
  const KvAttnWs L = kv_attn_ws_layout(B, H, c.Hkv, c.D, Nq);
  return launch_join(attn_params(c, L, nullptr, O, LSE, ws, B, H, Nq), L.rows, st);
}

}  // namespace sage
