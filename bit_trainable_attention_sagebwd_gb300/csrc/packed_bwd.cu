// Attention over packed sequences, backward (sage_attn_packed_bwd).  With P = e^(S - LSE) recomputed and
// delta_i = sum_d dO_id O_id:
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = sm_scale dS K,  dK = sm_scale dS^T Q.
// Three kernels:
//   packed_pre   -LSE log2 e and -delta of every query row
//   packed_dkv   a 128-key tile against the row tiles that see it: dK and dV
//   packed_dq    a row tile against the key tiles that it sees: dQ
// dQ in a kernel of its own recomputes S and dP, seven products in place of five.  In exchange nothing is added up in
// memory: no fp32 sums of dQ go to L2 for every tile (64 KB beside 160 KB of operands from shared memory, which already
// set the pace), none are cleared and converted, and the gradients are the same bits every time.
//
// The two main kernels are alike.  One CTA an SM walks its units (packed.cuh):
//  - warp 19 walks, warp 17 brings the operands by TMA;
//  - warps 16 and 18 issue the products (bf16 operands, fp32 accumulators in TMEM): one alone spends more time on its
//    waits than the products leave it;
//  - warps 0-15 turn S into P and dP into dS, each group of four 32 of the tile's columns; P and dS go back to TMEM as
//    bf16 over the columns that they come from and are the A operands of the products that take them.
// While the warps compute, the products of the tile before and after run: P(i) lets dV(i) and S(i + 1) in, dS(i) lets
// dK(i) and dP(i + 1) in.
// Rows that belong to the next sequence: those that a product would sum over are zeroed in shared memory (up to 15 of a
// tile; the product stops there), the others end in rows that are not stored.
//
// 8192 tokens, 32 heads of 8, D = 128, causal: 1.34 ms, 1.02 PFLOP/s of the five products' operations (1.43 of the seven's
// that run, 75% of what a bf16 product reaches here in a burst): 0.72 ms dK and dV, 0.59 ms dQ, 0.03 ms the row terms, each
// alone.  Repeated for seconds, under the power limit: 1.45 ms, 0.95 PFLOP/s (1.33 of the seven's, 76% of what one reaches
// then).
// What bounds it: shared memory's bandwidth and the tensor core (70% and 66% active) with the chain between the products.
#include "issue.cuh"
#include "launch.h"
#include "packed.cuh"
#include "timer.h"

namespace sage {

namespace {

constexpr int kWorkWarps = 16, kWarps = kWorkWarps + 4, kThreads = 32 * kWarps;  // (five a scheduler: 96 registers a thread)
constexpr int kIssuer = 16, kLoader = 17, kSecond = 18, kWalker = 19;  // kSecond: the second issuer
constexpr uint32_t kCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  PackedShape s;
  const float *nlse, *ndelta;  // [Hkv][T][G]: -LSE log2 e, -delta (packed_dq)
  const uint4* more;           // [Hkv][T][G]: the same as further channels of Q and dO (packed_dkv)
  sage_rows dout;              // packed_dq
  sage_rows d0, d1;            // packed_dkv: dK, dV; packed_dq: dQ
  float* part;                 // of each worker two places: [D / 4][128] sums of four channels of d0, and of d1
  float alpha, sm_scale;       // alpha: sm_scale log2 e
};

// ------------------------------------------------------------------ row statistics
struct PreParams {
  PackedShape s;
  sage_rows O, dO;
  const float* LSE;
  float *nlse, *ndelta;
  uint4* more;
  float sm_scale;
  unsigned long long inv_h, inv_g;  // 2^64 / H and / G, rounded up
};

// The row terms in the products.  packed_dkv has the query rows along the columns, so a row's LSE and delta are another
// number in every register of a thread; read from shared memory by 16 warps they took half of the time (the tensor core
// takes all of its bandwidth).  Instead they are channels: Q gets -LSE / sm_scale and dO -delta, each as three bf16 whose
// sum has 24 bits, K and V ones; one more step along K, and S sm_scale - LSE and dP - delta are there.
constexpr float kNever = -3e38f;  // in the place of -LSE / sm_scale: P = 0
__device__ __forceinline__ uint32_t bf16_of(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ void split3(float x, uint32_t (&b)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    b[k] = bf16_of(x);
    x -= __uint_as_float(b[k] << 16);
    if (!(fabsf(x) < INFINITY)) x = 0.f;  // (an infinity or a NaN is all in the first)
  }
}
// channels 0-2 of LSE, 3-5 of delta
__device__ __forceinline__ uint4 more_channels(float l, float d) {
  uint32_t a[3], b[3];
  split3(l, a);
  split3(d, b);
  return make_uint4(a[0] | a[1] << 16, a[2] | b[0] << 16, b[1] | b[2] << 16, 0u);
}

// n / d by the quotient's upper half: inv = 2^64 / d rounded up, exact for n d < 2^64
__device__ __forceinline__ unsigned over(unsigned long long n, unsigned d, unsigned long long inv) {
  return d > 1 ? (unsigned)__umul64hi(n, inv) : (unsigned)n;
}

// D / 8 lanes a row, rows in the order of [T, H].  It should be bound by DRAM (O and dO once) and was by its instructions:
// hence divisions that are products, and terms that a lane each makes for the four rows of a thread, not one lane for
// all (every lane issues what one does).  8892 tokens of 16 heads: the whole backward 194 us against 201 us.
template <int D>
__global__ void __launch_bounds__(256) packed_pre_kernel(const PreParams p) {
  constexpr int kLanes = D / 8, kRows = 4, kStep = 256 / kLanes;  // rows of a thread, and between them
  const int tid = threadIdx.x, lane = tid % kLanes;
  const unsigned H = p.s.Hkv * p.s.G;
  const unsigned long long r0 = (unsigned long long)blockIdx.x * (kStep * kRows);
  const unsigned t0 = over(r0, H, p.inv_h), h0 = (unsigned)(r0 - (unsigned long long)t0 * H);  // the block's first row
  pdl_wait();
  pdl_trigger();
  auto row = [&](int x, unsigned& t, unsigned& h) {
    const unsigned n = h0 + x * kStep + tid / kLanes, more = over(n, H, p.inv_h);
    t = t0 + more, h = n - more * H;
    return t < (unsigned)p.s.T;
  };
  uint4 a[kRows], b[kRows];
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    unsigned t, h;
    a[x] = b[x] = make_uint4(0u, 0u, 0u, 0u);
    if (row(x, t, h)) {
      auto piece = [&](const sage_rows& y) {
        return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(y.p) + t * y.token + h * y.head) + lane);
      };
      a[x] = piece(p.O), b[x] = piece(p.dO);
    }
  }
  float delta = 0.f;  // of the lane's row
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    float s = 0.f;
    const uint32_t u[4] = {a[x].x, a[x].y, a[x].z, a[x].w}, v[4] = {b[x].x, b[x].y, b[x].z, b[x].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(v[e] << 16), s);
      s = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(v[e] & 0xffff0000u), s);
    }
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == x) delta = s;
  }
  unsigned t, h;
  if (lane < kRows && row(lane, t, h)) {
    const unsigned hk = over(h, p.s.G, p.inv_g);
    const size_t at = ((size_t)hk * p.s.T + t) * p.s.G + (h - hk * p.s.G);
    const float lse = p.LSE[(size_t)h * p.s.T + t];
    p.nlse[at] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;  // (a row that saw nothing: P = 0)
    p.ndelta[at] = -delta;
    p.more[at] = more_channels(lse == -INFINITY ? kNever : -lse / p.sm_scale, -delta);
  }
}

// ------------------------------------------------------------------ shared memory
template <int D, int XS, int YS>
struct BwdSmem {
  uint8_t x[XS][kTile * D * 2];  // what the unit walks over: Q, or K
  uint8_t y[YS][kTile * D * 2];  // dO, or V
  uint8_t a[XS == 2 ? 2 : 1][kTile * D * 2];  // the unit's own tiles: packed_dkv K and V, packed_dq Q
  // packed_dkv: the further channels of the tiles walked over, and ones in the places of LSE's and of delta's; 16 channels
  // unswizzled, the first eight of 128 rows, then the others (zeros)
  __align__(128) uint8_t more[XS == 2 ? 2 : 1][XS == 2 ? kTile * 32 : 16];
  __align__(128) uint8_t ones[2][XS == 2 ? kTile * 32 : 16];
  __align__(128) uint4 low[XS == 2 ? 1 : 4 * kTile];  // packed_dq: the second halves of dS (see there), [group][row]
  uint64_t bar_a_full[2], bar_a_empty[2], bar_x_full[XS], bar_x_empty[XS], bar_y_full[YS], bar_y_empty[YS], bar_raw;
  uint64_t bar_s[2], bar_dp, bar_p, bar_ds, bar_acc, bar_acc_read, bar_s_read, bar_dp_read, bar_ds_free;
  FeedRing ring;
  Meeting meeting;
  long long wsum[kWarps];
  long long pre[kPackedGroups + 1];
  unsigned long long tokens;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(BwdSmem<128, 2, 2>) + 1024 <= 227 * 1024 && sizeof(BwdSmem<128, 3, 2>) + 1024 <= 227 * 1024,
              "shared memory of a CTA");

template <int D, int XS, int YS>
__device__ __forceinline__ void init_barriers(BwdSmem<D, XS, YS>& sm, int readers) {
  for (int t = 0; t < 2; ++t) {
    mbar_init(&sm.bar_a_full[t], XS == 3 && t == 1 ? kWorkWarps : 1);  // (packed_dq's dO comes through the work warps)
    mbar_init(&sm.bar_a_empty[t], 1);
    mbar_init(&sm.bar_s[t], 1);
  }
  mbar_init(&sm.bar_raw, 1);
  for (int t = 0; t < XS; ++t) {
    mbar_init(&sm.bar_x_full[t], 1);
    mbar_init(&sm.bar_x_empty[t], 1);
  }
  for (int t = 0; t < YS; ++t) {
    mbar_init(&sm.bar_y_full[t], 1);
    mbar_init(&sm.bar_y_empty[t], XS == 2 ? 2 : 1);  // (packed_dkv: dV and dP have dO)
  }
  sm.ring.init(readers);
  sm.meeting.init(kWorkWarps);
  mbar_init(&sm.bar_dp, 1);
  mbar_init(&sm.bar_p, kWorkWarps);
  mbar_init(&sm.bar_ds, kWorkWarps);
  mbar_init(&sm.bar_acc, XS == 2 ? 2 : 1);  // (packed_dkv: dV and dK)
  mbar_init(&sm.bar_acc_read, kWorkWarps);
  mbar_init(&sm.bar_s_read, kWorkWarps);
  mbar_init(&sm.bar_dp_read, kWorkWarps);
  mbar_init(&sm.bar_ds_free, 1);
  sm.abort = 0;
  sm.tokens = 0;
  fence_mbar_init();
}

// A place in a ring of N: how often it has come round, and where it stands
template <int N>
struct Turn {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, ++round;
  }
};

// rows [from, to) of a tile in shared memory become zero (a warp)
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to) {
  constexpr int kPieces = D / 8;  // of 16 bytes
  for (int e = threadIdx.x & 31; e < (to - from) * kPieces; e += 32) {
    const int row = from + e / kPieces, c = e % kPieces;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (kTile * 128) + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// One tile by TMA (a warp; lane 0 issues): `load` issues the copies onto the barrier that it gets.  Of a tile with
// `rows` rows of its own, fewer than the copy brings, those up to the next multiple of 16 are zeroed (and `fill`ed) before
// `full` is signalled.
template <int D, class Load, class Fill>
__device__ __forceinline__ bool bring(uint8_t* tile, int rows, int copied, uint32_t bytes, uint64_t* full, uint64_t* raw,
                                      uint32_t& raws, volatile int* abort, Load&& load, Fill&& fill) {
  const int lane = threadIdx.x & 31;
  const bool ragged = rows < copied && (rows & 15);
  uint64_t* bar = ragged ? raw : full;
  if (lane == 0) {
    mbar_arrive_expect_tx(bar, bytes);
    load(bar);
  }
  __syncwarp();
  if (!ragged) return true;
  int give_up = 0;
  if (!__all_sync(0xffffffffu, mbar_wait(raw, raws++ & 1, &give_up))) {
    *abort = 1;
    return false;
  }
  zero_rows<D>(tile, rows, (rows + 15) & ~15);
  fill(rows, (rows + 15) & ~15);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(full);
  return true;
}

// One tile of the parts after another.  `first`, `last`: of a part.
struct Tiles {
  Feed feed;
  Part s{};
  int j = 0;
  bool first = false, last = true;
  __device__ __forceinline__ Tiles(FeedRing& ring, volatile int* abort) : feed(ring, abort) {}
  // false: there are no more
  __device__ __forceinline__ bool next() {
    first = last;
    if (!last) {
      ++j;
    } else {
      if (!feed.next(s)) return false;
      j = s.c0;
    }
    last = j + 1 == s.c1;
    return true;
  }
};

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// columns of an A operand in TMEM, 16 bf16 each: P or dS as the four groups write them
__device__ __forceinline__ uint32_t a_col(int k) { return 32 * (k >> 1) + 8 * (k & 1); }

// D (+)= A B over `rows` rows of B, 16 at a time
__device__ __forceinline__ void issue_rows(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int rows, bool acc) {
  if (rows > kTile - 16) {
    issue_ts_x4_pairs(d, a, b, idesc, acc);
    issue_ts_x4_pairs(d, a + 64, b + (4 * 2048 >> 4), idesc, 1);
  } else {
#pragma unroll 1
    for (int k = 0; k * 16 < rows; ++k) issue_ts(d, a + a_col(k), b + (k * 2048 >> 4), idesc, acc || k > 0);
  }
}

// ------------------------------------------------------------------ dK and dV
// TMEM: S^T (keys x query rows), then P^T, at 0; dP^T, then dS^T, at 128; dV at 256; dK at 384
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dkv_kernel(const BwdParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do) {
  constexpr int kAtoms = D / 64, kAtom = kTile * 128;
  constexpr uint32_t cS = 0, cDP = 128, cDV = 256, cDK = 384;
  extern __shared__ uint8_t smem_raw[];
  using Smem = BwdSmem<D, 2, 2>;
  Smem& sm = *reinterpret_cast<Smem*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int box = p.s.G * p.s.w;  // rows of a row tile
  if (tid == 0) init_barriers(sm, kWorkWarps + 3);
  if (warp < 4 && box < kTile) zero_rows<D>(warp < 2 ? sm.x[warp] : sm.y[warp - 2], box, kTile);  // the rows that no copy brings
  for (int e = tid; e < 4 * kTile; e += kThreads) {
    // the further channels: P = 0 in rows that no copy brings; ones
    const int what = e / kTile, r = e % kTile;
    uint4* to = reinterpret_cast<uint4*>(what < 2 ? sm.more[what] : sm.ones[what - 2]);
    to[r] = what < 2    ? more_channels(kNever, 0.f)
            : what == 2 ? make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u)
                        : make_uint4(0u, 0x3f800000u, 0x3f803f80u, 0u);
    to[kTile + r] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  pdl_wait();
  if (blockIdx.x == 0 && tid == kThreads - 1) pdl_tell(p.s.status + kTermsTold);
  if (warp == kIssuer) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  const int group = ceil_div(p.s.S, kPackedGroups);
  prefix_of_sequences<kKeys, kThreads>(p.s, group, sm.pre, sm.wsum, &sm.tokens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const Shares line(sm.pre[kPackedGroups], gridDim.x);
  const bool idle = line.total == 0 || too_many(p.s, sm.tokens) || (int)blockIdx.x >= line.parts;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, abort); };
  // the row tile at hand: the sequence's tile, and its rows
  auto tile_of = [&](const Tiles& t) { return Units<kKeys>(p.s, t.s.len).first(t.s.i) + t.j; };
  auto rows_of = [&](const Tiles& t, int rt) { return min(p.s.w, t.s.len - rt * p.s.w) * p.s.G; };

  if (warp >= kWorkWarps) {
    constexpr uint32_t id_s = idesc_bf16(kTile, kTile, false, false), id_g = idesc_bf16(kTile, D, false, true);
    constexpr uint64_t kNext = (uint64_t)kTile * D * 2 >> 4, kAtomStep = kAtom >> 4, kMore = kTile * 32 >> 4;
    if (warp == kIssuer || warp == kSecond) {
      // ---------------- MMA issuers: the first dV of a tile and S of the next one, the second dK and dP of the next one
      const int v = warp == kSecond;
      const uint64_t own_k = sdesc_sw128(smem_u32(sm.a[v]), 16, 1024);                              // K, or V
      const uint64_t walked_k = sdesc_sw128(smem_u32(v ? sm.y[0] : sm.x[0]), 16, 1024);             // Q, or dO
      const uint64_t summed = sdesc_sw128(smem_u32(v ? sm.x[0] : sm.y[0]), kAtom, 1024);            // dO, or Q
      const uint64_t one_k = sdesc_none(smem_u32(sm.ones[v]), kTile * 16, 128);
      const uint64_t more_k = sdesc_none(smem_u32(sm.more[0]), kTile * 16, 128);
      uint64_t *full = v ? sm.bar_y_full : sm.bar_x_full, *given = v ? sm.bar_x_empty : sm.bar_y_empty;
      uint64_t *ready = v ? &sm.bar_dp : &sm.bar_s[0], *due = v ? &sm.bar_ds : &sm.bar_p;
      const uint32_t d_s = tmem + (v ? cDP : cS), d_g = tmem + (v ? cDK : cDV);
      bool ok = true;
      uint32_t units = 0, done = 0;
      int rows = 0;
      Tiles t(sm.ring, abort);
      // dV or dK of tile n - 1, then S or dP of tile n
#pragma unroll 1
      for (uint32_t n = 0;; ++n) {
        const bool first = t.first, last = t.last, more = t.next();
        if (n > 0) {
          if (first && done) ok = wait(&sm.bar_acc_read, (done - 1) & 1);
          if (!v) ok = ok && wait(&sm.bar_y_full[(n - 1) & 1], ((n - 1) >> 1) & 1);  // (dO, which S did not need)
          ok = ok && wait(due, (n - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_rows(d_g, d_s, summed + ((n - 1) & 1) * kNext, id_g, rows, !first);
          commit(&given[(n - 1) & 1]);
          if (last) {
            commit(&sm.bar_acc);
            ++done;
          }
        }
        if (!more) break;
        rows = rows_of(t, tile_of(t));
        if (t.first) ok = wait(&sm.bar_a_full[v], units++ & 1);
        ok = ok && wait(&full[n & 1], (n >> 1) & 1);
        if (v) ok = ok && wait(&sm.bar_x_full[n & 1], (n >> 1) & 1);  // (the further channels come with Q)
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < kAtoms; ++h)
          issue_ss_x4(d_s, own_k + h * kAtomStep, walked_k + (n & 1) * kNext + h * kAtomStep, id_s, h > 0);
        issue_ss(d_s, one_k, more_k + (n & 1) * kMore, id_s, 1);
        commit(ready);
        if (v) commit(&sm.bar_y_empty[n & 1]);
        if (t.last) commit(&sm.bar_a_empty[v]);
      }
    } else if (warp == kLoader) {
      // ---------------- K and V; dO and Q, in the order in which they are given back
      uint32_t units = 0, raws = 0, n = 0;  // (both kinds of tile: each is waited for before the next)
      bool ok = true;
      Tiles t(sm.ring, abort);
#pragma unroll 1
      for (; ok && t.next(); ++n) {
        const uint32_t st = n & 1;
        const int rt = tile_of(t), rows = rows_of(t, rt);
        // a unit's first: K, Q, V, dO; then dO, Q
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int v = t.first ? x : x ^ 1;
          if (t.first) {
            ok = ok && (units == 0 || wait(&sm.bar_a_empty[v], (units - 1) & 1));
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(&sm.bar_a_full[v], kTile * D * 2);
#pragma unroll
              for (int h = 0; h < kAtoms; ++h)
                tma_load_3d(sm.a[v] + h * kAtom, v ? &tm_v : &tm_k, h * 64, t.s.at + t.s.i * kTile, t.s.hk, &sm.bar_a_full[v]);
            }
            __syncwarp();
          }
          uint8_t* tile = v ? sm.y[st] : sm.x[st];
          ok = ok && (n < 2 || wait(v ? &sm.bar_y_empty[st] : &sm.bar_x_empty[st], ((n >> 1) - 1) & 1));
          ok = ok && bring<D>(tile, rows, box, box * D * 2 + (v ? 0 : rows * 16), v ? &sm.bar_y_full[st] : &sm.bar_x_full[st],
                              &sm.bar_raw, raws, abort,
                              [&](uint64_t* bar) {
#pragma unroll
                                for (int h = 0; h < kAtoms; ++h)
                                  tma_load_3d(tile + h * kAtom, v ? &tm_do : &tm_q, h * 64, t.s.hk * p.s.G, t.s.at + rt * p.s.w,
                                              bar);
                                if (v == 0)  // (with Q: dP of the tile before is done once Q's tile is free)
                                  bulk_load(sm.more[st], p.more + ((size_t)t.s.hk * p.s.T + t.s.at + (size_t)rt * p.s.w) * p.s.G,
                                            rows * 16, bar);
                              },
                              [&](int from, int to) {
                                if (v == 0 && from + lane < to)
                                  reinterpret_cast<uint4*>(sm.more[st])[from + lane] = more_channels(kNever, 0.f);
                              });
        }
        if (t.first) ++units;
      }
      // (copies in flight after a wait that ran out)
      int give_up = 0;
      for (int v = 0; v < 2; ++v)
        if (units) mbar_wait(&sm.bar_a_full[v], (units - 1) & 1, &give_up);
      for (uint32_t e = 0; e < 2; ++e)
        if (n > e) {
          mbar_wait(&sm.bar_x_full[(n - 1 - e) & 1], ((n - 1 - e) >> 1) & 1, &give_up);
          mbar_wait(&sm.bar_y_full[(n - 1 - e) & 1], ((n - 1 - e) >> 1) & 1, &give_up);
        }
    } else if (warp == kWalker) {
      feed<kKeys>(p.s, sm.ring, sm.pre, group, line, idle, abort);
    }
  } else {
    // ---------------- thread r of group g: key r of the tile, columns [32 g, 32 g + 32)
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + cS + 32 * g, dp_col = tmem + lanes + cDP + 32 * g;
    bool ok = true;
    uint32_t units = 0, joins = 0, n = 0;
    Feed parts(sm.ring, abort);
    Part s{};
    const uint64_t a2 = f2(p.alpha, p.alpha);
    while (ok && parts.next(s)) {
      const int key = s.i * kTile + r;
      // causal: columns of tokens before the key are masked
      int ahead = p.s.causal ? key - (Units<kKeys>(p.s, s.len).first(s.i) + s.c0) * p.s.w : 0;
#pragma unroll 1
      for (int j = s.c0; j < s.c1; ++j, ++n, ahead -= p.s.w) {
        const int mask = min(ahead, kTile) * p.s.G - 32 * g;  // the group's columns before it
        ok = wait(&sm.bar_s[0], n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(s_col, sv);
        tmem_wait32(sv);
        if (__any_sync(0xffffffffu, mask > 0)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e < mask) sv[e] = 0xff800000u;
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2split(fmul2(f2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), a2), x, y);
          x = ex2(x), y = ex2(y);
          sv[e] = __float_as_uint(x), sv[e + 1] = __float_as_uint(y);
          w[e >> 1] = bf2(x, y);
        }
        tmem_st16(s_col, w);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.bar_p);
        ok = wait(&sm.bar_dp, n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t dv[32];
        tmem_ld32(dp_col, dv);
        tmem_wait32(dv);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2split(fmul2(f2(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])),
                        f2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]))),
                  x, y);
          w[e >> 1] = bf2(x, y);
        }
        tmem_st16(dp_col, w);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.bar_ds);
      }
      // ---- the unit's sums: groups 0 and 1 half of dK's channels each, groups 2 and 3 of dV's
      ok = ok && wait(&sm.bar_acc, units++ & 1);
      if (!ok) break;
      tc_fence_after();
      const bool live = key < s.len, whole = s.whole();
      const int x = g >> 1, d0 = (g & 1) * (D / 2);
      const sage_rows& to = x ? p.d1 : p.d0;
      const RowStore out(live ? static_cast<__nv_bfloat16*>(to.p) + (long long)(s.at + key) * to.token + s.hk * to.head : nullptr);
      auto part_of = [&](int place) { return p.part + (size_t)(2 * place + x) * kTile * D; };
      const float f = x ? 1.f : p.sm_scale;
#pragma unroll 1
      for (int round = whole ? 1 : 0; round < 2; ++round) {  // a unit's part goes to memory before its sums, if it has others
#pragma unroll 1
        for (int d = d0; d < d0 + D / 2; d += 32) {
          uint32_t o[32];
          if (whole || round == 0) {
            tmem_ld32(tmem + lanes + (x ? cDV : cDK) + d, o);
            tmem_wait32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
#pragma unroll 1
            for (int k = 0; k < s.parts(); ++k) add_sums(part_of(s.place(k)), d, r, 1.f, reinterpret_cast<float(&)[32]>(o));
          }
          if (round)
            out.put(reinterpret_cast<const float(&)[32]>(o), d, f);
          else
            store_sums(part_of(s.place()), d, r, o);
        }
        if (whole || round == 0) {
          tc_fence_before();
          warp_arrive(&sm.bar_acc_read);
        }
        if (round == 0 &&
            !sm.meeting.was_last(p.s.status + kKeyCounters + 2 * s.first(), s.parts(), joins++, warp == 0, abort, ok))
          break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, kCols);
  if (tid == 0 && sm.abort) atomicMax(p.s.status, (int)kDevTimeout);
}

// ------------------------------------------------------------------ dQ
// TMEM: S (query rows x keys) at 0, dP at 128, dQ at 256; behind it dO, from where it is dP's A operand (in shared memory
// it would take 32 KB of its bandwidth for each key tile), and dS.  S and dP of the next tile go in as soon as this
// one's have been read, so the warps do not wait for them.
// dS's rounding to bf16 is most of what dQ is off by: a row of dS sums to zero, its roundings do not, so what the keys
// have in common stays in their error.  Of the first eight of every 32 keys the rounding's rest goes into dQ as well
// (`low`, a further bf16, 16 keys an MMA): a quarter of that error's square for 4% of the time, 1.29 to 1.35 ms for
// 8192 tokens.  For all keys TMEM has no columns left at D = 128; at D = 64, where 96 are free, it was not tried.  (A last tile
// of 32 keys or fewer: of the first sixteen; of 33 to 96: of the first two groups of 32.)
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_dq_kernel(const BwdParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kAtoms = D / 64, kAtom = kTile * 128;
  // (K's tile is held by dQ's product until dS is there, V's only by dP)
  constexpr int kStagesK = 3, kStagesV = 2;
  constexpr uint32_t cS = 0, cDP = 128, cDQ = 256, cDO = cDQ + D, cDS = cDO + D / 2;
  static_assert(cDS + 64 <= kCols, "TMEM");
  extern __shared__ uint8_t smem_raw[];
  using Smem = BwdSmem<D, kStagesK, kStagesV>;
  Smem& sm = *reinterpret_cast<Smem*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) init_barriers(sm, kWorkWarps + 3);
  // (packed_dkv, of which nothing is read, may still run: its CTAs let this kernel in behind their wait for packed_pre.
  // With the ordinary wait for all of packed_dkv: gradients of 4 short sequences 42.3 us, not 32.0, documents 203, not 188.)
  pdl_wait_unless(p.s.status + kTermsTold);
  if (warp == kIssuer) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  const int group = ceil_div(p.s.S, kPackedGroups);
  prefix_of_sequences<kRows, kThreads>(p.s, group, sm.pre, sm.wsum, &sm.tokens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const Shares line(sm.pre[kPackedGroups], gridDim.x);
  const bool idle = line.total == 0 || too_many(p.s, sm.tokens) || (int)blockIdx.x >= line.parts;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, abort); };

  if (warp >= kWorkWarps) {
    constexpr uint32_t id_s = idesc_bf16(kTile, kTile, false, false), id_g = idesc_bf16(kTile, D, false, true);
    constexpr uint64_t kNext = (uint64_t)kTile * D * 2 >> 4, kAtomStep = kAtom >> 4;
    if (warp == kIssuer) {
      // ---------------- MMA issuer of S and dP
      const uint64_t k_k = sdesc_sw128(smem_u32(sm.x[0]), 16, 1024), v_k = sdesc_sw128(smem_u32(sm.y[0]), 16, 1024);
      const uint64_t q_k = sdesc_sw128(smem_u32(sm.a[0]), 16, 1024);
      bool ok = true;
      Turn<kStagesK> kt;
      Turn<kStagesV> vt;
      uint32_t units = 0, n = 0;
      Tiles t(sm.ring, abort);
#pragma unroll 1
      for (; t.next(); ++n) {
        if (t.first) ok = ok && wait(&sm.bar_a_full[0], units & 1);
        ok = ok && wait(&sm.bar_x_full[kt.at], kt.round & 1);
        if (n > 0) ok = ok && wait(&sm.bar_s_read, (n - 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < kAtoms; ++h)
          issue_ss_x4(tmem + cS, q_k + h * kAtomStep, k_k + kt.at * kNext + h * kAtomStep, id_s, h > 0);
        commit(&sm.bar_s[0]);
        if (t.last) commit(&sm.bar_a_empty[0]);
        kt.next();
        if (t.first) ok = wait(&sm.bar_a_full[1], units++ & 1);
        ok = ok && wait(&sm.bar_y_full[vt.at], vt.round & 1);
        if (n > 0) ok = ok && wait(&sm.bar_dp_read, (n - 1) & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < kAtoms; ++h)
          issue_ts_x4_rows(tmem + cDP, tmem + cDO + 32 * h, v_k + vt.at * kNext + h * kAtomStep, id_s, h > 0);
        commit(&sm.bar_dp);
        commit(&sm.bar_y_empty[vt.at]);
        vt.next();
      }
    } else if (warp == kSecond) {
      // ---------------- MMA issuer of dQ
      const uint64_t k_n = sdesc_sw128(smem_u32(sm.x[0]), kAtom, 1024);
      // the low halves: eight keys each of two groups, 32 keys apart
      const uint64_t k_far = sdesc_sw128(smem_u32(sm.x[0]), kAtom, 4096), low = sdesc_none(smem_u32(sm.low), kTile * 16, 128);
      bool ok = true;
      Turn<kStagesK> kt;
      uint32_t done = 0, n = 0;
      Tiles t(sm.ring, abort);
#pragma unroll 1
      for (; t.next(); ++n) {
        if (t.first && done) ok = wait(&sm.bar_acc_read, (done - 1) & 1);
        const int keys = t.s.len - t.j * kTile;
        const uint64_t b = k_n + kt.at * kNext;
        ok = ok && wait(&sm.bar_x_full[kt.at], kt.round & 1) && wait(&sm.bar_ds, n & 1);
        if (!ok) break;
        tc_fence_after();
        if (keys > kTile - 16) {
          issue_ts_x4(tmem + cDQ, tmem + cDS, b, id_g, !t.first);
          issue_ts_x4(tmem + cDQ, tmem + cDS + 32, b + (4 * 2048 >> 4), id_g, 1);
        } else {
#pragma unroll 1
          for (int k = 0; k * 16 < keys; ++k)
            issue_ts(tmem + cDQ, tmem + cDS + 8 * k, b + (k * 2048 >> 4), id_g, k > 0 || !t.first);
        }
        // (not where a group's keys lie behind the sequence; 32 keys or fewer: the first sixteen)
#pragma unroll 1
        for (int k = 0; k == 0 || (k < 2 && keys > 64 * k + 32); ++k)
          issue_ss(tmem + cDQ, low + k * (2 * kTile * 16 >> 4), (keys > 32 ? k_far : k_n) + kt.at * kNext + k * (8 * 1024 >> 4),
                   id_g, 1);
        commit(&sm.bar_ds_free);
        commit(&sm.bar_x_empty[kt.at]);
        kt.next();
        if (t.last) {
          commit(&sm.bar_acc);
          ++done;
        }
      }
    } else if (warp == kLoader) {
      // ---------------- Q; K and V
      Turn<kStagesK> kt;
      Turn<kStagesV> vt;
      uint32_t units = 0, raws = 0;
      const int lane = tid & 31, box = p.s.G * p.s.w;
      bool ok = true;
      Tiles t(sm.ring, abort);
#pragma unroll 1
      while (ok && t.next()) {
        if (t.first) {
          ok = units == 0 || wait(&sm.bar_a_empty[0], (units - 1) & 1);
          if (!ok) break;
          ++units;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.bar_a_full[0], box * D * 2);
#pragma unroll
            for (int h = 0; h < kAtoms; ++h)
              tma_load_3d(sm.a[0] + h * kAtom, &tm_q, h * 64, t.s.hk * p.s.G, t.s.at + t.s.i * p.s.w, &sm.bar_a_full[0]);
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          const uint32_t st = v ? vt.at : kt.at, round = v ? vt.round : kt.round;
          uint8_t* tile = v ? sm.y[st] : sm.x[st];
          ok = ok && (round == 0 || wait(v ? &sm.bar_y_empty[st] : &sm.bar_x_empty[st], (round - 1) & 1));
          ok = ok && bring<D>(tile, min(kTile, t.s.len - t.j * kTile), kTile, kTile * D * 2,
                              v ? &sm.bar_y_full[st] : &sm.bar_x_full[st], &sm.bar_raw, raws, abort,
                              [&](uint64_t* bar) {
#pragma unroll
                                for (int h = 0; h < kAtoms; ++h)
                                  tma_load_3d(tile + h * kAtom, v ? &tm_v : &tm_k, h * 64, t.s.at + t.j * kTile, t.s.hk, bar);
                              },
                              [](int, int) {});
        }
        if (!ok) break;
        kt.next();
        vt.next();
      }
      // (copies in flight after a wait that ran out)
      int give_up = 0;
      if (units) mbar_wait(&sm.bar_a_full[0], (units - 1) & 1, &give_up);
      for (uint32_t e = 0; e < kStagesK; ++e)
        if (e < kt.at || kt.round > 0) mbar_wait(&sm.bar_x_full[e], (e < kt.at ? kt.round : kt.round - 1) & 1, &give_up);
      for (uint32_t e = 0; e < kStagesV; ++e)
        if (e < vt.at || vt.round > 0) mbar_wait(&sm.bar_y_full[e], (e < vt.at ? vt.round : vt.round - 1) & 1, &give_up);
    } else if (warp == kWalker) {
      feed<kRows>(p.s, sm.ring, sm.pre, group, line, idle, abort);
    }
  } else {
    // ---------------- thread r of group g: row r of the tile, keys [32 g, 32 g + 32)
    const int g = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + cS + 32 * g, dp_col = tmem + lanes + cDP + 32 * g;
    const int token = r / p.s.G, head = r - token * p.s.G;
    bool ok = true;
    uint32_t joins = 0, units = 0, n = 0;
    Feed parts(sm.ring, abort);
    Part s{};
    const uint64_t a2 = f2(p.alpha, p.alpha);
    float nl = 0.f, nd = 0.f;
    int i = 0;
    bool live = false;
    // The row of a unit: its terms, and the group's D / 4 channels of dO to TMEM (dP of the unit before is done: its result
    // has been read)
    auto begin_unit = [&]() {
      i = s.i * p.s.w + token;
      live = token < p.s.w && i < s.len;
      const size_t at = ((size_t)s.hk * p.s.T + s.at + i) * p.s.G + head;
      nl = live ? __ldcg(p.nlse + at) : -INFINITY;
      nd = live ? __ldcg(p.ndelta + at) : 0.f;
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.dout.p) +
                                                        (long long)(s.at + i) * p.dout.token +
                                                        (s.hk * p.s.G + head) * p.dout.head + g * (D / 4));
      uint4 v[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) v[e] = live ? row[e] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < D / 32; e += 2) {
        const uint32_t w[8] = {v[e].x, v[e].y, v[e].z, v[e].w, v[e + 1].x, v[e + 1].y, v[e + 1].z, v[e + 1].w};
        tmem_st8(tmem + lanes + cDO + g * (D / 8) + 4 * e, w);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&sm.bar_a_full[1]);
    };
    bool more = parts.next(s);
    if (more) begin_unit();
    while (ok && more) {
      int left = (live && p.s.causal ? i + 1 : s.len) - s.c0 * kTile - 32 * g;  // keys that the row sees
#pragma unroll 1
      for (int j = s.c0; j < s.c1; ++j, ++n, left -= kTile) {
        // (of 32 keys or fewer the second group gives keys 8 to 15 their low halves)
        const int back = g == 1 && s.len - j * kTile <= 32 ? 24 : 0;
        ok = wait(&sm.bar_s[0], n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld32(s_col - back, sv);
        tmem_wait32(sv);
        tc_fence_before();
        warp_arrive(&sm.bar_s_read);
        if (__any_sync(0xffffffffu, left + back < 32)) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= left + back) sv[e] = 0xff800000u;
        }
        const uint64_t l2 = f2(nl, nl), d2 = f2(nd, nd);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2split(ffma2(f2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), a2, l2), x, y);
          sv[e] = __float_as_uint(ex2(x));
          sv[e + 1] = __float_as_uint(ex2(y));
        }
        ok = wait(&sm.bar_dp, n & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t dv[32], w[16], low[4];
        tmem_ld32(dp_col - back, dv);
        tmem_wait32(dv);
        tc_fence_before();
        warp_arrive(&sm.bar_dp_read);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          f2split(fmul2(fadd2(f2(__uint_as_float(dv[e]), __uint_as_float(dv[e + 1])), d2),
                        f2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]))),
                  x, y);
          w[e >> 1] = bf2(x, y);
          if (e < 8) low[e >> 1] = bf2(x - __uint_as_float(w[e >> 1] << 16), y - __uint_as_float(w[e >> 1] & 0xffff0000u));
        }
        if (n > 0) ok = wait(&sm.bar_ds_free, (n - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        tmem_st16(tmem + lanes + cDS + 16 * g, w);
        sm.low[g * kTile + r] = make_uint4(low[0], low[1], low[2], low[3]);
        tmem_st_wait();
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sm.bar_ds);
      }
      if (!ok) break;
      const Part done = s;
      const int row_i = i;
      const bool was_live = live;
      more = parts.next(s);
      if (more) begin_unit();
      // ---- the unit's sums, 32 channels a group (D = 64: the first two store)
      ok = wait(&sm.bar_acc, units++ & 1);
      if (!ok) break;
      tc_fence_after();
      const int d = 32 * g % D;
      const bool mine = 32 * g < D, whole = done.whole();
      uint32_t o[32];
      tmem_ld32(tmem + lanes + cDQ + d, o);
      tmem_wait32(o);
      if (mine && !whole) store_sums(p.part + (size_t)done.place() * kTile * D, d, r, o);
      tc_fence_before();
      warp_arrive(&sm.bar_acc_read);
      if (!whole) {
        if (!sm.meeting.was_last(p.s.status + kRowCounters + 2 * done.first(), done.parts(), joins++, warp == 0, abort, ok))
          continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0;
#pragma unroll 1
        for (int k = 0; k < done.parts(); ++k)
          add_sums(p.part + (size_t)done.place(k) * kTile * D, d, r, 1.f, reinterpret_cast<float(&)[32]>(o));
      }
      RowStore(was_live && mine ? static_cast<__nv_bfloat16*>(p.d0.p) + (long long)(done.at + row_i) * p.d0.token +
                                      (done.hk * p.s.G + head) * p.d0.head
                                : nullptr)
          .put(reinterpret_cast<const float(&)[32]>(o), d, p.sm_scale);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, kCols);
  if (tid == 0 && sm.abort) atomicMax(p.s.status, (int)kDevTimeout);
  pdl_wait();
  if (blockIdx.x == 0 && tid == 0) atomicExch(p.s.status + kTermsTold, 0);
}

template <int D>
int launch(const BwdParams& dkv, const BwdParams& dq, const PreParams& pre, const sage_rows& Q, const sage_rows& K,
           const sage_rows& V, int H, int sms, cudaStream_t st) {
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_queries(&tq, Q, D, H, dkv.s) || !make_tmap_keys(&tk, K, D, dkv.s) || !make_tmap_keys(&tv, V, D, dkv.s) ||
      !make_tmap_queries(&to, pre.dO, D, H, dkv.s))
    return SAGE_ERR_CUDA;
  const size_t smem = sizeof(BwdSmem<D, 2, 2>) + 1024, smem_q = sizeof(BwdSmem<D, 3, 2>) + 1024;
  if (cudaFuncSetAttribute(packed_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
      cudaFuncSetAttribute(packed_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_q) != cudaSuccess)
    return SAGE_ERR_CUDA;
  constexpr int kPerBlock = 256 / (D / 8) * 4;
  const long long blocks = ((long long)dkv.s.T * H + kPerBlock - 1) / kPerBlock;
  if (blocks > 0x7fffffffll) return SAGE_ERR_UNSUPPORTED;
  const int grid = sms < kMaxParts ? sms : kMaxParts;
  if (launch_pdl(packed_pre_kernel<D>, dim3((unsigned)blocks), dim3(256), 0, st, pre) != cudaSuccess ||
      launch_pdl(packed_dkv_kernel<D>, dim3(grid), dim3(kThreads), smem, st, dkv, tq, tk, tv, to) != cudaSuccess ||
      launch_pdl(packed_dq_kernel<D>, dim3(grid), dim3(kThreads), smem_q, st, dq, tq, tk, tv) != cudaSuccess)
    return SAGE_ERR_CUDA;
  return SAGE_OK;
}

}  // namespace

int launch_packed_bwd(const sage_rows& Q, const sage_rows& K, const sage_rows& V, const sage_rows& O, const float* LSE,
                      const sage_rows& dO, const int* cu, const sage_rows& dQ, const sage_rows& dK, const sage_rows& dV,
                      void* ws, int T, int S, int H, int Hkv, int D, int causal, float sm_scale, cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SAGE_ERR_CUDA;
  const PackedWs l = packed_ws_layout(T, S, H, Hkv, D, true);
  const PackedShape s = packed_shape(cu, ws, T, S, H, Hkv, causal);
  float* nlse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.stats);
  float* ndelta = nlse + (size_t)T * H;
  uint4* more = reinterpret_cast<uint4*>(ndelta + (size_t)T * H + ((4 - 2 * (size_t)T * H % 4) & 3));
  auto inverse = [](int d) { return ~0ull / (unsigned)d + 1; };  // (d = 1 has none: over())
  const PreParams pre{s, O, dO, LSE, nlse, ndelta, more, sm_scale, inverse(H), inverse(s.G)};
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part);
  const BwdParams dkv{s, nlse, ndelta, more, dO, dK, dV, part, sm_scale * kLog2e, sm_scale};
  const BwdParams dq{s,  nlse, ndelta, more, dO, dQ, dQ, part + (size_t)2 * kMaxParts * 2 * kTile * D, sm_scale * kLog2e,
                     sm_scale};
  ScopedTimer timer("packed_bwd", st);
  return D == 128 ? launch<128>(dkv, dq, pre, Q, K, V, H, sms, st) : launch<64>(dkv, dq, pre, Q, K, V, H, sms, st);
}

}  // namespace sage
