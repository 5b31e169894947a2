// Attention over packed sequences, forward: O = softmax(sm_scale Q K^T) V and LSE for every sequence of a packed
// batch, in bf16 with fp32 sums (sage_attn_packed_fwd).
//
// One CTA an SM walks its share of the units (packed.cuh): two row tiles of 128 rows and the 128-key tiles that
// they see.
//  - warp 12 walks, warp 9 brings Q and K by TMA, warp 10 V; two key tiles deep (four at D = 64: no difference);
//  - warps 8 and 11 issue S = Q K^T and O += P V (fp32 accumulators in TMEM), one for each row tile, in turns where both
//    have the key tile, so that the tensor core works on one while the softmax works on the other;
//  - warps 0-3 and 4-7 own a row tile each, a thread a row: S from TMEM, P as bf16 back into TMEM over S's
//    columns, from where the second product takes it.  With m the row's running reference, P = 2^(S a - m),
//    a = sm_scale log2 e; m follows the maximum only when that has grown by 2^kRaise, so O is seldom rescaled.  P's
//    rounding to bf16 (what the product takes) is the only one on the way; row sums are of P before it.
// A unit that was cut leaves its parts' sums in the workspace; whoever finishes last adds them up.
//
// 16001 tokens, 16 heads of 2, D = 128, causal: 0.66 ms, 1.58 PFLOP/s, 82% of what a bf16 product reaches here in a burst;
// repeated for seconds, under the power limit, 0.715 ms, 1.47 PFLOP/s, 84% of what one reaches then.  What bounds it: the
// chain S, softmax, P V of a row tile, of which two run at once (tensor core 65%, issue slots 41%, the exponentials' unit
// 33%; the softmax warps wait for TMEM most).  What the code of the five roles takes to fetch counts as much: the softmax
// unrolled whole costs 12%, copies of the issue for place and stage 10%.  A row's columns shared by two threads (16 softmax
// warps, maxima exchanged): 0.70 ms.  At D = 64 the same chain is 0.71 us a tile beside 0.89 us; S three tiles ahead of P V
// there (a third place for S in TMEM) took 0.18 ms where this takes 0.15: both softmaxes then run at once.
// TMA copies whole boxes: what lies behind a sequence's end is the next one's.  Rows of S behind it are not
// stored, columns are masked; of V's rows those that a product reads (up to 15) are zeroed in shared memory, so that
// nothing of another sequence, a NaN or an infinity among it, enters a sum.  (Of its own sequence's later keys a causal row
// takes V with weight 0, as far as its tile goes: 0 times an infinity is NaN, as in the formula.)
#include "issue.cuh"
#include "launch.h"
#include "packed.cuh"
#include "timer.h"

namespace sage {

namespace {

constexpr int kThreads = 416;
constexpr uint32_t kCols = 512, kColO = 256;  // TMEM: S of place t at 128 t, O at 256 + 128 t
constexpr float kRaise = 8.f;

struct FwdParams {
  PackedShape s;
  __nv_bfloat16* O;
  long long o_token, o_head;
  float* LSE;
  float* part;  // of each worker two places, of each two row tiles: [D / 4][128] sums of four, [128] references, [128] row sums
  float alpha;  // sm_scale log2 e
};

template <int D>
struct FwdSmem {
  uint8_t q[2][kTile * D * 2];
  uint8_t k[2][kTile * D * 2];
  uint8_t v[2][kTile * D * 2];
  uint64_t bar_q_full[2], bar_q_empty[2], bar_k_full[2], bar_k_empty[2], bar_v_full[2], bar_v_empty[2], bar_v_raw;
  uint64_t bar_s[2], bar_p[2], bar_o[2], bar_o_read[2], bar_turn[2];
  FeedRing ring;
  Meeting meeting[2];
  long long wsum[kThreads / 32];
  long long pre[kPackedGroups + 1];
  unsigned long long tokens;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(FwdSmem<128>) + 1024 <= 227 * 1024, "shared memory of a CTA");

// The key tiles of a unit's two row tiles: place `t0` has the first row tile, the other one the second, if there is one.
// Row tiles alone in their unit take the places in turns (`solo` counts them).
struct Places {
  int t0, rows;    // rows: row tiles
  int end0, end1;  // by row tile: where its key tiles end
  __device__ __forceinline__ Places() : t0(0), rows(0), end0(0), end1(0) {}
  __device__ __forceinline__ Places(const PackedShape& p, const Part& s, int& solo) {
    rows = (2 * s.i + 1) * p.w < s.len ? 2 : 1;
    t0 = rows == 1 ? (solo++ & 1) : 0;
    end0 = p.causal ? min(s.c1, (min(s.len, (2 * s.i + 1) * p.w) + kTile - 1) / kTile) : s.c1;
    end1 = s.c1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    packed_fwd_kernel(const FwdParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kAtoms = D / 64;      // 128-byte columns of a tile row
  constexpr int kAtom = kTile * 128;  // bytes of one
  extern __shared__ uint8_t smem_raw[];
  FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      sm.meeting[t].init(4);
      mbar_init(&sm.bar_q_full[t], 1);
      mbar_init(&sm.bar_q_empty[t], 1);
      mbar_init(&sm.bar_k_full[t], 1);
      mbar_init(&sm.bar_k_empty[t], 2);
      mbar_init(&sm.bar_v_full[t], 1);
      mbar_init(&sm.bar_v_empty[t], 2);
      mbar_init(&sm.bar_s[t], 1);
      mbar_init(&sm.bar_turn[t], 1);
      mbar_init(&sm.bar_p[t], 4);
      mbar_init(&sm.bar_o[t], 1);
      mbar_init(&sm.bar_o_read[t], 4);
    }
    mbar_init(&sm.bar_v_raw, 1);
    sm.ring.init(12);
    sm.abort = 0;
    sm.tokens = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 8) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  const int group = ceil_div(p.s.S, kPackedGroups);
  prefix_of_sequences<kPairs, kThreads>(p.s, group, sm.pre, sm.wsum, &sm.tokens);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // dependents may come once this CTA holds its TMEM: a later kernel that allocates all columns
  // must not reach this SM before
  pdl_trigger();
  constexpr uint32_t tmem = 0;  // (where an allocation of all columns begins)
  volatile int* abort = &sm.abort;
  const Shares line(sm.pre[kPackedGroups], gridDim.x);
  const int w0 = blockIdx.x;
  if (sm.tmem_base != tmem && tid == 0) atomicMax(p.s.status, (int)kDevSetup);
  const bool idle = line.total == 0 || too_many(p.s, sm.tokens) || w0 >= line.parts || sm.tmem_base != tmem;
  Feed parts(sm.ring, abort);
  Part s;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, abort); };
  int solo = 0;

  if (warp >= 8) {
    if (warp == 8 || warp == 11) {
      // ---------------- MMA issuers, warp 8 for the first place, warp 11 for the second.  P V of a key tile and S of the
      // next one go in together; what comes early (K, V, Q, the turn) is waited for before P.  Every MMA stands here
      // once: copies for each place and stage, whose descriptors would be constants, take longer to fetch than they save.
      const int t = warp == 8 ? 0 : 1;
      constexpr uint32_t id_s = idesc_bf16(kTile, kTile, false, false), id_o = idesc_bf16(kTile, D, false, true);
      constexpr uint64_t kNext = (uint64_t)kTile * D * 2 >> 4, kAtomStep = kAtom >> 4;
      const uint64_t dq = sdesc_sw128(smem_u32(sm.q[t]), 16, 1024), dk = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sm.v[0]), kAtom, 1024);
      const uint32_t s_col = t * 128, o_col = kColO + t * 128;
      uint32_t kc = 0, np = 0, nu = 0, turns = 0;  // key tiles that came by, P tiles and units here, turns taken
      bool ok = true;
#pragma unroll 1
      while (ok && parts.next(s)) {
        const Places pl(p.s, s, solo);
        const int x = t ^ pl.t0, end = x < pl.rows ? (x ? pl.end1 : pl.end0) : s.c0;
        // P V of tile j (kc) and S of tile j + 1; before the first tile S alone
#pragma unroll 1
        for (int j = s.c0 - 1; ok && j < end && s.c0 < end; ++j) {
          const bool pv = j >= s.c0, more = j + 1 < end;
          const uint32_t st = kc & 1, next = pv ? kc + 1 : kc;
          bool paired = false;
          if (more) ok = wait(&sm.bar_k_full[next & 1], (next >> 1) & 1);
          if (!pv) {
            ok = ok && wait(&sm.bar_q_full[t], nu & 1);
          } else {
            ok = ok && wait(&sm.bar_v_full[st], (kc >> 1) & 1);
            if (j == s.c0) ok = ok && (nu == 0 || wait(&sm.bar_o_read[t], (nu - 1) & 1));
            // Where both places have the key tile their products go in in turns: mixed they would end together, and the
            // tensor core wait for both softmaxes.
            paired = pl.rows == 2 && j < pl.end0;
            if (paired) {
              if (turns + t > 0) ok = ok && wait(&sm.bar_turn[t], (turns + t - 1) & 1);
              ++turns;
            }
            ok = ok && wait(&sm.bar_p[t], np++ & 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (pv) {
            const uint64_t b = dv + st * kNext;
            const int keys = s.len - j * kTile;
            if (keys >= kTile) {
              issue_ts_x4(o_col, s_col, b, id_o, j > s.c0);
              issue_ts_x4(o_col, s_col + 32, b + (4 * 2048 >> 4), id_o, 1);
            } else {
#pragma unroll 1
              for (int e = 0; e * 16 < keys; ++e) issue_ts(o_col, s_col + 8 * e, b + (e * 2048 >> 4), id_o, e > 0 || j > s.c0);
            }
            commit(&sm.bar_v_empty[st]);
            if (!more) commit(&sm.bar_o[t]);
            ++kc;
          }
          if (more) {
            const uint64_t b = dk + (next & 1) * kNext;
#pragma unroll
            for (int h = 0; h < kAtoms; ++h) issue_ss_x4(s_col, dq + h * kAtomStep, b + h * kAtomStep, id_s, h > 0);
            commit(&sm.bar_s[t]);
            commit(&sm.bar_k_empty[next & 1]);
            if (j + 2 == end) commit(&sm.bar_q_empty[t]);
          }
          if (paired && lane == 0) mbar_arrive(&sm.bar_turn[t ^ 1]);
          __syncwarp();
        }
        if (s.c0 < end) ++nu;
        // tiles that only the other place takes
#pragma unroll 1
        for (int j = max(end, s.c0); ok && j < s.c1; ++j, ++kc) {
          ok = wait(&sm.bar_k_full[kc & 1], (kc >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(&sm.bar_k_empty[kc & 1]);
          ok = ok && wait(&sm.bar_v_full[kc & 1], (kc >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(&sm.bar_v_empty[kc & 1]);
        }
      }
    } else if (warp == 9) {
      // ---------------- Q and K
      uint32_t kc = 0, nq[2] = {0, 0};
      bool ok = true;
      const uint32_t q_bytes = p.s.G * p.s.w * D * 2;
      while (ok && parts.next(s)) {
        const Places pl(p.s, s, solo);
        auto load_q = [&](int x) {
          const int t = x ^ pl.t0;
          ok = ok && (nq[t] == 0 || wait(&sm.bar_q_empty[t], (nq[t] - 1) & 1));
          ++nq[t];
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&sm.bar_q_full[t], q_bytes);
#pragma unroll
            for (int h = 0; h < kAtoms; ++h)
              tma_load_3d(sm.q[t] + h * kAtom, &tm_q, h * 64, s.hk * p.s.G, s.at + (2 * s.i + x) * p.s.w, &sm.bar_q_full[t]);
          }
        };
        // the first row tile, a key tile, the second row tile, the other key tiles
#pragma unroll 1
        for (int j = s.c0; ok && j < max(s.c1, s.c0 + pl.rows); ++j) {
          if (j - s.c0 < pl.rows) load_q(j - s.c0);
          if (!ok || j >= s.c1) continue;
          const uint32_t st = kc & 1;
          ok = kc < 2 || wait(&sm.bar_k_empty[st], ((kc >> 1) - 1) & 1);
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&sm.bar_k_full[st], kTile * D * 2);
#pragma unroll
            for (int h = 0; h < kAtoms; ++h)
              tma_load_3d(sm.k[st] + h * kAtom, &tm_k, h * 64, s.at + j * kTile, s.hk, &sm.bar_k_full[st]);
          }
          __syncwarp();
          ++kc;
        }
      }
      // (the last copies are waited for by those who use them, or, after a wait that ran out, here)
      int give_up = 0;
      for (int t = 0; t < 2; ++t) {
        if (nq[t]) mbar_wait(&sm.bar_q_full[t], (nq[t] - 1) & 1, &give_up);
        if (kc > (uint32_t)t) mbar_wait(&sm.bar_k_full[(kc - 1 - t) & 1], ((kc - 1 - t) >> 1) & 1, &give_up);
      }
    } else if (warp == 12) {
      feed<kPairs>(p.s, sm.ring, sm.pre, group, line, idle, abort);
    } else if (warp == 10) {
      // ---------------- V
      uint32_t kc = 0, nr = 0;
      bool ok = true;
      while (ok && parts.next(s)) {
        for (int j = s.c0; ok && j < s.c1; ++j, ++kc) {
          const uint32_t st = kc & 1;
          ok = kc < 2 || wait(&sm.bar_v_empty[st], ((kc >> 1) - 1) & 1);
          if (!ok) break;
          const int keys = s.len - j * kTile;
          const bool ragged = keys < kTile && (keys & 15);
          uint64_t* bar = ragged ? &sm.bar_v_raw : &sm.bar_v_full[st];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, kTile * D * 2);
#pragma unroll
            for (int h = 0; h < kAtoms; ++h) tma_load_3d(sm.v[st] + h * kAtom, &tm_v, h * 64, s.at + j * kTile, s.hk, bar);
          }
          __syncwarp();
          if (ragged) {
            // rows up to the next multiple of 16: the product reads them
            int give_up = 0;
            ok = __all_sync(0xffffffffu, mbar_wait(bar, nr++ & 1, &give_up));
            if (!ok) {
              *abort = 1;
              break;
            }
            const int rows = (16 - keys) & 15;
            for (int x = lane; x < rows * kAtoms * 8; x += 32) {
              const int row = keys + x / (kAtoms * 8), c = x % (kAtoms * 8);
              *reinterpret_cast<uint4*>(sm.v[st] + (c >> 3) * kAtom + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.bar_v_full[st]);
          }
        }
      }
      int give_up = 0;
      for (uint32_t t = 0; t < 2; ++t)
        if (kc > t) mbar_wait(&sm.bar_v_full[(kc - 1 - t) & 1], ((kc - 1 - t) >> 1) & 1, &give_up);
    }
  } else {
    // ---------------- softmax: thread r of the group owns row r of the row tile at place t
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + t * 128, o_col = tmem + lanes + kColO + t * 128;
    const int token = r / p.s.G, head = r - token * p.s.G;  // of the tile
    uint32_t ns = 0, no = 0, joins = 0;
    bool ok = true;
    while (ok && parts.next(s)) {
      const Places pl(p.s, s, solo);
      const int x = t ^ pl.t0;
      if (x >= pl.rows) continue;
      const int i = (2 * s.i + x) * p.s.w + token;
      const bool live = token < p.s.w && i < s.len;
      const int lim = live && p.s.causal ? i + 1 : s.len;
      float m = -INFINITY, l = 0.f;
      const int end = x ? pl.end1 : pl.end0;
#pragma unroll 1
      for (int j = s.c0; ok && j < end; ++j) {
        ok = wait(&sm.bar_s[t], ns++ & 1);
        if (!ok) break;
        tc_fence_after();
        // (twice over S in loops: unrolled whole, the code of the warps' roles together takes longer to fetch than to run)
        const int left = lim - j * kTile;
        if (__any_sync(0xffffffffu, left < kTile)) {  // masked in TMEM, so that the loops behind need not ask
#pragma unroll 1
          for (int c = 0; c < kTile; c += 32) {
            uint32_t v[32];
            tmem_ld32(s_col + c, v);
            tmem_wait32(v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e >= left) v[e] = 0xff800000u;
            tmem_st32(s_col + c, v);
          }
          tmem_st_wait();
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (apart: one chain of maxima would wait for itself)
#pragma unroll 1
        for (int c = 0; c < kTile; c += 64) {
          uint32_t v[2][32];
          tmem_ld32(s_col + c, v[0]);
          tmem_ld32(s_col + c + 32, v[1]);
          tmem_ld_wait();
          reg_fence32(v[0]);
          reg_fence32(v[1]);
#pragma unroll
          for (int e = 0; e < 64; e += 2)
            tops[(e >> 1) & 3] =
                max3(tops[(e >> 1) & 3], __uint_as_float(v[e >> 5][e & 31]), __uint_as_float(v[e >> 5][(e & 31) + 1]));
        }
        float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        top *= p.alpha;
        const bool raise = top > m + kRaise;  // (m = -infinity: whenever there is a key)
        if (__any_sync(0xffffffffu, raise)) {
          const float corr = raise ? ex2(m - top) : 1.f;
          if (raise) m = top;
          l *= corr;
          if (j > s.c0) {  // (the part's first product overwrites O; P V of the tile before is done: S came after it)
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_ld32(o_col + d, o);
              tmem_wait32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st32(o_col + d, o);
            }
          }
        }
        const float sub = m == -INFINITY ? 0.f : m;
        const uint64_t a2 = f2(p.alpha, p.alpha), m2 = f2(-sub, -sub);
        uint64_t sums[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        // P of 64 keys at once: a store of 32 columns takes no longer than one of 16
        uint32_t w[32];
        auto exps = [&](const uint32_t (&v)[32], int at) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float u0, u1;
            f2split(ffma2(f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), a2, m2), u0, u1);
            u0 = ex2(u0), u1 = ex2(u1);
            sums[(e >> 1) & 1] = fadd2(sums[(e >> 1) & 1], f2(u0, u1));
            w[at + (e >> 1)] = bf2(u0, u1);
          }
        };
#pragma unroll 1
        for (int c = 0; c < kTile; c += 64) {
          uint32_t v0[32], v1[32];
          tmem_ld32(s_col + c, v0);
          tmem_wait32(v0);
          tmem_ld32(s_col + c + 32, v1);
          exps(v0, 0);
          tmem_wait32(v1);
          exps(v1, 16);
          tmem_st32(s_col + (c >> 1), w);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sm.bar_p[t]);
        float y0, y1;
        f2split(fadd2(sums[0], sums[1]), y0, y1);
        l += y0 + y1;
      }
      // ---- the part's result
      ok = ok && wait(&sm.bar_o[t], no++ & 1);
      if (!ok) break;
      tc_fence_after();
      const int h = s.hk * p.s.G + head;
      const RowStore out(live ? p.O + (long long)(s.at + i) * p.o_token + h * p.o_head : nullptr);
      constexpr size_t kPart = (size_t)kTile * (D + 2);
      auto part_of = [&](int k) { return p.part + (size_t)(2 * s.place(k) + x) * kPart; };
      const bool whole = s.whole();
      if (!whole) {
        float* part = p.part + (size_t)(2 * s.place() + x) * kPart;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + d, o);
          tmem_wait32(o);
          store_sums(part, d, r, o);
        }
        tc_fence_before();
        warp_arrive(&sm.bar_o_read[t]);
        part[(size_t)kTile * D + r] = m;
        part[(size_t)kTile * (D + 1) + r] = l;
        if (!sm.meeting[t].was_last(p.s.status + kFwdCounters + 2 * s.first() + x, s.parts(), joins++, (warp & 3) == 0, abort,
                                    ok))
          continue;
        // O = sum O_k 2^(m_k - M) / sum l_k 2^(m_k - M)
        m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int k = 0; k < s.parts(); ++k) m = fmaxf(m, __ldcg(part_of(k) + (size_t)kTile * D + r));
        const float sub = m == -INFINITY ? 0.f : m;
#pragma unroll 1
        for (int k = 0; k < s.parts(); ++k)
          l = fmaf(__ldcg(part_of(k) + (size_t)kTile * (D + 1) + r), ex2(__ldcg(part_of(k) + (size_t)kTile * D + r) - sub), l);
      }
      const float g = l != 0.f ? 1.f / l : 0.f, sub = m == -INFINITY ? 0.f : m;
      if (live) p.LSE[(size_t)h * p.s.T + s.at + i] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        if (whole) {
          tmem_ld32(o_col + d, o);
          tmem_wait32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
#pragma unroll 1
          for (int k = 0; k < s.parts(); ++k)
            add_sums(part_of(k), d, r, ex2(__ldcg(part_of(k) + (size_t)kTile * D + r) - sub), reinterpret_cast<float(&)[32]>(o));
        }
        out.put(reinterpret_cast<const float(&)[32]>(o), d, g);
      }
      if (whole) {
        tc_fence_before();
        warp_arrive(&sm.bar_o_read[t]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(sm.tmem_base, kCols);
  if (tid == 0 && sm.abort) atomicMax(p.s.status, (int)kDevTimeout);
}

template <int D>
int launch(const FwdParams& p, const sage_rows& Q, const sage_rows& K, const sage_rows& V, int H, int sms, cudaStream_t st) {
  auto kern = packed_fwd_kernel<D>;
  CUtensorMap tq, tk, tv;
  if (!make_tmap_queries(&tq, Q, D, H, p.s) || !make_tmap_keys(&tk, K, D, p.s) || !make_tmap_keys(&tv, V, D, p.s))
    return SAGE_ERR_CUDA;
  const size_t smem = sizeof(FwdSmem<D>) + 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return SAGE_ERR_CUDA;
  const int grid = sms < kMaxParts ? sms : kMaxParts;
  if (launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, p, tq, tk, tv) != cudaSuccess)
    return SAGE_ERR_CUDA;
  return SAGE_OK;
}

}  // namespace

PackedWs packed_ws_layout(int T, int, int H, int, int D, bool backward) {
  auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  PackedWs l;
  l.part = kHeader * sizeof(int);
  // (the backward's are dK, dV and dQ of 128 rows each)
  l.stats = l.part + up((size_t)2 * kMaxParts * kTile * (backward ? 3 * D : 2 * (D + 2)) * sizeof(float));
  l.total = l.stats + (backward ? up((size_t)T * H * (2 * sizeof(float) + 16) + 16) : 0);
  return l;
}

int launch_packed_fwd(const sage_rows& Q, const sage_rows& K, const sage_rows& V, const int* cu, const sage_rows& O,
                      float* LSE, void* ws, int T, int S, int H, int Hkv, int D, int causal, float sm_scale,
                      cudaStream_t st) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SAGE_ERR_CUDA;
  FwdParams p;
  p.s = packed_shape(cu, ws, T, S, H, Hkv, causal);
  p.O = static_cast<__nv_bfloat16*>(O.p);
  p.o_token = O.token, p.o_head = O.head;
  p.LSE = LSE;
  const PackedWs l = packed_ws_layout(T, S, H, Hkv, D, false);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part);
  p.alpha = sm_scale * 1.4426950408889634f;
  ScopedTimer timer("packed_fwd", st);
  return D == 128 ? launch<128>(p, Q, K, V, H, sms, st) : launch<64>(p, Q, K, V, H, sms, st);
}

}  // namespace sage
