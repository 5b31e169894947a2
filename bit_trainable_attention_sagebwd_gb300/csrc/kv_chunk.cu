// Attention of many query rows over the 8-bit paged cache: a chunk of a prompt behind what the cache
// holds of it (sage_attn_kv_attention, more than 32 query rows of a shared head).
//
// The products are what counts here: 4 D operations for every (query row, key) pair against
// 2 D bytes for every key that 256 rows share.  One CTA an SM takes units of 256 rows (two tiles of
// 128: the queries of the G heads of a key/value head, token by token) and walks the unit's
// 128-key tiles; a unit of one row tile takes its key tiles in turns (Mode):
//  - warps 17 and 18 bring the codes of K and V by TMA, half a tile at a time; warps 8-11 (K) and 12-15 (V)
//    turn them into fp16 (exact) and store them where tcgen05.mma reads them (128-byte swizzle), two
//    tiles deep;
//  - warp 16 issues S = Q K^T and O += P V (kind::f16, fp32 accumulators in TMEM) for the two row
//    tiles in turn, so the tensor core works on one tile while the softmax works on the other;
//  - warps 0-3 and 4-7 own a row tile each, a thread a row: S from TMEM, P back into TMEM over S's
//    columns, from where the second product takes it.  The maximum is found with the exponentials,
//    not before them: the reference that they need moves seldom (see kRaise).
// Units are cut over the grid like those of the few-row kernel (kv_attn.cu), in 128-key tiles.
//
// Measured: the newest 2048 queries of 32 heads on 32k keys of 8 (D = 128, e4m3, 1.07 TFLOP) in 0.90 to
// 0.92 ms, 1.17 PFLOP/s, 61 % of a large library product's rate in a burst, 68 % of its sustained one; DRAM is idle
// (0.26 GB).  The tensor core
// works for half of the time and the issue slots are taken for two thirds of it: the conversion of the codes
// (0.78 ms without it) and the exponentials share the SM's instruction slots.  The conversion
// instruction for e4m3 in place of shifts took 1.22 ms, a wider softmax (896 threads) was slower.
#include <type_traits>

#include "kv_attn.cuh"
#include "launch.h"
#include "tmap.h"

namespace sage {

namespace {

constexpr int kThreads = 640;
constexpr int kTile = 128, kHalf = 64;       // keys of a tile (and of half of one), rows of a row tile
constexpr int kGroups = 128;                 // the batch rows in at most so many groups
constexpr int kRegsSoftmax = 144, kRegsLoad = 64, kRegsIssue = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsLoad + kRegsIssue <= 5 * 96, "the launch's registers");
constexpr uint32_t kCols = 512, kColO = 256; // TMEM: S of row tile t at 128 t, O at 256 + 128 t

// half tiles of codes on their way or being converted, for K and for V: what fits
template <int D>
constexpr int kRaw = D == 64 ? 4 : 2;

template <int D>
struct ChunkSmem {
  uint8_t q[2][kTile * D * 2];
  uint8_t k[2][kTile * D * 2];
  uint8_t v[2][kTile * D * 2];
  uint8_t raw[2][kRaw<D>][kHalf * D];  // codes of K and V
  uint64_t bar_half, bar_joined;  // turns: the second group's part of the rows is there, has been read
  uint64_t bar_q[2], bar_k_full[2], bar_k_empty[2], bar_v_full[2], bar_v_empty[2], bar_raw[2][kRaw<D>], bar_raw_empty[2][kRaw<D>], bar_s[2], bar_p[2], bar_o[2];
  long long wsum[kThreads / 32];
  long long pre[kGroups + 1];  // tiles before each group of batch rows
  uint32_t tmem_base;
  int abort;
  int seg[2];                  // for the MMA issuer: 4 x tiles of a part + its Mode, 0: no more
};
static_assert(sizeof(ChunkSmem<128>) + 1024 <= 227 * 1024, "shared memory of a CTA");

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Issue by a whole warp: one lane (always the same) is elected inside the asm, so the operands stay in
// uniform registers, where tcgen05 takes them from.  (In a branch of one lane each MMA's descriptors are
// moved there first, which took longer than the MMA.)  acc == 0: the first of the four overwrites D.
// S: D[tmem] (+)= A[smem] * B[smem]^T, four along K, the descriptors moving by 32 bytes
__device__ __forceinline__ void issue_ss_x4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p, q;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, %4, %4;\n"
      " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
      " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// O: D[tmem] (+)= A[tmem] * B[smem], four along K: A's rows are the lanes, two fp16 along K in a column, 8
// columns an MMA; B's descriptor moves by 16 rows
__device__ __forceinline__ void issue_ts_x4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred e, p, q;\n .reg .b64 b1, b2, b3;\n .reg .b32 a1, a2, a3;\n"
      " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 q, %4, %4;\n"
      " add.s32 a1, %1, 8;\n add.s32 a2, %1, 16;\n add.s32 a3, %1, 24;\n"
      " add.s64 b1, %2, 128;\n add.s64 b2, %2, 256;\n add.s64 b3, %2, 384;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// A part of a unit: key tiles [c0, c1) of row tile pair rt of (batch row b, key/value head hk).
// How the two row tiles' places (operands, TMEM, softmax groups) are used in a part: kOne: the first one
// alone; kTwo: a row tile each, the same key tiles; kTurns: the one row tile in both, the key tiles in
// turns, joined at the part's end.  (48 rows on 4 sequences of 100k to 131k tokens, 8 heads of D = 128: 334 us,
// with the first place alone 376 us.)
enum Mode { kOne, kTwo, kTurns };
struct Seg {
  int b, slot, hk, rt, len, q_len, c0, c1, chunks;
  Mode mode;
  long long unit_at;
};

__device__ __forceinline__ int pair_chunks(const AttnParams& p, int len, int q_len, int rt) {
  const int i0 = rt * kChunkRows / p.G;
  if (i0 >= q_len) return 0;
  const int last = min(q_len - 1, (int)(((long long)rt * kChunkRows + kChunkRows - 1) / p.G));
  return max(1, (row_end(p, len, q_len, last) + kTile - 1) / kTile);
}

// tiles of all units of batch row b
__device__ __forceinline__ long long row_chunks(const AttnParams& p, int b) {
  int slot;
  const int len = row_length(p, b, slot), q_len = row_queries(p, b);
  long long n = 0;
#pragma unroll 1
  for (int rt = 0; rt < p.tiles; ++rt) n += pair_chunks(p, len, q_len, rt);
  return n * p.c.Hkv;
}

// A worker's way along the line: the parts from `at` to `stop`, in order.  It stands at the units of
// row tile pair rt of batch row b, n tiles each, the first of them at `base`.
struct Walk {
  long long at, stop, base;
  int b, rt, n, slot, len, q_len;
  __device__ Walk(const AttnParams& p, const long long* pre, int group, long long begin, long long end)
      : at(begin), stop(end), base(0), b(0) {
    if (begin >= end) return;
    const int g = row_at(pre, kGroups, begin);
    b = g * group;
    base = pre[g];
    enter(p);
  }
  __device__ void enter(const AttnParams& p) {
    len = row_length(p, b, slot);
    q_len = row_queries(p, b);
    rt = 0;
    n = pair_chunks(p, len, q_len, 0);
  }
  __device__ bool more() const { return at < stop; }
  __device__ Seg next(const AttnParams& p) {
#pragma unroll 1
    while (at >= base + (long long)n * p.c.Hkv) {
      base += (long long)n * p.c.Hkv;
      if (++rt < p.tiles) {
        n = pair_chunks(p, len, q_len, rt);
      } else {
        ++b;
        enter(p);
      }
    }
    Seg s;
    s.b = b, s.slot = slot, s.len = len, s.q_len = q_len, s.rt = rt, s.chunks = n;
    s.hk = (int)mul_div(at - base, 1, n);
    s.unit_at = base + (long long)s.hk * n;
    s.c0 = (int)(at - s.unit_at);
    s.c1 = (int)min((long long)n, stop - s.unit_at);
    s.mode = (long long)rt * kChunkRows + kTile < (long long)q_len * p.G ? kTwo : s.c1 - s.c0 > 1 ? kTurns : kOne;
    at = s.unit_at + s.c1;
    return s;
  }
};

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1) kv_chunk_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kAtoms = D / 64;       // 128-byte columns of a tile row
  constexpr int kAtom = kTile * 128;   // bytes of one
  extern __shared__ uint8_t smem_raw[];
  ChunkSmem<D>& sm = *reinterpret_cast<ChunkSmem<D>*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.bar_q[s], 128);
      mbar_init(&sm.bar_k_full[s], 128);
      mbar_init(&sm.bar_k_empty[s], 1);
      mbar_init(&sm.bar_v_full[s], 128);
      mbar_init(&sm.bar_v_empty[s], 1);
      for (int h = 0; h < kRaw<D>; ++h) {
        mbar_init(&sm.bar_raw[s][h], 1);
        mbar_init(&sm.bar_raw_empty[s][h], 128);
      }
      mbar_init(&sm.bar_s[s], 1);
      mbar_init(&sm.bar_p[s], 128);
      mbar_init(&sm.bar_o[s], 1);
    }
    mbar_init(&sm.bar_half, 128);
    mbar_init(&sm.bar_joined, 128);
    sm.abort = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 16) {
    tmem_alloc(&sm.tmem_base, kCols);
    tmem_relinquish();
  }
  const int group = (p.B + kGroups - 1) / kGroups;
  prefix_of<kThreads>(kGroups, sm.pre, sm.wsum, [&](int g) {
    long long n = 0;
#pragma unroll 1
    for (int b = g * group; b < min(p.B, (g + 1) * group); ++b) n += row_chunks(p, b);
    return n;
  });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // dependents may come once this CTA holds its TMEM: a later kernel that allocates all columns
  // must not reach this SM before
  pdl_trigger();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort = &sm.abort;
  const long long total = sm.pre[kGroups];
  const Line line{total, (int)min((long long)gridDim.x, max(total, 1ll))};
  const int w0 = blockIdx.x;
  const bool idle = total == 0 || w0 >= line.parts;
  const long long begin = idle ? 0 : line.start(w0), stop = idle ? 0 : line.start(w0 + 1);
  const int per_page = p.c.page >> 4;  // 16-key groups of a page
  const int page_shift = 31 - __clz(per_page);
  // the page of the 16-key group `grp` of a slot; -1: no key there
  auto page_of = [&](int slot, int len, int grp) {
    if (grp * 16 >= len) return -1;
    const int page = p.c.table[(size_t)slot * p.c.max_pages + (grp >> page_shift)];
    if ((unsigned)page < (unsigned)p.c.n_pages) return page;
    atomicMax(p.c.status, kDevIndex);
    return -1;
  };

  if (warp >= 16) {
    regs_decrease<kRegsIssue>();
    if (warp == 16 && begin < stop) {
      // ---------------- MMA issuer
      constexpr uint32_t id_s = idesc_f16(kTile, kTile, false), id_o = idesc_f16(kTile, D, true);
      uint32_t kc = 0, ns[2] = {0, 0}, np[2] = {0, 0};  // key tiles, segments and P tiles so far
      // descriptors of the first tile of each kind; the second one lies kTile rows behind
      constexpr uint64_t kNext = (uint64_t)kTile * D * 2 >> 4, kAtomStep = kAtom >> 4;
      const uint64_t dq = sdesc_sw128(smem_u32(sm.q[0]), 16, 1024), dk = sdesc_sw128(smem_u32(sm.k[0]), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sm.v[0]), kAtom, 1024);
      auto issue_s = [&](int t, uint32_t kv) {
        const uint64_t a = dq + t * kNext, b = dk + (kv & 1) * kNext;
#pragma unroll
        for (int h = 0; h < kAtoms; ++h) issue_ss_x4(tmem + t * 128, a + h * kAtomStep, b + h * kAtomStep, id_s, h > 0);
        commit(&sm.bar_s[t]);
      };
      auto issue_pv = [&](int t, uint32_t kv, uint32_t acc) {
        const uint64_t b = dv + (kv & 1) * kNext;
        const uint32_t d = tmem + kColO + t * 128, a = tmem + t * 128;
        issue_ts_x4(d, a, b, id_o, acc);
        issue_ts_x4(d, a + 32, b + (4 * 2048 >> 4), id_o, 1);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity, abort); };
      bool ok = true;
      while (ok) {
        // a part: its tiles and mode, said with the first row tile's Q
        if (!wait(&sm.bar_q[0], ns[0] & 1)) break;
        const int said = *const_cast<volatile int*>(&sm.seg[ns[0] & 1]), n = said >> 2;
        const bool two = (said & 3) == kTwo;
        if (n == 0) break;
        if ((said & 3) == kTurns) {
          ok = wait(&sm.bar_q[1], ns[1] & 1);
          auto first = [&](int t) {
            ok = ok && wait(&sm.bar_k_full[(kc + t) & 1], ((kc + t) >> 1) & 1);
            if (!ok) return;
            tc_fence_after();
            issue_s(t, kc + t);
            commit(&sm.bar_k_empty[(kc + t) & 1]);
          };
          // P V of key tile kc, which is place t's, then S of the place's next one
          auto turn = [&](int t, int j) {
            ok = ok && wait(&sm.bar_v_full[kc & 1], (kc >> 1) & 1) && wait(&sm.bar_p[t], np[t] & 1);
            if (!ok) return;
            ++np[t];
            tc_fence_after();
            issue_pv(t, kc, j > 1);
            commit(&sm.bar_v_empty[kc & 1]);
            if (j + 2 >= n) {
              commit(&sm.bar_o[t]);
            } else {
              ok = wait(&sm.bar_k_full[kc & 1], ((kc + 2) >> 1) & 1);
              if (!ok) return;
              tc_fence_after();
              issue_s(t, kc + 2);
              commit(&sm.bar_k_empty[kc & 1]);
            }
            ++kc;
          };
          first(0);
          first(1);
          for (int j = 0; ok && j < n; j += 2) {
            turn(0, j);
            if (ok && j + 1 < n) turn(1, j + 1);
          }
          ++ns[0];
          ++ns[1];
          continue;
        }
        ok = (!two || wait(&sm.bar_q[1], ns[1] & 1)) && wait(&sm.bar_k_full[kc & 1], (kc >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, kc);
        if (two) issue_s(1, kc);
        commit(&sm.bar_k_empty[kc & 1]);
        for (int j = 0; j < n; ++j, ++kc) {
          const bool more = j + 1 < n;
          ok = wait(&sm.bar_v_full[kc & 1], (kc >> 1) & 1) && wait(&sm.bar_p[0], np[0] & 1);
          if (!ok) break;
          ++np[0];
          tc_fence_after();
          issue_pv(0, kc, j > 0);
          if (!more) commit(&sm.bar_o[0]);
          if (more) {
            ok = wait(&sm.bar_k_full[(kc + 1) & 1], ((kc + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, kc + 1);
          }
          if (two) {
            ok = wait(&sm.bar_p[1], np[1] & 1);
            if (!ok) break;
            ++np[1];
            tc_fence_after();
            issue_pv(1, kc, j > 0);
            if (!more) commit(&sm.bar_o[1]);
          }
          commit(&sm.bar_v_empty[kc & 1]);
          if (more) {
            if (two) issue_s(1, kc + 1);
            commit(&sm.bar_k_empty[(kc + 1) & 1]);
          }
        }
        ++ns[0];
        if (two) ++ns[1];
      }
    }
    if ((warp == 17 || warp == 18) && begin < stop) {
      // ---------------- the codes of K (warp 17) or V (18), half a tile at a time: a lane for each page.  The
      // pages' numbers come in windows of 32 boxes, the next window's a window ahead: a load for each half
      // tile would hold the copies up.
      const int v = warp - 17, box = p.c.page < kHalf ? p.c.page : kHalf, boxes = kHalf / box, box_bytes = box * D;
      const CUtensorMap* tm = v ? &tm_v : &tm_k;
      Walk walk(p, sm.pre, group, begin, stop);
      Seg s = walk.next(p);
      int c = 2 * s.c0;  // in half tiles
      const int box_shift = 31 - __clz(boxes), page_shift = 31 - __clz(p.c.page), per = 32 >> box_shift;
      auto window = [&](int half) {
        const int at = half + (lane >> box_shift), token = at * kHalf + (lane & (boxes - 1)) * box;
        return at < 2 * s.c1 && token < s.len ? p.c.table[(size_t)s.slot * p.c.max_pages + (token >> page_shift)] : -1;
      };
      int here = 0, ids = window(c), ids_next = window(c + per);  // here: half tiles of the window so far
      uint32_t n = 0;  // half tiles so far
      for (;; ++n) {
        // (what has no page stays as it was: finite, and masked)
        const int id = __shfl_sync(0xffffffffu, ids, ((here << box_shift) + lane) & 31);
        const bool ok = lane < boxes && (unsigned)id < (unsigned)p.c.n_pages;
        if (!ok && lane < boxes && id != -1) atomicMax(p.c.status, kDevIndex);
        const uint32_t all = __ballot_sync(0xffffffffu, ok);
        const uint32_t at = n % kRaw<D>;
        uint64_t* full = &sm.bar_raw[v][at];
        if (n >= kRaw<D> && !mbar_wait_warp(&sm.bar_raw_empty[v][at], (n / kRaw<D> - 1) & 1, abort)) break;
        if (lane == 0) {
          if (all)
            mbar_arrive_expect_tx(full, __popc(all) * box_bytes);
          else
            mbar_arrive(full);
        }
        __syncwarp();
        if (ok)
          tma_load_3d(sm.raw[v][at] + lane * box_bytes, tm, 0,
                      s.hk * p.c.page + ((c * kHalf + lane * box) & (p.c.page - 1)), id, full);
        if (++c < 2 * s.c1) {
          if (++here == per) {
            here = 0;
            ids = ids_next;
            ids_next = window(c + per);
          }
        } else {
          if (!walk.more()) {
            ++n;
            break;
          }
          s = walk.next(p);
          c = 2 * s.c0;
          here = 0;
          ids = window(c);
          ids_next = window(c + per);
        }
      }
      // the last copies (after a wait that ran out nobody else waits for them)
      for (uint32_t k = n < kRaw<D> ? 0 : n - kRaw<D>; k < n; ++k) {
        int give_up = 0;
        mbar_wait(&sm.bar_raw[v][k % kRaw<D>], (k / kRaw<D>) & 1, &give_up);
      }
    }
  } else if (warp >= 8) {
    regs_decrease<kRegsLoad>();
    // ---------------- loaders: thread `lt` takes 16 bytes of kRows rows of a K or V tile
    constexpr int kPerRow = D / 16, kRowStep = 128 / kPerRow, kRows = kTile / kRowStep;
    const int v = (warp >> 2) - 2, lt = tid & 127, r0 = lt / kPerRow, piece = lt % kPerRow;
    const uint32_t n = (uint32_t)(stop - begin);
    for (uint32_t kc = 0; kc < n; ++kc) {
      const uint32_t st = kc & 1;
      if (kc >= 2 && !mbar_wait(v ? &sm.bar_v_empty[st] : &sm.bar_k_empty[st], ((kc >> 1) - 1) & 1, abort)) break;
      // 16 codes of a row -> two 16-byte chunks of the swizzled tile; lanes whose chunks would meet
      // in the same banks store them in the other order
      uint8_t* tile = v ? sm.v[st] : sm.k[st];
      bool ok = true;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t half = 2 * kc + h, at = half % kRaw<D>;
        ok = ok && mbar_wait(&sm.bar_raw[v][at], (half / kRaw<D>) & 1, abort);
#pragma unroll 2  // (instruction fetch is shared: unrolled in full the kernel took a tenth longer)
        for (int i = 0; i < kRows / 2; ++i) {
          const uint4 y = *reinterpret_cast<const uint4*>(sm.raw[v][at] + (i * 128 + lt) * 16);
          const int r = h * kHalf + r0 + i * kRowStep, u = (piece * 2) & 7;
          uint4 lo, hi;
          codes_to_half<KIND>(y.x, lo.x, lo.y);
          codes_to_half<KIND>(y.y, lo.z, lo.w);
          codes_to_half<KIND>(y.z, hi.x, hi.y);
          codes_to_half<KIND>(y.w, hi.z, hi.w);
          uint8_t* row = tile + (piece >> 2) * kAtom + (r >> 3) * 1024 + (r & 7) * 128;
          const bool swap = D == 128 && ((piece >> 2) & 1);
          *reinterpret_cast<uint4*>(row + (((u + swap) ^ (r & 7)) << 4)) = swap ? hi : lo;
          *reinterpret_cast<uint4*>(row + (((u + !swap) ^ (r & 7)) << 4)) = swap ? lo : hi;
        }
        mbar_arrive(&sm.bar_raw_empty[v][at]);
      }
      if (!ok) break;
      fence_proxy_async_smem();
      mbar_arrive(v ? &sm.bar_v_full[st] : &sm.bar_k_full[st]);
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // ---------------- softmax: thread r of the group owns row r of row tile t
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + t * 128, o_col = tmem + lanes + kColO + t * 128;
    uint32_t n_s = 0, n_o = 0, n_turns = 0;
    bool ok = true;  // (of the warp)
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait_warp(bar, parity, abort); };
    Walk walk(p, sm.pre, group, begin, stop);
    while (ok && walk.more()) {
      const Seg s = walk.next(p);
      const long long unit_id = ((long long)s.b * p.tiles + s.rt) * p.c.Hkv + s.hk;
      if (s.c0 == 0 && tid == 0)
        p.info[unit_id] = make_int2(w0, line.holder(s.unit_at + s.chunks - 1));
      if (t == 1 && s.mode == kOne) continue;
      const bool turns = s.mode == kTurns;
      const long long row = (long long)s.rt * kChunkRows + (turns ? 0 : t * kTile) + r;
      const int i = (int)(row / p.G);
      const bool live = i < s.q_len;
      const size_t orow =
          ((size_t)s.b * p.H + (size_t)s.hk * p.G + (size_t)(row % p.G)) * p.Nq + (live ? i : 0);
      // Q: the row times its power of two, as fp16 (the last part's S have been read: free)
      float a_row;
      {
        const uint4* q = reinterpret_cast<const uint4*>(p.Q + orow * D);
        uint4 w[D / 8];
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          w[u] = live ? q[u] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = max3(top, fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u)));
        }
        float up, down;
        row_power(top, up, down);
        a_row = p.alpha * down * kCodeUnit<KIND>;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {  // channels 0, 2 and 1, 3 of each four, as the codes come
            h[e] = h2bits(__floats2half2_rn(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e + 1] << 16) * up));
            h[e + 1] = h2bits(
                __floats2half2_rn(__uint_as_float(x[e] & 0xffff0000u) * up, __uint_as_float(x[e + 1] & 0xffff0000u) * up));
          }
          *reinterpret_cast<uint4*>(sm.q[t] + (u >> 3) * kAtom + (r >> 3) * 1024 + (r & 7) * 128 +
                                    (((u & 7) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_proxy_async_smem();
      if (tid == 0) sm.seg[n_o & 1] = 4 * (s.c1 - s.c0) + s.mode;
      mbar_arrive(&sm.bar_q[t]);
      const int lim = live ? row_end(p, s.len, s.q_len, i) : s.len;
      float m = -INFINITY, l = 0.f, ref = 0.f;
      bool careful = false;  // (of the warp)
      // lanes 0-7: the tile's eight 16-key groups; scales one tile ahead, pages two.  A group without a page
      // (past the keys, or a page number out of range) has V's scale at -infinity: its P is 2^-infinity, whatever
      // codes its places in shared memory still hold.
      auto scales = [&](int id, float& ks, float& vs) {
        ks = 0.f, vs = -INFINITY;
        if (id >= 0) {
          ks = p.c.k_scale[(size_t)id * p.c.Hkv + s.hk];
          vs = p.c.v_scale[(size_t)id * p.c.Hkv + s.hk];
        }
      };
      auto id_at = [&](int c) { return lane < 8 && c < s.c1 ? page_of(s.slot, s.len, c * 8 + lane) : -1; };
      float ks, vs, ks_n, vs_n;
      const int c0 = s.c0 + (turns ? t : 0), step = turns ? 2 : 1;
      int id = id_at(c0);
      scales(id, ks, vs);
      id = id_at(c0 + step);
#pragma unroll 1
      for (int c = c0; c < s.c1; c += step) {
        scales(id, ks_n, vs_n);
        id = id_at(c + 2 * step);
        // the groups' factors of S, log2 of V's scale and its inverse
        if (lane < 8) ref = fmaxf(ref, vs);
        if (__any_sync(0xffffffffu, lane < 8 && !(vs > 0.f))) {
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
        }
        const float ve = value_scale(vs, ref);
        const float lg = vs == -INFINITY ? -INFINITY : lg2(ve), iv = __frcp_rn(ve);
        wait(&sm.bar_s[t], n_s & 1);
        ++n_s;
        tc_fence_after();
        const bool edge = __any_sync(0xffffffffu, lim < (c + 1) * kTile);
        const int left = lim - c * kTile;
        // P of the row with the reference as it stands, in registers, and the largest u - m; where that
        // passes kRaise (a part's first tile, and seldom again) the reference is raised and P is
        // computed once more from S.  The exponent is s f + (g - m), rounded once; where the reference
        // would pass 2^18 that no longer agrees with the maximum it was raised to, and the rest of the
        // part uses (s f + g) - m and the largest s f + g, in the code of the edge tiles (`careful`).
        uint32_t w[4][16];
        float top, sum_l, sub;  // top: the largest u - m, careful: the largest u
        auto exponentials = [&](auto careful_tile) {
          constexpr bool kCareful = decltype(careful_tile)::value;
          top = -INFINITY, sum_l = 0.f;
          uint32_t sv[2][32];
          tmem_ld32(s_col, sv[0]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            tmem_wait32(sv[x & 1]);
            if (x < 3) tmem_ld32(s_col + 32 * (x + 1), sv[(x + 1) & 1]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float f = __shfl_sync(0xffffffffu, ks, 2 * x + y) * a_row;
              const float lgx = __shfl_sync(0xffffffffu, lg, 2 * x + y), g = lgx - sub;
              const uint64_t f2v = f2(f, f), g2v = f2(g, g);
              uint64_t sum = f2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const float s0 = __uint_as_float(sv[x & 1][y * 16 + e]), s1 = __uint_as_float(sv[x & 1][y * 16 + e + 1]);
                float u0, u1;
                f2split(ffma2(f2(s0, s1), f2v, kCareful ? f2(lgx, lgx) : g2v), u0, u1);
                if (kCareful) {
                  if (x * 32 + y * 16 + e >= left) u0 = -INFINITY;
                  if (x * 32 + y * 16 + e + 1 >= left) u1 = -INFINITY;
                }
                top = max3(top, u0, u1);
                if (kCareful) f2split(fadd2(f2(u0, u1), f2(-sub, -sub)), u0, u1);
                u0 = ex2(u0), u1 = ex2(u1);
                sum = fadd2(sum, f2(u0, u1));
                w[x][y * 8 + (e >> 1)] = h2bits(__floats2half2_rn(u0, u1));
              }
              float y0, y1;
              f2split(sum, y0, y1);
              sum_l = fmaf(y0 + y1, __shfl_sync(0xffffffffu, iv, 2 * x + y), sum_l);
            }
          }
        };
        bool exact = edge || careful;
#pragma unroll 1
        for (;;) {
          sub = m == -INFINITY ? 0.f : m;
          if (exact)
            exponentials(std::true_type());
          else
            exponentials(std::false_type());
          const bool raise = (exact ? top - sub : top) > (m == -INFINITY ? -INFINITY : kRaise);
          if (!__any_sync(0xffffffffu, raise)) break;
          const float to = raise ? (exact ? top : top + sub) - kBelow : m, corr = raise ? ex2(m - to) : 1.f;
          if (!exact && __any_sync(0xffffffffu, raise && fabsf(to) > 0x1p18f)) {
            careful = exact = true;
            continue;
          }
          m = to;
          l *= corr;
          careful = careful || __any_sync(0xffffffffu, raise && fabsf(to) > 0x1p18f);
          if (c > c0) {  // (the part's first product overwrites O; PV of the tile before is done: S came after it)
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
        l += sum_l;
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_st16(s_col + x * 16, w[x]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.bar_p[t]);
        ks = ks_n, vs = vs_n;
      }
      // ---- the part's result
      wait(&sm.bar_o[t], n_o & 1);
      ++n_o;
      tc_fence_after();
      // turns: both places hold a part of the same rows, thread r of both groups the same row in the same
      // TMEM lanes: the first group takes both
      float2* half = reinterpret_cast<float2*>(sm.q[1]);  // (the second place's S are done with Q)
      float f0 = 1.f, f1 = 0.f;
      if (turns && t == 1) {
        half[r] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive(&sm.bar_half);
        wait(&sm.bar_joined, n_turns & 1);
        ++n_turns;
        tc_fence_after();
        continue;
      }
      if (turns) {
        wait(&sm.bar_half, n_turns & 1);
        ++n_turns;
        tc_fence_after();
        const float2 x = half[r];
        const float mt = fmaxf(m, x.x), sub = mt == -INFINITY ? 0.f : mt;
        f0 = ex2(m - sub), f1 = ex2(x.x - sub);
        l = l * f0 + x.y * f1;
        m = mt;
      }
      const bool whole = s.c0 == 0 && s.c1 == s.chunks;
      float* part = p.part + (size_t)(2 * w0 + (s.c0 == 0 ? 1 : 0)) * kChunkRows * (D + 2);
      const float f = whole ? (l != 0.f ? kCodeUnit<KIND> / l : 0.f) : kCodeUnit<KIND>;
      const int pr = t * kTile + r;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        tmem_ld32(o_col + d, o);
        tmem_wait32(o);
        if (turns) {
          uint32_t y[32];
          tmem_ld32(o_col + 128 + d, y);
          tmem_wait32(y);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), f1, __uint_as_float(o[e]) * f0));
        }
        if (!(ok && live)) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 y;
            __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&y);
#pragma unroll
            for (int z = 0; z < 4; ++z)  // (V's channels came as 0, 2, 1, 3 too)
              h[z] = __floats2bfloat162_rn(__uint_as_float(o[8 * e + (z >> 1) * 4 + (z & 1)]),
                                           __uint_as_float(o[8 * e + (z >> 1) * 4 + (z & 1) + 2]));
            *reinterpret_cast<uint4*>(p.O + orow * D + d + 8 * e) = y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(part + (size_t)pr * D + d + 4 * e) =
                make_uint4(o[4 * e], o[4 * e + 2], o[4 * e + 1], o[4 * e + 3]);
        }
      }
      if (turns) {
        tc_fence_before();
        mbar_arrive(&sm.bar_joined);
      }
      if (ok && live) {
        if (whole)
          p.LSE[orow] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
        else
          part[(size_t)kChunkRows * D + pr] = m, part[(size_t)kChunkRows * D + kChunkRows + pr] = l;
      }
    }
    if (t == 0) {
      if (tid == 0) sm.seg[n_o & 1] = 0;
      mbar_arrive(&sm.bar_q[0]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tmem_dealloc(tmem, kCols);
  if (tid == 0 && sm.abort) atomicMax(p.c.status, (int)kDevTimeout);
}

template <int D, int KIND>
int launch(const AttnParams& p, int sms, cudaStream_t st) {
  auto kern = kv_chunk_kernel<D, KIND>;
  // a page's rows [head, token]: boxes of a page's tokens of a head, at most half a tile
  const int box = p.c.page < kHalf ? p.c.page : kHalf;
  CUtensorMap tk, tv;
  if (!make_tmap_3d(&tk, p.c.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, (uint64_t)p.c.Hkv * p.c.page, p.c.n_pages, D,
                    box, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_tmap_3d(&tv, p.c.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, D, (uint64_t)p.c.Hkv * p.c.page, p.c.n_pages, D,
                    box, CU_TENSOR_MAP_SWIZZLE_NONE))
    return 3;
  const size_t smem = sizeof(ChunkSmem<D>) + 1024;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 3;
  const int grid = sms < kMaxChunkParts ? sms : kMaxChunkParts;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, p, tk, tv) == cudaSuccess ? 0 : 3;
}

}  // namespace

int launch_kv_chunk(const AttnParams& p, int kind, int sms, cudaStream_t st) {
  if (p.c.D == 128)
    return kind == SAGE_KV_INT8 ? launch<128, SAGE_KV_INT8>(p, sms, st) : launch<128, SAGE_KV_E4M3>(p, sms, st);
  return kind == SAGE_KV_INT8 ? launch<64, SAGE_KV_INT8>(p, sms, st) : launch<64, SAGE_KV_E4M3>(p, sms, st);
}

}  // namespace sage
