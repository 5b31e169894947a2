// What the kernels over packed sequences share: the sequences, the tiles, and the line of work that is cut over
// the grid.
//
// The G query heads of a key/value head share its keys, so their rows lie in one tile: row r of a row tile is
// token r / G of the tile and head r % G, w = 128 / G tokens a tile (a tile has G w rows, 128 where G divides it).
// A unit is what one CTA accumulates without a join; it walks the unit's tiles:
//   kPairs  two row tiles against the key tiles that they see     (the forward)
//   kRows   one row tile against the same                         (dQ)
//   kKeys   one key tile (128 keys) against the row tiles that see it  (dK, dV)
// The units of a sequence follow each other, key/value head by head.  Every unit counts the tokens that it sees
// (kKeys: `per` times) and kUnitCost more, so that the line of all units can be cut into equal shares of time.  One warp
// of a CTA walks its share and hands the parts to the others (Feed).
#pragma once

#include <cuda_bf16.h>

#include "line.cuh"
#include "packed.h"
#include "ptx.cuh"
#include "tmap.h"

namespace sage {

constexpr int kPackedGroups = 512;

struct PackedShape {
  const int* cu;
  int* status;
  int T, S, Hkv, G, w, causal;
  int per;                  // kKeys: places a token, so that a row tile counts about what a key tile does
  unsigned inv_w, inv_pw;  // 2^32 / w, rounded up (w > 1); the same of per w
  __device__ __forceinline__ int over_w(int n) const { return w > 1 ? (int)__umulhi((unsigned)n, inv_w) : n; }  // n / w, n < 2^25
};

namespace {  // internal linkage: each translation unit keeps its own copy

constexpr int kDevSequence = 7;  // (kDevIndex of the cache calls: a number on the device is out of range)
constexpr int kTile = 128;
enum UnitKind { kPairs, kRows, kKeys };
template <int KIND>
// A unit's beginning and end, in places.  By measurement (64 to 768 tried): kPairs at 320 in place of 192 takes prompts of
// 17 to 2048 tokens from 123 to 129 us, 512 to 138 us; kRows and kKeys at 384 each take documents of 100 to 2048 tokens from
// 189 to 194 us, at 256 each D = 64 from 442 to 461 us.
constexpr int kUnitCost = KIND == kPairs ? 192 : KIND == kRows ? 384 : 192;

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1) / (unsigned)b); }

// One arrival of a warp, for all of its lanes (one of each lane queues up at the barrier)
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
  __syncwarp();
}

// first token and length of sequence b; one that does not lie in the tensors counts as empty
__device__ __forceinline__ void sequence(const PackedShape& p, int b, int& at, int& len) {
  const int x = __ldcg(p.cu + b), y = __ldcg(p.cu + b + 1);
  const bool ok = x >= 0 && y >= x && y <= p.T;
  if (!ok) atomicMax(p.status, kDevSequence);
  at = ok ? x : 0, len = ok ? y - x : 0;
}

// A sequence's units, for one key/value head
template <int KIND>
struct Units {
  int len, u;  // u: tokens of a unit
  const PackedShape& p;
  __device__ __forceinline__ Units(const PackedShape& p_, int len_)
      : len(len_), u(KIND == kPairs ? 2 * p_.w : KIND == kRows ? p_.w : kTile), p(p_) {}
  __device__ __forceinline__ int row_tiles() const { return p.over_w(len + p.w - 1); }
  __device__ __forceinline__ int count() const {
    return KIND == kKeys ? (len + kTile - 1) / kTile : KIND == kRows ? row_tiles() : (row_tiles() + 1) / 2;
  }
  // the first tile that unit i sees, of those of the sequence (kKeys; elsewhere 0)
  __device__ __forceinline__ int first(int i) const { return KIND == kKeys && p.causal ? p.over_w(i * kTile) : 0; }
  // tiles of unit i
  __device__ __forceinline__ int tiles(int i) const {
    if (KIND == kKeys) return row_tiles() - first(i);
    return ((p.causal ? min(len, (i + 1) * u) : len) + kTile - 1) / kTile;
  }
  // places of the line before unit i, and its own (tokens as if every unit were whole; below 2^50)
  __device__ __forceinline__ int per() const { return KIND == kKeys ? p.per : 1; }
  __device__ __forceinline__ long long before(int i) const {
    const long long all = (long long)i * ((long long)len * per() + kUnitCost<KIND>);
    if (!p.causal) return all;
    if (KIND == kKeys) return all - (long long)i * (i - 1) / 2 * (kTile * per());
    return (long long)i * (i + 1) / 2 * u + (long long)i * kUnitCost<KIND>;
  }
  __device__ __forceinline__ long long own(int i) const {
    return kUnitCost<KIND> + (long long)(!p.causal ? len : KIND == kKeys ? len - i * kTile : (i + 1) * u) * per();
  }
  __device__ __forceinline__ long long total() const { return before(count()); }
  // the unit that holds place x of a head: the root of before(i) = x, put right
  __device__ __forceinline__ int at(long long x) const {
    const float c = kUnitCost<KIND>, f = (float)x;
    float i;
    if (!p.causal) {
      i = f / ((float)len * per() + c);
    } else if (KIND == kKeys) {
      const float t = kTile * per(), a = (float)len * per() + c + t / 2;
      i = (a - sqrtf(fmaxf(0.f, a * a - 2 * t * f))) / t;
    } else {
      const float a = (float)u / 2 + c;
      i = (sqrtf(fmaf(a, a, 2 * (float)u * f)) - a) / (float)u;
    }
    int k = min(max((int)i, 0), count() - 1);
    while (k > 0 && before(k) > x) --k;
    while (k + 1 < count() && before(k + 1) <= x) ++k;
    return k;
  }
  // the tile of a unit where a cut at offset `off` is made: not within kSnap tiles of its ends, since each part costs
  // its way through memory and the join (6 in place of 3: gradients of 4 documents 35.3 us, not 32.2 us, the others within
  // 2%; the forward counts on 2 at least, so that both row tiles of a unit have tiles in each part)
  __device__ __forceinline__ int cut(long long off, int n) const {
    if (off <= 0) return 0;
    const int c = KIND != kKeys ? (int)min(off / kTile, (long long)n)
                  : off < (1 << 25) ? (int)__umulhi((unsigned)off, p.inv_pw) : (int)min(off / (p.per * p.w), (long long)n);
    return c >= n - kSnap ? n : c <= kSnap ? 0 : c;
  }
  static constexpr int kSnap = 3;
  static_assert(kSnap >= 2, "a part's tiles of both row tiles");
};

// places of all of sequence b's units, and its tokens
template <int KIND>
__device__ __forceinline__ long long places(const PackedShape& p, int b, int& len) {
  int at;
  sequence(p, b, at, len);
  return len > 0 ? Units<KIND>(p, len).total() * p.Hkv : 0;
}

// The line of all units, cut into equal parts for the CTAs of a grid, of kLeast places at least: two cuts must not fall into
// one tile, and a part of fewer than four key tiles would be mostly beginning and end (not measured against 256, which would
// do for the first; short calls leave CTAs without work by it: 700 tokens of 32 heads of 8 take 99 of 152).
constexpr int kLeast = 512;
static_assert(kLeast >= 2 * kTile, "a tile between two cuts");
struct Shares {
  long long total, each;
  int parts, rest;
  __device__ __forceinline__ Shares(long long total_, int most) : total(total_) {
    parts = (int)min((long long)most, max(total / kLeast, 1ll));
    each = total / parts;
    rest = (int)(total - each * parts);
  }
  // where part v begins
  __device__ __forceinline__ long long start(int v) const { return each * v + (unsigned)(rest * v) / (unsigned)parts; }
};

// A part of a unit: tiles [c0, c1) of its n, of key/value head hk of the sequence at token `at`.  c1 = 0: no more parts.
// A unit that was cut has parts with the workers `first`, .. `first` + parts - 1, who leave their sums at places: that
// of the unit's beginning at 2 first + 1, the others at 2 w.  (A worker has two such parts at most: its first and its last.)
struct Part {
  int at, len, hk, i, n, c0, c1, cut;  // cut: first << 16 | parts
  __device__ __forceinline__ bool whole() const { return c0 == 0 && c1 == n; }
  __device__ __forceinline__ int first() const { return cut >> 16; }
  __device__ __forceinline__ int parts() const { return cut & 0xffff; }
  __device__ __forceinline__ int place(int k) const { return 2 * (first() + k) + (k == 0 ? 1 : 0); }  // of part k
  __device__ __forceinline__ int place() const { return 2 * blockIdx.x + (c0 == 0 ? 1 : 0); }         // of this one
};

// A worker's way along the line: the parts from place `begin` to `end`, in order.  All lanes of a warp walk together.
template <int KIND>
struct Walk {
  long long stop, unit_at;  // places: where the walk ends, where the unit at hand begins
  int b, at, len, hk, i, c0;
  bool more;
  __device__ __forceinline__ Walk(const PackedShape& p, const long long* pre, int group, long long begin, long long end)
      : stop(end), unit_at(0), b(0), at(0), len(0), hk(0), i(0), c0(0), more(begin < end) {
    if (!more) return;
    const int lane = threadIdx.x & 31;
    const int g = row_at(pre, kPackedGroups, begin);
    long long base = pre[g];
    b = g;
    if (group > 1) {
      // the sequence, 32 of the group at a time
      const int end_b = min(p.S, (g + 1) * group);
      b = end_b;
      for (int b0 = g * group; b0 < end_b; b0 += 32) {
        int n;
        long long s = b0 + lane < end_b ? places<KIND>(p, b0 + lane, n) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += x;
        }
        const int k = __popc(__ballot_sync(0xffffffffu, base + s <= begin));
        const long long before = __shfl_sync(0xffffffffu, s, max(k - 1, 0));
        if (k > 0) base += before;
        b = min(end_b, b0 + k);
        if (k < 32) break;
      }
    }
    if (b < p.S) sequence(p, b, at, len);
    if (len <= 0) {  // (not while the sequences stand still)
      more = false;
      return;
    }
    const Units<KIND> us(p, len);
    const long long head = us.total();
    hk = min((int)((float)(begin - base) / (float)head), p.Hkv - 1);
    while (hk > 0 && hk * head > begin - base) --hk;
    while (hk + 1 < p.Hkv && (hk + 1) * head <= begin - base) ++hk;
    base += hk * head;
    i = us.at(begin - base);
    unit_at = base + us.before(i);
    const int n = us.tiles(i);
    c0 = us.cut(begin - unit_at, n);
    if (c0 >= n) advance(p);
    settle(p);
  }
  // to the next unit
  __device__ __forceinline__ void advance(const PackedShape& p) {
    const Units<KIND> us(p, len);
    unit_at += us.own(i);
    c0 = 0;
    if (++i < us.count()) return;
    i = 0;
    if (++hk < p.Hkv) return;
    hk = 0;
    do {
      if (++b >= p.S) {
        more = false;
        return;
      }
      sequence(p, b, at, len);
    } while (len <= 0);
  }
  // whether anything of the unit at hand lies before the end
  __device__ __forceinline__ void settle(const PackedShape& p) {
    if (!more) return;
    const Units<KIND> us(p, len);
    if (us.cut(stop - unit_at, us.tiles(i)) <= c0) more = false;
  }
  __device__ __forceinline__ Part next(const PackedShape& p, const Shares& line) {
    const Units<KIND> us(p, len);
    const int n = us.tiles(i);
    Part s{at, len, hk, i, n, c0, us.cut(stop - unit_at, n), 0};
    if (!s.whole()) {
      int v = blockIdx.x;
      if (c0 > 0)
        while (v > 0 && us.cut(line.start(v) - unit_at, n) > 0) --v;
      int last = v;
      while (last + 1 < line.parts && us.cut(line.start(last + 1) - unit_at, n) < n) ++last;
      s.cut = v << 16 | (last - v + 1);
    }
    if (s.c1 < n) {
      more = false;
    } else {
      advance(p);
      settle(p);
    }
    return s;
  }
};

constexpr int kMaxParts = 160;  // CTAs of a grid (one an SM)

// The parts, from the warp that walks to those that work: a ring in shared memory.
constexpr int kRing = 8;
struct FeedRing {
  alignas(16) Part part[kRing];
  uint64_t full[kRing], empty[kRing];
  __device__ __forceinline__ void init(int readers) {  // (warps)
    for (int x = 0; x < kRing; ++x) {
      mbar_init(&full[x], 1);
      mbar_init(&empty[x], readers);
    }
  }
};

// The walking warp's part: everything of its CTA's share.
template <int KIND>
__device__ __forceinline__ void feed(const PackedShape& p, FeedRing& ring, const long long* pre, int group, const Shares& line,
                                     bool idle, volatile int* abort) {
  const int w0 = blockIdx.x, lane = threadIdx.x & 31;
  Walk<KIND> walk(p, pre, group, idle ? 0 : line.start(w0), idle ? 0 : line.start(w0 + 1));
  for (uint32_t n = 0;; ++n) {
    const bool more = walk.more;
    Part s{};
    if (more) s = walk.next(p, line);
    const uint32_t x = n % kRing;
    if (n >= kRing && !mbar_wait_warp(&ring.empty[x], (n / kRing - 1) & 1, abort)) return;
    if (lane == 0) {
      ring.part[x] = s;
      mbar_arrive(&ring.full[x]);
    }
    __syncwarp();
    if (!more) return;
  }
}

// A working warp's view: next() is false behind the last part, or after a wait that ran out.
struct Feed {
  FeedRing& ring;
  volatile int* abort;
  uint32_t n = 0;
  __device__ __forceinline__ Feed(FeedRing& ring_, volatile int* abort_) : ring(ring_), abort(abort_) {}
  __device__ __forceinline__ bool next(Part& s) {
    const uint32_t x = n % kRing;
    if (!mbar_wait_warp(&ring.full[x], (n / kRing) & 1, abort)) return false;
    const int4* from = reinterpret_cast<const int4*>(&ring.part[x]);
    const int4 a = from[0], b = from[1];
    s = Part{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ring.empty[x]);
    ++n;
    return s.c1 > 0;
  }
};

// The joining of a unit that was cut, by those who finish its last part (in time, whichever it is): a group of
// warps has written its part's sums; true in all of them if it was the last to do so.  Sums are then added in the order
// of the parts, so the bits do not depend on who came last.  The counter is zero before and after.  The lane that counts
// has fences of its own on both sides: the sums of the other warps, which it knows of by `written`, go out with its count,
// and what the other parts' counts brought is there for those that it tells.
struct Meeting {
  uint64_t written, told;
  int last;
  __device__ __forceinline__ void init(int warps) {
    mbar_init(&written, warps);
    mbar_init(&told, 1);
  }
  // n: how often the group has met here before; leads: whether the warp is the group's first
  __device__ __forceinline__ bool was_last(int* counter, int parts, uint32_t n, bool leads, volatile int* abort, bool& ok) {
    __threadfence();
    warp_arrive(&written);
    if (leads) {
      ok = ok && mbar_wait_warp(&written, n & 1, abort);
      if (ok && (threadIdx.x & 31) == 0) {
        __threadfence();
        last = atomicAdd(counter, 1) == parts - 1;
        __threadfence();
        if (last) atomicExch(counter, 0);
        mbar_arrive(&told);
      }
      __syncwarp();
    }
    ok = ok && mbar_wait_warp(&told, n & 1, abort);
    __threadfence();
    return ok && *const_cast<volatile int*>(&last);
  }
};
// words of the workspace's header behind the status word: whether packed_dkv has seen packed_pre's results (pdl_tell), and
// counters
constexpr int kTermsTold = 32;
constexpr int kCounters = 2 * kMaxParts;  // of each kernel: two of each worker
enum { kFwdCounters = 64, kKeyCounters = kFwdCounters + kCounters, kRowCounters = kKeyCounters + kCounters,
       kHeader = kRowCounters + kCounters };  // in words
static_assert(kHeader == 1024, "the workspace's first 4096 bytes");

// Sums of a part: float4 of four channels, [D / 4][128 rows], so that a warp's threads, a row each, meet in memory
__device__ __forceinline__ void store_sums(float* part, int d, int r, const uint32_t (&o)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4)
    *reinterpret_cast<uint4*>(part + (size_t)((d + e) * kTile + r * 4)) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
}
// o += f * those
__device__ __forceinline__ void add_sums(const float* part, int d, int r, float f, float (&o)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(part + (size_t)((d + e) * kTile + r * 4)));
    o[e] = fmaf(x.x, f, o[e]), o[e + 1] = fmaf(x.y, f, o[e + 1]);
    o[e + 2] = fmaf(x.z, f, o[e + 2]), o[e + 3] = fmaf(x.w, f, o[e + 3]);
  }
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Rows of bf16 to memory, a thread a row.  Four neighbours exchange 16-byte pieces so that each store of a warp writes 64
// bytes of eight rows, not 16 of 32 (half sectors, a line each).
struct RowStore {
  __nv_bfloat16* to[4];  // of the four's rows; null: not stored
  __device__ __forceinline__ explicit RowStore(__nv_bfloat16* row) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      to[s] = reinterpret_cast<__nv_bfloat16*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), (threadIdx.x & 28) + s));
  }
  // channels [d, d + 32) times f (all lanes of the warp)
  __device__ __forceinline__ void put(const float (&o)[32], int d, float f) const {
    uint32_t u[4][4];
#pragma unroll
    for (int e = 0; e < 32; e += 2) u[e >> 3][(e >> 1) & 3] = bf2(o[e] * f, o[e + 1] * f);
    auto swap = [&](uint32_t (&x)[4], uint32_t (&y)[4], int bit) {
      const bool up = threadIdx.x & bit;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[e] : y[e], bit);
        x[e] = up ? got : x[e];
        y[e] = up ? y[e] : got;
      }
    };
    swap(u[0], u[1], 1);
    swap(u[2], u[3], 1);
    swap(u[0], u[2], 2);
    swap(u[1], u[3], 2);
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (to[s]) *reinterpret_cast<uint4*>(to[s] + d + 8 * (threadIdx.x & 3)) = make_uint4(u[s][0], u[s][1], u[s][2], u[s][3]);
  }
};

// pre[g]: the places before each group of sequences, and their number behind the last; `tokens`, zero before: of all
// sequences (all threads of the CTA, which must synchronise before they read either).  Every CTA sums all of them: the forward
// of 512 empty sequences takes 3.4 us, of 4096 9.4 us, of 65536 121 us (of one token each, 8 heads of 2: 1.8 ms).
template <int KIND, int NT>
__device__ __forceinline__ void prefix_of_sequences(const PackedShape& p, int group, long long* pre, long long* wsum,
                                                    unsigned long long* tokens) {
  unsigned long long sum = 0;
  prefix_of<NT>(kPackedGroups, pre, wsum, [&](int g) {
    long long n = 0;
#pragma unroll 1
    for (int b = g * group; b < min(p.S, (g + 1) * group); ++b) {
      int len;
      n += places<KIND>(p, b, len);
      sum += len;
    }
    return n;
  });
  if (sum) atomicAdd(tokens, sum);
}
// Sequences that lie over one another (cu_seqlens out of order) could be any amount of work: beyond twice the tensors'
// tokens none of it is done.
__device__ __forceinline__ bool too_many(const PackedShape& p, unsigned long long tokens) {
  return tokens > 2 * (unsigned long long)p.T;
}

inline PackedShape packed_shape(const int* cu, void* ws, int T, int S, int H, int Hkv, int causal) {
  const int G = H / Hkv;
  const int w = kTile / G, per = kTile / w;
  auto inverse = [](int n) { return n > 1 ? (unsigned)(((1ull << 32) + n - 1) / n) : 0u; };
  return PackedShape{cu, static_cast<int*>(ws), T, S, Hkv, G, w, causal, per, inverse(w), inverse(per * w)};
}

// Row tiles of queries: w tokens of the G heads of a key/value head, 64 channels
inline bool make_tmap_queries(CUtensorMap* map, const sage_rows& x, int D, int H, const PackedShape& s) {
  const cuuint64_t one = (cuuint64_t)D * 2;  // (the stride of an axis of one)
  return encode_tmap_3d(map, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)s.T},
                        {H > 1 ? (cuuint64_t)x.head * 2 : one, s.T > 1 ? (cuuint64_t)x.token * 2 : one},
                        {64, (cuuint32_t)s.G, (cuuint32_t)s.w}, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Key tiles: 128 tokens of a key/value head, 64 channels
inline bool make_tmap_keys(CUtensorMap* map, const sage_rows& x, int D, const PackedShape& s) {
  const cuuint64_t one = (cuuint64_t)D * 2;
  return encode_tmap_3d(map, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, {(cuuint64_t)D, (cuuint64_t)s.T, (cuuint64_t)s.Hkv},
                        {s.T > 1 ? (cuuint64_t)x.token * 2 : one, s.Hkv > 1 ? (cuuint64_t)x.head * 2 : one}, {64, kTile, 1},
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

}  // namespace sage
