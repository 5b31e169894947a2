// What the kernels over packed sequences share: the sequences, the tiles, and the line of work that is cut over
// the grid.
//
// The G query heads of a key/value head share its keys, so their rows lie in one tile: row r of a row tile is
// token r / G of the tile and head r % G, w = 128 / G tokens a tile (a tile has G w rows, 128 where G divides it).
// A unit is what one CTA accumulates without a join; it walks the unit's tiles:
//   kPairs  two row tiles against the key tiles that they see     (the forward)
//   kRows   one row tile against the same                         (dQ)
//   kKeys   one key tile (128 keys) against the row tiles that see it  (dK, dV)
// The units of a sequence follow each other, key/value head by head; every unit counts its tiles and kUnitCost
// more, so that the line of all units can be cut into equal shares of time.
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
};

namespace {  // internal linkage: each translation unit keeps its own copy

constexpr int kDevSequence = 7;  // (kDevIndex of the cache calls: a number on the device is out of range)
constexpr int kTile = 128;
constexpr int kUnitCost = 1;

enum UnitKind { kPairs, kRows, kKeys };

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1) / (unsigned)b); }

// first token and length of sequence b; one that does not lie in the tensors counts as empty
__device__ __forceinline__ void sequence(const PackedShape& p, int b, int& at, int& len) {
  const int x = __ldcg(p.cu + b), y = __ldcg(p.cu + b + 1);
  const bool ok = x >= 0 && y >= x && y <= p.T;
  if (!ok) atomicMax(p.status, kDevSequence);
  at = ok ? x : 0, len = ok ? y - x : 0;
}

// sum of floor((a i + b) / m) over i < n, by exchanging the roles of the two axes as in Euclid's algorithm
// (a n + b stays below 2^31 here)
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned a, unsigned b, unsigned m) {
  long long sum = 0;
#pragma unroll 1
  while (n) {
    if (a >= m) {
      sum += (long long)n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += (long long)n * (b / m);
      b %= m;
    }
    const unsigned y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const unsigned x = m;
    m = a;
    a = x;
  }
  return sum;
}

// A sequence's units, for one key/value head
template <int KIND>
struct Units {
  int len, u;  // u: tokens of a unit
  int causal, w;
  __device__ __forceinline__ Units(const PackedShape& p, int len_)
      : len(len_), u(KIND == kPairs ? 2 * p.w : KIND == kRows ? p.w : kTile), causal(p.causal), w(p.w) {}
  __device__ __forceinline__ int count() const { return ceil_div(len, u); }
  // the first tile that unit i sees, of those of the sequence (kKeys; elsewhere 0)
  __device__ __forceinline__ int first(int i) const { return KIND == kKeys && causal ? i * kTile / w : 0; }
  // tiles of unit i
  __device__ __forceinline__ int tiles(int i) const {
    if (KIND == kKeys) return ceil_div(len, w) - first(i);
    return ceil_div(causal ? min(len, (i + 1) * u) : len, kTile);
  }
  // places of the line before unit i
  __device__ __forceinline__ long long before(int i) const {
    long long n = (long long)i * kUnitCost;
    if (i == 0) return n;
    if (!causal) return n + (long long)i * tiles(0);
    if (KIND == kKeys) return n + (long long)i * ceil_div(len, w) - floor_sum(i, kTile, 0, w);
    const bool all = i == count();  // (the last unit ends with the sequence)
    return n + floor_sum(all ? i - 1 : i, u, u + kTile - 1, kTile) + (all ? ceil_div(len, kTile) : 0);
  }
  __device__ __forceinline__ long long total() const { return before(count()); }
};

// places of all of sequence b's units
template <int KIND>
__device__ __forceinline__ long long places(const PackedShape& p, int b) {
  int at, len;
  sequence(p, b, at, len);
  return len > 0 ? Units<KIND>(p, len).total() * p.Hkv : 0;
}

// Where a cut at offset `off` of a unit of n tiles is made: not within kSnap tiles of its ends, since each part costs
// its way through memory and the join.
constexpr int kSnap = 2;
__device__ __forceinline__ int snap(long long off, int n) {
  if (off >= n) return n;
  return off <= kSnap ? 0 : off >= n - kSnap ? n : (int)off;
}

// A part of a unit: tiles [c0, c1) of its n, of key/value head hk of the sequence at token `at`.
struct Part {
  int b, at, len, hk, i, n, c0, c1;
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
    // the sequence, 32 of the group at a time
    long long base = pre[g];
    const int end_b = min(p.S, (g + 1) * group);
    b = end_b;
    for (int b0 = g * group; b0 < end_b; b0 += 32) {
      long long s = b0 + lane < end_b ? places<KIND>(p, b0 + lane) : 0;
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
    if (b >= end_b) {  // (not reached while the sequences stand still)
      more = false;
      return;
    }
    sequence(p, b, at, len);
    const Units<KIND> us(p, len);
    const long long head = us.total();
    hk = (int)mul_div(begin - base, 1, head);
    base += hk * head;
    // the unit, by a search with a place for each lane
    int lo = 0, hi = us.count();
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, c = lo + (lane + 1) * step;
      const int k = __popc(__ballot_sync(0xffffffffu, c < hi && base + us.before(c) <= begin));
      hi = min(hi, lo + (k + 1) * step);
      lo += k * step;
    }
    i = lo;
    unit_at = base + us.before(lo);
    const int n = us.tiles(lo);
    c0 = snap(begin - unit_at, n);
    if (c0 >= n) advance(p, n);
    settle(p);
  }
  // to the next unit
  __device__ __forceinline__ void advance(const PackedShape& p, int n) {
    unit_at += n + kUnitCost;
    c0 = 0;
    if (++i < Units<KIND>(p, len).count()) return;
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
    const long long off = stop - unit_at;
    if (off <= 0 || snap(off, Units<KIND>(p, len).tiles(i)) <= c0) more = false;
  }
  __device__ __forceinline__ Part next(const PackedShape& p) {
    const int n = Units<KIND>(p, len).tiles(i);
    Part s{b, at, len, hk, i, n, c0, n};
    const long long off = stop - unit_at;
    if (off < n + kUnitCost) s.c1 = snap(off, n);
    if (s.c1 < n) {
      more = false;
    } else {
      advance(p, n);
      settle(p);
    }
    return s;
  }
};

// A unit that was cut, written by the worker behind its first cut: its parts are those of the workers before, where it
// begins, to `last`.  Worker x leaves its part of a unit at place 2 x + 1 if the unit begins with it, else 2 x.
struct Cut {
  int b, hk, i, last;  // b < 0: no such unit
};
constexpr int kMaxParts = 160;  // CTAs of a grid (one an SM)

// The record of worker w0, whose walk stands at its beginning
template <int KIND>
__device__ __forceinline__ Cut first_cut(const PackedShape& p, const Line& line, const Walk<KIND>& walk, int w0) {
  Cut c{-1, 0, 0, 0};
  if (!walk.more || walk.c0 == 0) return c;
  const int n = Units<KIND>(p, walk.len).tiles(walk.i);
  const long long before = line.start(w0 - 1) - walk.unit_at;
  if (before > 0 && snap(before, n) > 0) return c;  // (it lies in the unit too)
  int last = w0;
  while (last + 1 < line.parts) {
    const long long off = line.start(last + 1) - walk.unit_at;
    if (off >= n || snap(off, n) == n) break;
    ++last;
  }
  return Cut{walk.b, walk.hk, walk.i, last};
}
// what a join may read (after a wait that ran out records are whatever the workspace held)
__device__ __forceinline__ bool was_cut(const PackedShape& p, const Cut& c, int w0) {
  return c.b >= 0 && c.b < p.S && (unsigned)c.hk < (unsigned)p.Hkv && c.i >= 0 && c.last >= w0 && w0 > 0 && c.last < kMaxParts;
}

// pre[g]: the places before each group of sequences, and their number behind the last (all threads of the CTA, which
// must synchronise before they read it)
template <int KIND, int NT>
__device__ __forceinline__ void prefix_of_sequences(const PackedShape& p, int group, long long* pre, long long* wsum) {
  prefix_of<NT>(kPackedGroups, pre, wsum, [&](int g) {
    long long n = 0;
#pragma unroll 1
    for (int b = g * group; b < min(p.S, (g + 1) * group); ++b) n += places<KIND>(p, b);
    return n;
  });
}

inline PackedShape packed_shape(const int* cu, void* ws, int T, int S, int H, int Hkv, int causal) {
  const int G = H / Hkv;
  return PackedShape{cu, static_cast<int*>(ws), T, S, Hkv, G, kTile / G, causal};
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
