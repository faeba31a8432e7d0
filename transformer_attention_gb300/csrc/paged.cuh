// The paged KV cache: what its kernels share.
//
// A layer's cache is a pool of pages, K_pages and V_pages [n_pages, P, H_kv,
// d_h] fp16, P a power of two.  Slot s of sequence b is row (s mod P) of page
// page_table[b, s / P]; lens[b] slots are filled, and a filled slot's position
// is its number.  The new tokens of sequence b are the rows [row_start[b],
// row_start[b + 1]) of packed arrays; token i goes to slot lens[b] + i.  Its
// parent is an earlier new token of the sequence or -1 (the filled slots), and
// its position is lens[b] + its depth; without parents each token follows the
// one before it.
//
// Everything of a batch but its sizes lies on the device, where the kernels
// check it: a sequence whose rows, length or pages do not fit counts as one
// without new tokens, a parent that is not earlier as -1, an entry of the page
// table outside the pool as a page that is not there, and each records
// kDevErrBadPaged.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace g3 {

constexpr int kPagedTile = 128;     // slots per tile of the attention
constexpr int kTreeMax = 64;        // new tokens of a sequence with parents: bits of a mask

struct PagedSeq {
  int row0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& p, int b, int* status) {
  PagedSeq s;
  s.row0 = __ldcg(p.row_start + b);
  const int r1 = __ldcg(p.row_start + b + 1);
  s.len = __ldcg(p.lens + b);
  s.n = r1 - s.row0;
  const long long slots = static_cast<long long>(p.max_pages) << p.page_shift;
  if (s.row0 < 0 || r1 < s.row0 || r1 > p.M || s.n > p.T_max || s.len < 0 ||
      static_cast<long long>(s.len) + s.n > slots) {
    record_error(status, kDevErrBadPaged);
    s.row0 = s.n = s.len = 0;
  }
  return s;
}

// Row of the pool that holds slot s of sequence b, or -1.
__device__ __forceinline__ int paged_row(const PagedBatch& p, int b, int s, int* status) {
  const int page = __ldcg(p.page_table + static_cast<size_t>(b) * p.max_pages + (s >> p.page_shift));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
    record_error(status, kDevErrBadPaged);
    return -1;
  }
  return (page << p.page_shift) + (s & ((1 << p.page_shift) - 1));
}

// The sequence whose rows hold row m (whole warp; -1: behind the last one): the
// first that ends behind m, among [b, e], of which each round leaves a 32nd.
__device__ __forceinline__ int paged_find(const PagedBatch& p, int m, int lane) {
  int b = 0, e = p.B;
  while (b < e) {
    const int step = (e - b + 31) >> 5, at = b + (lane + 1) * step - 1;
    const int k = __popc(__ballot_sync(0xffffffffu, at < e && __ldcg(p.row_start + at + 1) <= m));
    b += k * step;
    e = min(e, b + step - 1);
  }
  return b < p.B ? b : -1;
}

// The trees of a warp: lane l holds tokens l and 32 + l of one sequence.
struct Ancestors {
  uint32_t lo[2], hi[2];   // ancestors and the token itself, a bit each
  int parent[2];

  // Bits of token t (the same or another for every lane).
  __device__ __forceinline__ uint64_t of(int t) const {
    const uint32_t a = __shfl_sync(0xffffffffu, lo[0], t & 31), b = __shfl_sync(0xffffffffu, hi[0], t & 31);
    const uint32_t c = __shfl_sync(0xffffffffu, lo[1], t & 31), d = __shfl_sync(0xffffffffu, hi[1], t & 31);
    const uint32_t l = t & 32 ? c : a, h = t & 32 ? d : b;
    return static_cast<uint64_t>(h) << 32 | l;
  }
  __device__ __forceinline__ int parent_of(int t) const {
    const int a = __shfl_sync(0xffffffffu, parent[0], t & 31), b = __shfl_sync(0xffffffffu, parent[1], t & 31);
    return t & 32 ? b : a;
  }
};

// Ancestors of every new token of a sequence (whole warp), by pointer
// doubling: after round k a token has those up to 2^k steps away.
__device__ __forceinline__ Ancestors paged_ancestors(const PagedBatch& p, const PagedSeq& s, int lane,
                                                     int* status) {
  Ancestors a;
  int ptr[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    int q = i < s.n ? __ldcg(p.parents + s.row0 + i) : -1;
    if (q < -1 || q >= i) {
      if (i < s.n) record_error(status, kDevErrBadPaged);
      q = -1;
    }
    a.parent[u] = ptr[u] = q;
    a.lo[u] = u == 0 ? 1u << lane : 0u;
    a.hi[u] = u == 0 ? 0u : 1u << lane;
  }
  while (__any_sync(0xffffffffu, ptr[0] >= 0 || ptr[1] >= 0)) {
    uint64_t up[2];
    int next[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int q = max(ptr[u], 0);
      const uint64_t m = a.of(q);
      const int n0 = __shfl_sync(0xffffffffu, ptr[0], q & 31), n1 = __shfl_sync(0xffffffffu, ptr[1], q & 31);
      up[u] = ptr[u] >= 0 ? m : 0;
      next[u] = ptr[u] >= 0 ? (q & 32 ? n1 : n0) : -1;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      a.lo[u] |= static_cast<uint32_t>(up[u]);
      a.hi[u] |= static_cast<uint32_t>(up[u] >> 32);
      ptr[u] = next[u];
    }
  }
  return a;
}

// ---------------------------------------------------------------- work units
// A unit of the attention is a kv head of one sequence and 2^ts of its new
// tokens; its work are the 128-slot tiles from the first slot that one of
// these tokens may see to the last.  window 0: none.  ts is 5 to 8.
constexpr int kTileShift = 7;
static_assert(1 << kTileShift == kPagedTile, "tile");

struct PagedUnit {
  int lo, hi, tile0, tiles;   // visible slots [lo, hi), tiles [tile0, tile0 + tiles)
};

__host__ __device__ inline int paged_units(int n, int ts) { return (n + (1 << ts) - 1) >> ts; }

__host__ __device__ inline PagedUnit paged_unit(int len, int n, int window, bool tree, int ts, int q) {
  PagedUnit u;
  const int from = len + (tree ? 0 : q << ts) - window + 1;   // (a tree's tokens may have any depth)
  const int end = (q + 1) << ts;
  u.lo = window > 0 && from > 0 ? from : 0;
  u.hi = len + (end < n ? end : n);
  u.tile0 = u.lo >> kTileShift;
  u.tiles = ((u.hi + kPagedTile - 1) >> kTileShift) - u.tile0;
  return u;
}

// sum over i < N of floor((x + i 2^ts) / 128), x >= 0
__host__ __device__ inline long long paged_floor_sum(long long x, long long N, int ts) {
  if (ts > kTileShift) return N * (x >> kTileShift) + ((N * (N - 1) / 2) << (ts - kTileShift));
  // with k = 128 / 2^ts: the sum of floor(i / k) from c = floor(x / 2^ts) to c + N
  const int ks = kTileShift - ts;
  auto upto = [ks](long long i) {
    const long long d = i >> ks, r = i & ((1LL << ks) - 1);
    return ((d * (d - 1) / 2) << ks) + d * r;
  };
  const long long c = x >> ts;
  return upto(c + N) - upto(c);
}

// Tiles of the first q units (of one kv head) of a sequence.
__host__ __device__ inline long long paged_prefix(int len, int n, int window, bool tree, int ts, int q) {
  if (q <= 0 || n <= 0) return 0;
  if (n <= 1 << ts) return paged_unit(len, n, window, tree, ts, 0).tiles;
  const int nq = paged_units(n, ts);
  // last tiles, as if every unit were full
  long long sum = paged_floor_sum(static_cast<long long>(len) + (1 << ts) + kPagedTile - 1, q, ts);
  if (q >= nq)   // the last unit ends at n
    sum += ((static_cast<long long>(len) + n + kPagedTile - 1) >> kTileShift) -
           ((static_cast<long long>(len) + (static_cast<long long>(nq) << ts) + kPagedTile - 1) >> kTileShift);
  if (window > 0) {
    const long long from = static_cast<long long>(len) - window + 1;
    if (tree) {
      if (from > 0) sum -= q * (from >> kTileShift);
    } else {
      const long long i1 = from > 0 ? 0 : (-from >> ts) + 1;   // first unit whose lo is above 0
      if (i1 < q) sum -= paged_floor_sum(from + (i1 << ts), q - i1, ts);
    }
  }
  return sum;
}

// ---------------------------------------------------------------- whole shares
constexpr int kTileCost = 2;        // of a tile, in the shares of the work
constexpr int kMaxCtas = 160;       // CTAs of a launch at most (workspace)

// Units of all heads of a sequence; more than any launch has CTAs count as one more.
__host__ __device__ inline int paged_count_units(int n, int ts, int H_kv) {
  constexpr int most = kMaxCtas + 1;
  const int nq = paged_units(n, ts), units = H_kv * (nq < most ? nq : most);
  return units < most ? units : most;
}

// Tiles of a unit of a sequence at most: with a window no unit has more than the
// slots that its tokens reach.
__host__ __device__ inline int paged_most_tiles(int len, int n, int window, bool tree, int ts) {
  const int t = (len + n + kPagedTile - 1) >> kTileShift;
  if (window <= 0) return t;
  const int w = static_cast<int>((static_cast<long long>(window) + (tree ? n : 1 << ts) + 2 * kPagedTile) >> kTileShift);
  return t < w ? t : w;
}

// Tiles that a CTA does rather than having the units cut into `parts`: a part of
// 128 x 256 or 256 x 128 sums takes 65 ns of the device, written and added, a
// tile 1.6 us (128 units of 64 tiles, 27B-shaped: 118 us cut, 115 whole; of 20
// tiles 59 and 53).
__host__ __device__ constexpr int uncut_tiles(int parts) { return 3 + parts / 24; }

// What CTAs take whole: every unit (uncut), or shares of so many tiles from the
// first tile of every unit on (0: nothing).
struct PagedWhole {
  int tiles;
  bool uncut;
};

// all: the units' cost; units: the sum of paged_count_units; longest: of paged_most_tiles.
__host__ __device__ inline PagedWhole paged_whole(long long all, int units, int longest, int grid, int window) {
  const long long per_cta =
      all < 1 << 30 ? (static_cast<unsigned>(all) + static_cast<unsigned>(grid * kTileCost) - 1) / static_cast<unsigned>(grid * kTileCost)
                    : (all + grid * kTileCost - 1) / (grid * kTileCost);
  const long long parts = all / kTileCost < grid + units ? all / kTileCost : grid + units;
  PagedWhole w;
  w.uncut = units <= grid && longest <= per_cta + uncut_tiles(static_cast<int>(parts));
  w.tiles = window == 0 && all > 0 && !w.uncut ? static_cast<int>(per_cta) : 0;
  return w;
}

// Whole shares of every unit of a sequence (no window: a unit's tiles grow with its number).
__host__ __device__ inline int paged_whole_shares(const PagedWhole& w, int len, int n, int window, bool tree, int ts) {
  if (w.uncut) return n > 0 ? 1 : 0;
  return w.tiles == 0 || n == 0 ? 0 : paged_unit(len, n, window, tree, ts, 0).tiles / w.tiles;
}

}  // namespace g3
