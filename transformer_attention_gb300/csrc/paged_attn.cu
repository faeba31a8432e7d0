// Attention of a batch's new tokens (steps, drafted trees, chunks) over the
// paged KV cache (paged.cuh), on the tcgen05 tensor cores.
//
//   O[i, h] = sum_s p_s v_s,  p = softmax of q . k_s over the slots s that token
//   i sees: the filled ones within its window, its ancestors and itself
//
// A work unit is a kv head of one sequence and up to NQ query tiles of 128 rows
// (128 / G tokens x the G heads); a step or a tree fills a few rows of one tile.
// Below some 280 rows per kv head the cache's bytes bound the call, above them
// the tensor cores, so one kernel serves both: the cache streams through a
// ring of 32 KB parts, 160 KB in flight per SM, and each 128-slot tile costs 1100
// (d_h = 128) or 2200 clocks of MMA however few its rows, against 2800 or 5600
// for its bytes at the HBM rate.  Measured: a token over 131071 slots, 27B-shaped,
// 158 to 163 us (1.07 GB: 97 to 100% of the copy rate); 1024 tokens over 31744 slots
// 385 to 397 us with the clocks that the power limit leaves (1.36 to 1.41 PFLOP/s:
// of a tile pair's 3100 clocks 2048 are MMA).
//
// Sequences have lengths of their own, known on the device alone: each CTA adds
// up the work of all units and takes an equal share of it, cut wherever it
// falls (a unit's parts are then added by paged_merge_kernel, always in the
// same order).  Units of one kv head read the same slots: where units are longer
// than a share, CTAs take whole shares from a unit's first tile on, so that the
// units of a head run side by side and read their slots from L2 (1024 tokens
// over 31744 slots, 27B-shaped: 2.1 GB from DRAM without this), and the other
// CTAs share out what is left of the units.
//
// Warps:
//   0, 3   TMA of K and V, half of every part each: a copy costs its warp some
//          100 clocks, and pages of 16 slots take 24 (d_h = 128) or 40 per tile
//   1      TMEM allocation and MMA issue
//   2      the CTA's pieces of units, published through a ring, and TMA of Q
//   4-7    softmax of query tile 0, one thread per row (NQ = 2: its epilogue too)
//   8-11   NQ = 2: the same of query tile 1; NQ = 1: the epilogue, so that the
//          softmax goes on with the next piece
// TMEM: NQ = 1: S of even and odd tiles at 0 and 128; NQ = 2: S of query tile e
// at 128 e.  P (fp16 pairs) is written over the first 64 columns of its S.  O
// from column 256.
// Slots outside [lo, hi) of a unit are left out of the product with V, 16 at a
// time, or zeroed in its tile, so that what they hold (a NaN, say) cannot reach
// O through a zero probability.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "attention_common.cuh"
#include "paged.cuh"

namespace g3 {

namespace {

using attn::ex2;

constexpr int BM = 128, BN = kPagedTile;
constexpr uint32_t CHUNK = 128 * 128;       // 128 rows x 64 channels (128 B), swizzled
constexpr uint32_t PART = 32768;
constexpr uint32_t QSMALL = 32 * 128;       // 32 rows of a chunk: Q of few rows (the MMA reads on behind them)
constexpr uint32_t O_COL = 256;
constexpr float LOG2E = 1.4426950408889634f;
// A row's reference stays P_SHIFT below a past maximum while the present one
// is less than RESCALE_THRESHOLD above that (log2 units): the probabilities
// that are rounded to fp16 reach 2^15, so that those below its normal range, off
// by 2^-25, are off by 2^-32 at most of the row's largest.
constexpr float RESCALE_THRESHOLD = 8.0f, P_SHIFT = 7.0f;
constexpr int NPC = 4;                      // ring of pieces
constexpr int kMaxCluster = 16, kMergeTiles = 8;
constexpr int kMaxSlots = 1 << 30;          // of a sequence (validate_paged_sizes)

enum : int {
  kSiteQFull = 100, kSiteQEmpty, kSitePartFull, kSitePartEmpty, kSiteSFull, kSitePFull, kSitePvDone,
  kSiteOFinal, kSiteOFree, kSitePieceFull, kSitePieceEmpty, kSiteStatFull, kSiteStatEmpty
};

// A CTA's piece of a unit.  tiles 0: no more pieces.
struct alignas(16) Piece {
  int b, j, row0, ntok;     // packed row of the unit's first token, its tokens
  int i0, n, len, lo;       // number of that token, the sequence's new tokens and length; visible slots
  int hi, tile0, tiles, slot;   // slot: of its part in the workspace, -1: the whole unit
};

// Slots of parts: CTA c's first piece, if it begins inside a unit, has slot 2c,
// its last, if it ends inside one, 2c + 1; what is left of a unit behind its
// whole shares, the first of them CTA c's, has slot kRest + c if one piece
// holds it.
constexpr int kRest = 2 * kMaxCtas, kSlots = 3 * kMaxCtas;

// The unit whose first piece is a CTA's and that has others (parts 0: none).
struct alignas(16) Split {
  int row0, ntok, j, parts;
  int cta, shares;          // whole shares, of CTAs cta ..
  int rest, inside;         // the others: of CTAs rest .., or all in one piece

  __device__ __forceinline__ int slot(int i) const {
    if (i < shares) return 2 * (cta + i);
    if (inside) return kRest + cta;
    return i == shares ? 2 * rest + 1 : 2 * (rest + i - shares);
  }
};

struct Shared {
  uint64_t q_full[2], q_empty[2], part_full[8], part_empty[8], s_full[2], p_full[2], pv_done[2],
      o_final[2], o_free[2], stat_full[2], stat_empty[2], piece_full[NPC], piece_empty[NPC], drain;
  Piece piece[NPC];
  float2 stat[2][BM];     // NQ = 1: (reference, sum) of a piece's rows
  long long warp_sum[12];
  int warp_most[12], warp_units[12];
  long long start_off, start_base;   // of this CTA's share in its first sequence, which begins there
  int start_taken;        // whole shares before that sequence
  int unit_rows, unit_row0, unit_parts;   // of the cluster's unit
  int start_b, first_used, first_j;   // first_used: cost of the piece that is there already
  PagedSeq start_seq;
  uint32_t tmem;
  int abort_flag;
};

// Bounded wait for a phase; false after a timeout, whose site goes to *lost (it
// is recorded once, when the role ends), or when another thread gave up.  The
// roles share the instruction cache, so the waits are kept small.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site,
                                         int* lost) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (globaltimer() - t0 > kWaitTimeoutNs) {
      *lost = site;
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

template <int DH, int NQ_>
struct Cfg {
  static constexpr int NQ = NQ_;
  static_assert(NQ == 1 || DH == 128, "TMEM columns");
  static constexpr int NCH = DH / 64;
  static constexpr int PARTS = DH / 128;          // parts of a K or V tile
  static constexpr uint32_t QT_BYTES = BM * DH * 2;
  // Ring: five parts, 160 KB in flight.  The HBM serves some SMs worse the more
  // all of them ask for at once (a token over 131071 slots, 27B-shaped: 169 us with
  // six parts, 161.5 with five or four, 167 with three).
  static constexpr int NP = 5;
  static constexpr uint32_t SMEM = NQ * QT_BYTES + NP * PART + sizeof(Shared);
  static_assert(NQ * QT_BYTES + NP * PART <= 7 * PART && SMEM <= 232448, "shared memory budget");
  // What a unit costs besides its tiles, in halves of a tile: of units of few
  // rows alone, and where units of chunks and of steps meet (eight mixed 4B-shaped
  // batches: 56.7 us on average with 10, 54.2 with 6, 53.8 with 4).
  static constexpr int UC1 = 3, UCG = 5;
  static constexpr int THREADS = 384;
  // the control warps give registers to the others
  static constexpr int REGS_LAUNCH = 168, REGS_CTRL = NQ == 2 ? 104 : 120, REGS_SOFT = NQ == 2 ? 200 : 216;
  static constexpr int REGS_OTHER = NQ == 2 ? 200 : 168;   // warps 8-11
  static constexpr int REGS_SPLIT = 128 * (REGS_CTRL + REGS_SOFT + REGS_OTHER);
  static_assert(REGS_SPLIT <= THREADS * REGS_LAUNCH, "register split");
};

struct Params {
  PagedBatch batch;
  float2* pstat;          // [kSlots, rows] (reference, sum)
  float4* part;           // [kSlots, DH / 4, rows] unnormalised, 4 channels each
  Split* split;           // [grid]
  void* O;
  int o_f16, H, H_kv, gshift, window, ts, tokbox, rows, qsmall, vshift;   // ts: log2 of a unit's tokens, vshift: of a V box's slots
  int units;              // of a head, where clusters take them
  uint32_t zero;          // 0, which the compiler does not know
  int* status;
};

struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// exp2(s log2 e - m) of 32 columns: packed fp16 pairs to p[0..15], sums to acc.
__device__ __forceinline__ void exp_pack(const uint32_t (&s)[32], uint32_t* p, float2 (&acc)[4],
                                         float2 l2e, float2 negm) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 x = __ffma2_rn(
        make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), l2e, negm);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    acc[k & 3] = __fadd2_rn(acc[k & 3], e);
    p[k] = pack_half2(e.x, e.y);
  }
}

// Bits [a, z] of 32, for any a and z.
__device__ __forceinline__ uint32_t bits_from_to(int a, int z) {
  const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : 0xffffffffu << a);
  return from & (z < 0 ? 0u : (z >= 31 ? 0xffffffffu : (2u << z) - 1u));
}

// Bits [d, d + 32) of a mask, for any d.
__device__ __forceinline__ uint32_t bits_at(uint64_t m, int d) {
  if (d >= 0) return d < 64 ? static_cast<uint32_t>(m >> d) : 0u;
  return d > -32 ? static_cast<uint32_t>(m << -d) : 0u;
}

// A lane's running sums: reference, sum, VV vectors.
template <int VV>
struct MergeAcc {
  float m = -INFINITY, l = 0.f;
  float4 o[VV];

  __device__ __forceinline__ void add(float2 st, const float4 (&x)[VV]) {
    if (st.y == 0.f) return;                       // saw nothing
    const float to = fmaxf(m, st.x);
    const float fm = m == to ? 1.f : ex2(m - to), fx = ex2(st.x - to);
    m = to;
    l = l * fm + st.y * fx;
#pragma unroll
    for (int v = 0; v < VV; ++v) {
      o[v].x = o[v].x * fm + x[v].x * fx;
      o[v].y = o[v].y * fm + x[v].y * fx;
      o[v].z = o[v].z * fm + x[v].z * fx;
      o[v].w = o[v].w * fm + x[v].w * fx;
    }
  }

  // A vector's four channels over the sum, packed.
  __device__ __forceinline__ uint2 packed(int v, float inv, int f16) const {
    const float a = o[v].x * inv, b = o[v].y * inv, c = o[v].z * inv, d = o[v].w * inv;
    return f16 ? make_uint2(pack_half2(a, b), pack_half2(c, d)) : make_uint2(pack_bf162(a, b), pack_bf162(c, d));
  }
};

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The descriptor of a tile `bytes` (a multiple of 16) behind that of `base`: the
// addresses stay below 2^18, so that their sum does not leave its field.
__device__ __forceinline__ uint64_t sdesc_plus(uint64_t base, uint32_t bytes) {
  return (base & 0xffffffff00000000ull) | (static_cast<uint32_t>(base) + (bytes >> 4));
}

// How a launch's CTAs take their work.
enum : int {
  kAnyUnits,      // equal shares of all units' work
  kOneUnit,       // the same where the new tokens of every sequence fit one unit per head
  kClusterUnit    // one unit of one query tile per cluster, whose CTAs add their parts through distributed
                  // shared memory
};

template <int DH, int NQ, int MODE>
__global__ void __launch_bounds__(Cfg<DH, NQ>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQ32,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<DH, NQ>;
  constexpr bool ONE = MODE != kAnyUnits, CLUSTER = MODE == kClusterUnit;
  static_assert(NQ == 1 || !CLUSTER, "few rows");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& batch = p.batch;
  const bool tree = batch.parents != nullptr;

  // (the swizzled tiles need 1024-byte alignment; there is no other shared memory)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sP = smem + C::NQ * C::QT_BYTES;   // ring of parts
  Shared& sh = *reinterpret_cast<Shared*>(sP + C::NP * PART);
  if ((smem_u32(smem) & 1023u) != 0) {        // (never, by the declaration above)
    pdl_enter();
    if (tid == 0) record_error(p.status, kDevErrTimeoutBase + kSiteQFull);
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < C::NP; ++s) {
      mbar_init(smem_u32(&sh.part_full[s]), 2);   // both copying warps
      mbar_init(smem_u32(&sh.part_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), 1);
      mbar_init(smem_u32(&sh.q_empty[s]), 1);
      mbar_init(smem_u32(&sh.stat_full[s]), 4);
      mbar_init(smem_u32(&sh.stat_empty[s]), 4);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.p_full[s]), 4);
      mbar_init(smem_u32(&sh.pv_done[s]), 1);
      mbar_init(smem_u32(&sh.o_final[s]), 1);
      mbar_init(smem_u32(&sh.o_free[s]), 4);
    }
    for (int s = 0; s < NPC; ++s) {
      mbar_init(smem_u32(&sh.piece_full[s]), 1);
      mbar_init(smem_u32(&sh.piece_empty[s]), 11);   // all warps but 2
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort_flag = 0;
    sh.first_used = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }

  // (nothing before this reads or writes global memory)
  pdl_enter();
  const bool lost = lost_work(p.status, kLostWait);

  // ---------------- this CTA's share of all work
  // A unit costs kTileCost for each tile and kUnitCost: what a piece costs
  // besides its tiles.  Tile t of a unit is in the share that holds the unit's
  // position kUnitCost + t kTileCost.
  constexpr int TC = kTileCost, UC = ONE ? C::UC1 : C::UCG;
  const int per = CLUSTER ? 0 : (batch.B + C::THREADS - 1) / C::THREADS;   // sequences per thread
  PagedWhole share_of_all = {0, false};   // (ONE: there are no whole shares)
  const int& S = share_of_all.tiles;
  const bool& uncut = share_of_all.uncut;
  // whole shares of every unit of a sequence
  auto shares_of = [&](const PagedSeq& s) -> int {
    return ONE ? 0 : paged_whole_shares(share_of_all, s.len, s.n, p.window, tree, p.ts);
  };
  // cost of what is left of a kv head's first q units
  auto cost_of = [&](const PagedSeq& s, int whole, int q) -> long long {
    return TC * (paged_prefix(s.len, s.n, p.window, tree, p.ts, q) - static_cast<long long>(whole) * S * q) +
           static_cast<long long>(UC) * q;
  };
  auto head_cost = [&](const PagedSeq& s) -> long long {     // of a kv head of a sequence
    if constexpr (ONE)
      return s.n > 0 ? TC * paged_unit(s.len, s.n, p.window, tree, p.ts, 0).tiles + UC : 0;
    else
      return cost_of(s, shares_of(s), paged_units(s.n, p.ts));
  };
  auto tile_at = [](int o) { return max(0, (o - UC + TC - 1) / TC); };   // first tile at or behind position o
  // Sum over the block's threads and, in upto, over those up to this one.
  auto scan = [&](long long v, long long& upto, bool out) -> long long {
    upto = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    if (__syncthreads_or(out)) return -1;
    long long total = 0;
#pragma unroll
    for (int w = 0; w < C::THREADS / 32; ++w) {
      if (w < warp) upto += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    return total;
  };
  long long mine = 0, upto = 0;
  PagedSeq seq = {0, 0, 0};   // the thread's last one
  int units = 0, longest = 0; // (!ONE: units, and the longest one's tiles)
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b >= batch.B) break;
    seq = paged_seq(batch, b, p.status);
    mine += p.H_kv * head_cost(seq);
    if constexpr (!ONE) {
      if (seq.n == 0) continue;
      units += paged_count_units(seq.n, p.ts, p.H_kv);
      longest = max(longest, paged_most_tiles(seq.len, seq.n, p.window, tree, p.ts));
    }
  }
  long long total = 0;
  if constexpr (CLUSTER) {
    __syncthreads();
  } else if constexpr (ONE) {
    total = scan(mine, upto, lost);
  } else {
    // sums alone: what each CTA gets is settled below
    units = __reduce_add_sync(0xffffffffu, units);
    longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) {
      sh.warp_sum[warp] = mine;
      sh.warp_units[warp] = units;
      sh.warp_most[warp] = longest;
    }
    if (__syncthreads_or(lost)) {
      total = -1;
    } else {
      units = 0;
#pragma unroll
      for (int w = 0; w < C::THREADS / 32; ++w) {
        total += sh.warp_sum[w];
        units += sh.warp_units[w];
        longest = max(longest, sh.warp_most[w]);
      }
    }
  }
  tc_fence_after();
  const uint32_t tbase = sh.tmem;
  if (total < 0) {
    if (warp == 1) tmem_dealloc(tbase, 512);
    if (tid == 0) p.split[blockIdx.x].parts = 0;   // (the error may be cleared before the merge starts)
    return;
  }
  // Whole shares: CTAs 0 .. taken - 1.  What all shares and units cost leaves at
  // least one CTA over.
  int taken = 0, grid = gridDim.x, taken_mine = 0, taken_upto = 0;
  if constexpr (!ONE) {
    share_of_all = paged_whole(total, units, longest, grid, p.window);
    mine = 0;
    __syncthreads();
    for (int k = 0; k < per; ++k) {
      const int b = tid * per + k;
      if (b >= batch.B) break;
      if (per > 1) seq = paged_seq(batch, b, p.status);
      if (!uncut) mine += p.H_kv * head_cost(seq);
      taken_mine += p.H_kv * paged_units(seq.n, p.ts) * shares_of(seq);
    }
    // (at most kMaxCtas shares; costs below 2^48)
    total = scan(static_cast<long long>(taken_mine) << 48 | mine, upto, false);
    taken = static_cast<int>(total >> 48);
    taken_upto = static_cast<int>(upto >> 48);
    total &= (1LL << 48) - 1;
    upto &= (1LL << 48) - 1;
    grid -= taken;
  }
  const bool sharing = static_cast<int>(blockIdx.x) < taken;   // this CTA has a whole share
  const int me = blockIdx.x - taken;                           // its number among the others
  // (shares of a tile's cost or more: a unit's parts lie in consecutive CTAs)
  const bool small = total < 1 << 23;   // (64-bit divisions cost some 100 clocks each)
  const int ctas = static_cast<int>(min(static_cast<long long>(grid), total / TC));
  const bool idle = !sharing && me >= ctas;
  auto share = [&](int c) -> long long {   // first position of CTA c
    if (small) return static_cast<unsigned>(total) * static_cast<unsigned>(c) / static_cast<unsigned>(ctas);
    return total * c / ctas;
  };
  auto cta_of = [&](long long x) -> int {  // the CTA that holds position x
    if (small) return taken + (static_cast<unsigned>(x + 1) * static_cast<unsigned>(ctas) - 1) / static_cast<unsigned>(total);
    return taken + static_cast<int>(((x + 1) * ctas - 1) / total);
  };
  const long long from = idle || sharing ? 0 : share(me);
  const long long count = idle || sharing ? 0 : share(me + 1) - from;
  // The piece of a unit's tiles [t0, t0 + n); the part's slot is set by the caller.
  auto make_piece = [&](const PagedSeq& s, int b, int j, int q, const PagedUnit& u, int t0, int n) -> Piece {
    Piece pc;
    pc.b = b;
    pc.j = j;
    pc.i0 = q << p.ts;
    pc.row0 = s.row0 + pc.i0;
    pc.ntok = min(1 << p.ts, s.n - pc.i0);
    pc.n = s.n;
    pc.len = s.len;
    pc.lo = u.lo;
    pc.hi = u.hi;
    pc.tile0 = u.tile0 + t0;
    pc.tiles = n;
    const int c2 = 2 * static_cast<int>(blockIdx.x);
    pc.slot = t0 > 0 ? c2 : (n < u.tiles ? c2 + 1 : -1);
    return pc;
  };
  const bool finder = sharing ? static_cast<int>(blockIdx.x) < taken_upto &&
                                    static_cast<int>(blockIdx.x) >= taken_upto - taken_mine
                              : !idle && from < upto && from >= upto - mine;
  if (finder) {
    // the share's first sequence, and the position and share where that begins
    long long base = upto - mine;
    int b = tid * per, first = taken_upto - taken_mine;
    while (per > 1) {
      seq = paged_seq(batch, b, p.status);
      const long long n = uncut ? 0 : p.H_kv * head_cost(seq);
      const int t = ONE ? 0 : p.H_kv * paged_units(seq.n, p.ts) * shares_of(seq);
      if ((sharing ? static_cast<int>(blockIdx.x) < first + t : from < base + n) || b + 1 >= batch.B) break;
      base += n;
      first += t;
      ++b;
    }
    sh.start_b = b;
    sh.start_off = from - base;
    sh.start_base = base;
    sh.start_taken = first;
    sh.start_seq = seq;
    if constexpr (ONE) {   // the first piece at once: a step waits for it
      const long long off = from - base;
      const PagedUnit u = paged_unit(seq.len, seq.n, p.window, tree, p.ts, 0);
      const int cost = u.tiles * TC + UC;
      const int j = static_cast<int>(static_cast<unsigned>(off) / static_cast<unsigned>(cost));
      const int o = static_cast<int>(off) - j * cost;
      const int o1 = static_cast<int>(min(o + count, static_cast<long long>(cost)));
      const int t0 = tile_at(o), n = tile_at(o1) - t0;
      if (n > 0) {
        sh.piece[0] = make_piece(seq, b, j, 0, u, t0, n);
        sh.first_used = o1 - o;
        sh.first_j = j;
        mbar_arrive(smem_u32(&sh.piece_full[0]));
      }
    }
  }
  if constexpr (!CLUSTER) __syncthreads();

  int lost_site = 0;
  auto wait_warp = [&](uint64_t& bar, uint32_t parity, int site) -> bool {
    return __all_sync(0xffffffffu, wait_bar(smem_u32(&bar), parity, &sh.abort_flag, site, &lost_site));
  };
  // The next piece (whole warp); false at the end.  The release takes in every
  // word that was loaded (p.zero: 0, which the compiler does not know): it must
  // not overtake the loads.
  auto take = [&](int k, Piece& pc) -> bool {
    if (!wait_warp(sh.piece_full[k % NPC], (k / NPC) & 1, kSitePieceFull)) return false;
    pc = sh.piece[k % NPC];
    const int all = pc.b ^ pc.j ^ pc.row0 ^ pc.ntok ^ pc.i0 ^ pc.n ^ pc.len ^ pc.lo ^ pc.hi ^ pc.tile0 ^ pc.tiles ^ pc.slot;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh.piece_empty[k % NPC]) + (static_cast<uint32_t>(all) & p.zero));
    return pc.tiles > 0;
  };

  if (warp < 4) {
    regs_decrease<C::REGS_CTRL>();
    if (warp != 1 && warp != 2) {
      // ---------------- K and V: K of a tile, then V of the tile before; of
      // each part one half in each of two warps
      const int half = warp == 3 ? 1 : 0;
      const int ps = batch.page_shift, pool = batch.n_pages << ps, in_page = (1 << ps) - 1;
      Ring w;
      int issued = 0;
      // tile `tile` of a piece: lane k's `base` is the pool row of its page k
      auto load_part = [&](bool v, int part, int j, int tile, int base) -> bool {
        if (issued >= C::NP && !wait_warp(sh.part_empty[w.slot], w.phase ^ 1, kSitePartEmpty))
          return false;
        const uint32_t bar = smem_u32(&sh.part_full[w.slot]);
        if (lane == 0) mbar_arrive_expect_tx(bar, PART / 2);
        __syncwarp();
        // K: 64 of the part's channels of all slots; V: all channels of half
        // of its slots (d_h = 128 128, d_h = 256 64), a page's chunks together.
        // A lane per box: 100 clocks each, 400 in a loop of one lane's.
        constexpr int VS = 128 / C::PARTS / 2;
        const int shift = v ? p.vshift : min(ps, kTileShift), at = lane << shift;   // slots of a box
        const int so = v ? part * (2 * VS) + half * VS + at : at;
        const int row0 = __shfl_sync(0xffffffffu, base, ps < kTileShift ? so >> ps : 0);
        const int row = row0 < 0 ? pool : row0 + ((tile * BN + so) & in_page);
        const uint32_t dst = smem_u32(sP + w.slot * PART) + half * (PART / 2) + at * (v ? DH * 2 : 128);
        if (at < (v ? VS : BN)) {
          if (v) tma_load_4d(dst, &tmV, bar, 0, row, 0, j);
          else tma_load_3d(dst, &tmK, bar, (part * 2 + half) * 64, j, row);
        }
        w.next<C::NP>();
        ++issued;
        return true;
      };
      // A step: K of the next tile, then V of the one before (the first step
      // has no V, the last no K).
      bool ok = true;
      int pj = 0, ptile = -1, pbase = 0;   // the tile whose V is still to come
      Piece pc;
      pc.tiles = 0;
      int k = 0, i = 0, p_begin = 0, p_end = 0, first = 0, cur = 0, ahead = 0;
      const int32_t* table = nullptr;
      // page ids, 32 at a time: lane l holds entry first + l of the sequence
      auto in_table = [&](int at) { return at >= p_begin && at < p_end; };
      auto entry = [&](int at) { return in_table(at) ? __ldcg(table + at) : -1; };
      auto pool_row = [&](int at, int id) -> int {
        if (static_cast<unsigned>(id) < static_cast<unsigned>(batch.n_pages)) return id << ps;
        if (in_table(at)) record_error(p.status, kDevErrBadPaged);
        return -1;
      };
#pragma unroll 1
      while (ok) {
        bool more = true, fresh = false;
        if (i == pc.tiles) {
          more = take(k++, pc);
          i = 0;
          if (more) {
            table = batch.page_table + static_cast<size_t>(pc.b) * batch.max_pages;
            p_begin = pc.lo >> ps;                       // pages that hold visible slots
            p_end = ((pc.hi - 1) >> ps) + 1;
            first = ((pc.tile0 * BN) >> ps) - 32;
            fresh = true;
          }
        }
        const int tile = pc.tile0 + i, at = (tile * BN) >> ps;
        if (more && at >= first + 32) {
          first += 32;
          const int id0 = fresh ? entry(first + lane) : 0, id1 = entry(first + 32 + lane);
          cur = fresh ? pool_row(first + lane, id0) : ahead;
          ahead = pool_row(first + 32 + lane, id1);
        }
        const int base = __shfl_sync(0xffffffffu, cur, (at - first + (lane & 7)) & 31);
#pragma unroll 1
        for (int x = more ? 0 : C::PARTS; ok && x < (ptile >= 0 ? 2 * C::PARTS : C::PARTS); ++x) {
          const bool v = x >= C::PARTS;
          ok = load_part(v, v ? x - C::PARTS : x, v ? pj : pc.j, v ? ptile : tile, v ? pbase : base);
        }
        if (!more) break;
        pj = pc.j;
        ptile = tile;
        pbase = base;
        ++i;
      }
      // Every issued load lands before the CTA may exit.
      for (int n = max(0, issued - C::NP); n < issued; ++n)
        mbar_wait_drain(smem_u32(&sh.part_full[n % C::NP]), (n / C::NP) & 1);
    } else if (warp == 1) {
      // ---------------- MMA issue (whole warp, one elected lane)
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc_qk = idesc_f16(BM, BN, /*f16*/ 0, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f16(BM, DH, /*f16*/ 0, 0, /*B MN-major*/ 1);
      const uint32_t q_stride = p.qsmall ? QSMALL : CHUNK;
      Ring r;
      int g = 0;              // tiles whose S was issued
      int ge[2] = {0, 0};     // NQ = 2: the same of each query tile
      int pieces_e[2] = {0, 0};   // pieces whose first PV was issued
      // NQ = 1: S of a tile; for d_h = 256 its two parts are the channel halves.
      auto issue_s = [&](int g, uint32_t q_addr, uint64_t* q_done) -> bool {
#pragma unroll 1
        for (int part = 0; part < C::PARTS; ++part) {
          if (!wait_warp(sh.part_full[r.slot], r.phase, kSitePartFull)) return false;
          tc_fence_after();
          const uint64_t kd = sdesc_sw128(smem_u32(sP + r.slot * PART), 16, 1024);
          const uint64_t qd = sdesc_sw128(q_addr + part * 2 * q_stride, 16, 1024), qd1 = sdesc_plus(qd, q_stride);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss_lead(lead, tbase + (g & 1) * 128, sdesc_plus(k < 4 ? qd : qd1, (k & 3) * 32),
                        sdesc_plus(kd, (k >> 2) * CHUNK + (k & 3) * 32), idesc_qk, part > 0 || k > 0 ? 1u : 0u);
          mma_commit_lead(lead, smem_u32(&sh.part_empty[r.slot]));
          r.next<C::NP>();
        }
        mma_commit_lead(lead, smem_u32(&sh.s_full[g & 1]));
        if (q_done != nullptr) mma_commit_lead(lead, smem_u32(q_done));
        return true;
      };
      struct Pv {             // what the PV of a tile needs
        int tile, lo, hi, nq, first, last;
      };
      // O += P V of query tile e, from `part` of V at `vb`.
      // V lies in blocks of 2^vshift slots, a block's 64-channel chunks one
      // behind the other.
      const uint32_t v_chunk = 128u << p.vshift;
      constexpr int STEPS = 8 / C::PARTS;     // 16-slot steps of a part
      int from = 0, to = 0;                   // those of the part in hand that hold visible slots
      auto mma_pv = [&](int e, int buf, uint32_t vb, int part, bool first) {
        const uint64_t vd = sdesc_sw128(vb, v_chunk, 1024);
        auto step = [&](int k, bool sum) {
          const uint32_t rows = k * 2048, blocks = rows & ~(v_chunk - 1);   // (whole ones before it)
          mma_ts_lead(lead, tbase + O_COL + e * 128, tbase + buf * 128 + (part * STEPS + k) * 8,
                      sdesc_plus(vd, rows + blocks * (C::NCH - 1)), idesc_pv, sum ? 1u : 0u);
        };
        if (NQ == 2 || (from == 0 && to == STEPS)) {
#pragma unroll
          for (int k = 0; k < STEPS; ++k) step(k, !first || k > 0);
        } else {              // (a condition in each step instead: a tile 1.72 us, not 1.45)
#pragma unroll 1
          for (int k = from; k < to; ++k) step(k, !first || k > from);
        }
      };
      // V of the part in slot r.  NQ = 1: the steps without a visible slot are
      // left out, the slots outside [lo, hi) in the others zeroed; NQ = 2: all
      // of them zeroed (a second loop of steps costs chunks more than it saves).
      auto v_ready = [&](const Pv& t, int part, const Ring& r) -> bool {
        if (!wait_warp(sh.part_full[r.slot], r.phase, kSitePartFull)) return false;
        constexpr int ROWS = 128 / C::PARTS;
        const int s0 = t.tile * BN + part * ROWS;
        const int z = min(max(t.lo - s0, 0), ROWS), a = min(max(t.hi - s0, 0), ROWS);
        from = z >> 4;
        to = z < a ? (a + 15) >> 4 : 0;       // 0: none
        const int nz = NQ == 1 ? z & 15 : z, na = NQ == 1 ? -a & 15 : ROWS - a;
        if ((nz | na) != 0) {
          uint8_t* base = sP + r.slot * PART + (lane & 7) * 16;   // (8 lanes to a row's 128 bytes)
#pragma unroll 1
          for (int i = lane >> 3; i < nz + na; i += 4) {
            const int row = i < nz ? z - nz + i : a + i - nz;
            uint8_t* at = base + row * 128 + (row >> p.vshift) * (C::NCH - 1) * v_chunk;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c) *reinterpret_cast<uint4*>(at + c * v_chunk) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        return true;
      };
      // (before a piece's first PV: the piece before was read from O)
      auto pv_begin = [&](const Pv& t, int e) -> bool {
        if (!t.first) return true;
        const bool ok = pieces_e[e] == 0 || wait_warp(sh.o_free[e], (pieces_e[e] - 1) & 1, kSiteOFree);
        ++pieces_e[e];
        return ok;
      };
      // NQ = 1: the PV of tile number n.
      auto issue_pv1 = [&](const Pv& t, int n) -> bool {
        if (!pv_begin(t, 0) || !wait_warp(sh.p_full[n & 1], (n >> 1) & 1, kSitePFull)) return false;
        bool first = t.first;
#pragma unroll 1
        for (int part = 0; part < C::PARTS; ++part) {
          if (!v_ready(t, part, r)) return false;
          mma_pv(0, n & 1, smem_u32(sP + r.slot * PART), part, first);
          first = first && to == 0;
          mma_commit_lead(lead, smem_u32(&sh.part_empty[r.slot]));
          r.next<C::NP>();
        }
        mma_commit_lead(lead, smem_u32(&sh.pv_done[n & 1]));
        if (t.last) mma_commit_lead(lead, smem_u32(&sh.o_final[0]));
        return true;
      };
      // A step: S of the next tile, then PV of the one before (the first step
      // has no PV, the last no S).
      bool ok = true, pending = false;
      Pv prev = {};
      Piece pc;
      int k = 0, i = 0;       // pieces taken, tiles of the present one done
      int qbuf = 0;
      pc.tiles = 0;
#pragma unroll 1
      while (ok) {
        bool more = true;
        if (i == pc.tiles) {
          more = take(k, pc);
          if (more) {
            qbuf = p.qsmall ? k & 1 : 0;
            ok = wait_warp(sh.q_full[qbuf], (p.qsmall ? k >> 1 : k) & 1, kSiteQFull);
          }
          ++k;
          i = 0;
        }
        if (!ok || (!more && (!pending || sh.abort_flag))) break;
        const int nq = more ? (NQ == 2 && pc.ntok > (BM >> p.gshift) ? 2 : 1) : 0;
        const Pv cur = {pc.tile0 + i, pc.lo, pc.hi, nq, i == 0, i + 1 == pc.tiles};
        if constexpr (NQ == 1) {
          if (more) {
            ok = issue_s(g, smem_u32(sQ) + qbuf * (C::QT_BYTES / 2), cur.last ? &sh.q_empty[qbuf] : nullptr);
            if (!ok) break;
            ++g;
          }
          if (pending) ok = issue_pv1(prev, g - (more ? 2 : 1));
        } else {
          // S_e reuses the columns of P_e of the tile before, whose V comes
          // behind this tile's K in the ring.
          const Ring kr = r;
          if (more) r.next<C::NP>();
          if (pending) ok = v_ready(prev, 0, r);
          if (!ok) break;
          const uint32_t kb = smem_u32(sP + kr.slot * PART), vb = smem_u32(sP + r.slot * PART);
          const uint64_t kd = sdesc_sw128(kb, 16, 1024), qd = sdesc_sw128(smem_u32(sQ), 16, 1024);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (pending && e < prev.nq) {
              ok = pv_begin(prev, e) && wait_warp(sh.p_full[e], (ge[e] - 1) & 1, kSitePFull);
              if (!ok) break;
              tc_fence_after();
              mma_pv(e, e, vb, 0, prev.first);
              if (prev.last) mma_commit_lead(lead, smem_u32(&sh.o_final[e]));
              if (e + 1 == prev.nq) mma_commit_lead(lead, smem_u32(&sh.part_empty[r.slot]));
            }
            if (e == 0 && more) {
              ok = wait_warp(sh.part_full[kr.slot], kr.phase, kSitePartFull);
              if (!ok) break;
              tc_fence_after();
            }
            if (e < nq) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint32_t off = (c >> 2) * CHUNK + (c & 3) * 32;
                mma_ss_lead(lead, tbase + e * 128, sdesc_plus(qd, e * C::QT_BYTES + off), sdesc_plus(kd, off), idesc_qk,
                            c > 0 ? 1u : 0u);
              }
              mma_commit_lead(lead, smem_u32(&sh.s_full[e]));
              ++ge[e];
              if (e + 1 == nq) {
                mma_commit_lead(lead, smem_u32(&sh.part_empty[kr.slot]));
                if (cur.last) mma_commit_lead(lead, smem_u32(&sh.q_empty[0]));
              }
            }
          }
          if (pending) r.next<C::NP>();
        }
        if (!more) break;
        prev = cur;
        pending = true;
        ++i;
      }
      mma_commit_lead(lead, smem_u32(&sh.drain));
      mbar_wait_drain(smem_u32(&sh.drain), 0);
    } else {
      // ---------------- pieces
      Split split = {0, 0, 0, 0, 0, 0, 0, 0};
      long long left = count, pos = from, off = idle ? 0 : sh.start_off;
      int b = idle ? 0 : sh.start_b, k = 0, b0 = b + 1;
      PagedSeq win = {0, 0, 0};   // of sequence b0 + lane
      bool ok = true, first = true, have = false;
      // Q of piece k; few rows (qsmall) have two buffers.
      auto load_q = [&](const Piece& pc) {
        const int buf = p.qsmall ? k & 1 : 0, fill = p.qsmall ? k >> 1 : k;
        ok = fill == 0 || wait_warp(sh.q_empty[buf], (fill - 1) & 1, kSiteQEmpty);
        if (!ok) return;
        if (lane == 0) {
          const int tq1 = BM >> p.gshift, nt = NQ == 2 && pc.ntok > tq1 ? 2 : 1;
          const uint32_t bar = smem_u32(&sh.q_full[buf]), dst = smem_u32(sQ) + buf * (C::QT_BYTES / 2);
          // (a unit of few tokens does not read 128 rows)
          const bool few = (pc.ntok << p.gshift) <= 32;
          const int box = few ? min(p.tokbox << p.gshift, 32) : p.tokbox << p.gshift;   // rows
          mbar_arrive_expect_tx(bar, nt * C::NCH * box * 128);
#pragma unroll 1
          for (int x = 0; x < nt * C::NCH; ++x) {
            const int e = x / C::NCH, ch = x % C::NCH;
            tma_load_3d(dst + e * C::QT_BYTES + ch * (p.qsmall ? QSMALL : CHUNK), few ? &tmQ32 : &tmQ, bar, ch * 64,
                        pc.j << p.gshift, pc.row0 + e * tq1);
          }
        }
        ++k;
      };
      auto publish = [&](const Piece& pc) {
        ok = k < NPC || wait_warp(sh.piece_empty[k % NPC], ((k / NPC) & 1) ^ 1, kSitePieceEmpty);
        if (!ok) return;
        if (lane == 0) {
          sh.piece[k % NPC] = pc;
          mbar_arrive(smem_u32(&sh.piece_full[k % NPC]));
        }
        if (pc.tiles > 0) load_q(pc);
      };
      // A unit whose first piece is this CTA's, with others; what is left of it
      // behind `whole` shares, `rest` tiles, begins at position `start`.
      auto cut = [&](const Piece& pc, int whole, long long start, int rest) {
        split = {pc.row0, pc.ntok, pc.j, whole, static_cast<int>(blockIdx.x), whole, 0, 0};
        if (rest > 0) {
          split.rest = cta_of(start + UC);
          const int last = cta_of(start + UC + static_cast<long long>(rest - 1) * TC);
          split.inside = whole > 0 && last == split.rest;
          split.parts += last - split.rest + 1;
        }
      };
      if constexpr (CLUSTER) {
        // ---- this CTA's part of the cluster's unit
        const int cs = cluster_nctarank(), rank = cluster_ctarank(), unit = blockIdx.x / cs;
        const int head = unit / p.units, q = unit - head * p.units;
        const int seq_b = head / p.H_kv, j = head - seq_b * p.H_kv;
        const PagedSeq s = paged_seq(batch, seq_b, p.status);
        const PagedUnit u = paged_unit(s.len, s.n, p.window, tree, p.ts, q);
        const bool none = __any_sync(0xffffffffu, lost) || q << p.ts >= s.n;   // no such unit in the sequence
        const int tiles = none ? 0 : u.tiles, each = tiles / cs, more = tiles - each * cs;
        const int n = each + (rank < more ? 1 : 0);
        if (lane == 0) {
          sh.unit_rows = min(1 << p.ts, s.n - (q << p.ts)) << p.gshift;
          sh.unit_row0 = s.row0 + (q << p.ts);
          sh.unit_parts = min(tiles, cs);
        }
        if (n > 0) {
          Piece pc = make_piece(s, seq_b, j, q, u, rank * each + min(rank, more), n);
          pc.slot = cs > 1 ? 0 : -1;
          publish(pc);
        }
      }
      int passed = idle ? 0 : sh.start_taken;   // whole shares before the present sequence
      if (!ONE && sharing) {
        // ---- one whole share
        const PagedSeq s = sh.start_seq;
        const int whole = shares_of(s), nq = paged_units(s.n, p.ts), x = static_cast<int>(blockIdx.x) - passed;
        const int unit = x / max(whole, 1), at = x - unit * whole, j = unit / nq, q = unit - j * nq;
        const PagedUnit u = paged_unit(s.len, s.n, p.window, tree, p.ts, q);
        Piece pc = make_piece(s, b, j, q, u, uncut ? 0 : at * S, uncut ? u.tiles : S);
        if (pc.slot >= 0) pc.slot = 2 * blockIdx.x;
        publish(pc);
        if (at == 0 && pc.slot >= 0)
          cut(pc, whole, sh.start_base + j * cost_of(s, whole, nq) + cost_of(s, whole, q), u.tiles - whole * S);
      }
      while (ok && left > 0 && b < batch.B) {
        PagedSeq s = sh.start_seq;
        if (!first) {
          if (!have || b >= b0 + 32) {
            b0 = b;
            win = b0 + lane < batch.B ? paged_seq(batch, b0 + lane, p.status) : PagedSeq{0, 0, 0};
            have = true;
          }
          s.row0 = __shfl_sync(0xffffffffu, win.row0, b - b0);
          s.n = __shfl_sync(0xffffffffu, win.n, b - b0);
          s.len = __shfl_sync(0xffffffffu, win.len, b - b0);
        }
        const int whole = shares_of(s);
        int q = 0, j = 0, nq = 1, o = 0;   // unit and position in it
        if constexpr (ONE) {
          if (first && sh.first_used > 0) {
            // its first piece is there; it ends the unit or the CTA's share
            load_q(sh.piece[0]);
            const PagedUnit u = paged_unit(s.len, s.n, p.window, tree, p.ts, 0);
            if (sh.piece[0].slot == 2 * static_cast<int>(blockIdx.x) + 1)
              cut(sh.piece[0], 0, sh.start_base + static_cast<long long>(sh.first_j) * (u.tiles * TC + UC), u.tiles);
            left -= sh.first_used;
            pos += sh.first_used;
            j = sh.first_j + 1;
          } else {
            if (s.n == 0) {
              ++b;
              continue;
            }
            if (off > 0) {    // (inside the first sequence)
              const long long cost = head_cost(s);
              j = static_cast<int>(off / cost);
              o = static_cast<int>(off - j * cost);
            }
          }
        } else {
          // the unit of a head's position t: the last one that starts at or before it
          nq = paged_units(s.n, p.ts);
          int q1 = nq, at = nq;
          long long head = 0, start = 0, t = 0;
#pragma unroll 1
          while (true) {
            const long long to = cost_of(s, whole, at);
            if (head == 0) {
              if (to == 0) break;
              head = to;
              j = static_cast<int>(off / head);
              t = off - j * head;
            } else if (to <= t) {
              q = at;
              start = to;
            } else {
              q1 = at;
            }
            if (q1 - q <= 1) break;
            at = (q + q1) / 2;
          }
          if (head == 0) {
            ++b;
            continue;
          }
          o = static_cast<int>(t - start);
        }
        first = false;
        while (ok && left > 0 && j < p.H_kv) {
          const PagedUnit u = paged_unit(s.len, s.n, p.window, tree, p.ts, q);
          const int skip = whole * S, rest = u.tiles - skip;
          const int o1 = static_cast<int>(min(o + left, static_cast<long long>(rest) * TC + UC));
          const int t0 = tile_at(o), n = tile_at(o1) - t0;
          if (n > 0) {
            Piece pc = make_piece(s, b, j, q, u, skip + t0, n);
            const bool begun = t0 == 0 && n < rest;   // its first piece of several
            if (begun) pc.slot = 2 * blockIdx.x + 1;
            else if (t0 == 0 && whole > 0) pc.slot = kRest + passed + (j * nq + q) * whole;
            publish(pc);
            if (begun && whole == 0) cut(pc, 0, pos - o, rest);
          }
          left -= o1 - o;
          pos += o1 - o;
          o = 0;
          if (++q == nq) {
            q = 0;
            ++j;
          }
        }
        off = 0;
        ++b;
        passed += p.H_kv * nq * whole;
      }
      if (!CLUSTER && lane == 0) p.split[blockIdx.x] = split;   // (read by the merge)
      if (ok) publish(Piece{});
      // (every load that was issued lands before the CTA may exit)
      for (int i = max(0, k - (p.qsmall ? 2 : 1)); i < k; ++i)
        mbar_wait_drain(smem_u32(&sh.q_full[p.qsmall ? i & 1 : 0]), (p.qsmall ? i >> 1 : i) & 1);
    }
  } else {
    // ---------------- softmax of query tile e (thread r owns row r), epilogue
    const int e = NQ == 2 ? (warp - 4) >> 2 : 0;
    const int q = warp & 3;                // TMEM lane quarter
    const int r = q * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t o_base = tbase + lane_off + O_COL + e * 128;
    const int tq1 = BM >> p.gshift, tok = (e * BM + r) >> p.gshift;   // token of the unit
    // This row of a piece's O; np: the pieces before.
    auto epilogue = [&](const Piece& pc, float m_used, float l, int np) -> bool {
      if (!wait_warp(sh.o_final[e], np & 1, kSiteOFinal)) return false;
      const bool row_valid = tok < pc.ntok;
      const bool live = __any_sync(0xffffffffu, row_valid);
      if (live) {
        tc_fence_after();
        const bool whole = pc.slot < 0, have = row_valid && l != 0.f;
        const size_t orow = static_cast<size_t>(pc.row0 + tok) * p.H + (pc.j << p.gshift) +
                            (r & ((1 << p.gshift) - 1));
        const size_t slot = max(pc.slot, 0);
        // (a cluster's parts lie where the ring was: its last copies are read)
        float4* pdst = (CLUSTER ? reinterpret_cast<float4*>(sP) : p.part + slot * (DH / 4) * p.rows) + e * BM + r;
        float2* sdst = (CLUSTER ? reinterpret_cast<float2*>(sP + p.rows * DH * 4) : p.pstat + slot * p.rows) + e * BM + r;
        if (!whole && row_valid)
          *sdst = have ? make_float2(m_used, l) : make_float2(-INFINITY, 0.f);
        const float inv = have ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t ro[32];
          tmem_ld32(o_base + c * 32, ro);
          tmem_ld_wait(ro);
          if (row_valid && whole) {
            store_row32(static_cast<uint16_t*>(p.O) + orow * DH + c * 32, ro, inv, have, p.o_f16);
          } else if (row_valid) {
            // (rows next to each other: the lanes' stores are)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              pdst[static_cast<size_t>(c * 8 + x) * p.rows] =
                  make_float4(__uint_as_float(ro[4 * x]), __uint_as_float(ro[4 * x + 1]),
                              __uint_as_float(ro[4 * x + 2]), __uint_as_float(ro[4 * x + 3]));
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.o_free[e]));
      return true;
    };
    int g = 0, np = 0;                     // tiles and pieces of this query tile so far
    bool ok = true;
    Piece pc;
    if (NQ == 1 && warp >= 8) {
      regs_increase<C::REGS_OTHER>();
      for (; ok && take(np, pc); ++np) {
        ok = wait_warp(sh.stat_full[np & 1], (np >> 1) & 1, kSiteStatFull);
        if (!ok) break;
        const float2 st = sh.stat[np & 1][r];
        __syncwarp();
        if (lane == 0)   // (as in take)
          mbar_arrive(smem_u32(&sh.stat_empty[np & 1]) +
                      ((__float_as_uint(st.x) ^ __float_as_uint(st.y)) & p.zero));
        ok = epilogue(pc, st.x, st.y, np);
      }
    } else {
      regs_increase<C::REGS_SOFT>();
      for (int k = 0; ok && take(k, pc); ++k) {
        if (pc.ntok <= e * tq1) continue;    // no such query tile in the unit
        const bool row_valid = tok < pc.ntok;
        const bool live = __any_sync(0xffffffffu, row_valid);
        float m_used = -INFINITY, l = 0.f;
        const int i_tok = pc.i0 + tok;       // number among the sequence's new tokens
        // Visible slots of the row: [v_lo, v_hi], and with a tree the ones of
        // `family` from slot len on.
        int v_lo = 0, v_hi = pc.len + i_tok;
        uint64_t family = 0;
        if (live && tree) {
          const PagedSeq s = {pc.row0 - pc.i0, pc.n, pc.len};
          const Ancestors a = paged_ancestors(batch, s, lane, p.status);
          const int it = min(i_tok, kTreeMax - 1);
          family = a.of(it);
          const int at = pc.len + __popcll(family) - 1;            // position
          v_hi = pc.len - 1;
          if (p.window > 0) {
            v_lo = at - p.window + 1;
            if (p.window < kTreeMax) {       // ancestors fewer than `window` steps away
              family = 1ull << it;
              int up = a.parent_of(it);
              for (int d = 1; d < p.window; ++d) {
                if (up >= 0) family |= 1ull << up;
                const int next = a.parent_of(max(up, 0));
                up = up >= 0 ? next : -1;
              }
            }
          }
        } else if (p.window > 0) {
          v_lo = pc.len + i_tok - p.window + 1;
        }
        // tiles within [t_lo, t_hi] are seen whole by every row
        const int t_lo = __reduce_max_sync(0xffffffffu, row_valid ? v_lo : 0);
        const int t_hi = __reduce_min_sync(0xffffffffu, row_valid ? v_hi : 0x7fffffff);
        for (int i = 0; i < pc.tiles; ++i, ++g) {
          const int sb = NQ == 2 ? e : (g & 1);
          const uint32_t s_addr = tbase + lane_off + sb * 128;
          ok = wait_warp(sh.s_full[sb], NQ == 2 ? (g & 1) : ((g >> 1) & 1), kSiteSFull);
          if (!ok) break;
          if (live) {
            tc_fence_after();
            const int s_tile = (pc.tile0 + i) * BN;
            if (s_tile < t_lo || s_tile + BN - 1 > t_hi) {
              // hidden columns become -inf in place (rolled: a few tiles of a
              // unit run this, and the softmax's own code stays small)
#pragma unroll 1
              for (int c = 0; c < BN; c += 32) {
                uint32_t x[32];
                tmem_ld32(s_addr + c, x);
                uint32_t keep = bits_from_to(v_lo - s_tile - c, v_hi - s_tile - c);
                if (tree) keep |= bits_at(family, s_tile + c - pc.len);
                tmem_ld_wait(x);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (!((keep >> k) & 1u)) x[k] = 0xff800000u;
                tmem_st32(s_addr + c, x);
              }
              tmem_st_wait();
            }
            uint32_t ra[32], rb[32], rc[32], rd[32];
            float m0, m1, m2, m3;
            tmem_ld32_max(s_addr, ra, m0);
            tmem_ld32_max(s_addr + 32, rb, m1);
            tmem_ld32_max(s_addr + 64, rc, m2);
            tmem_ld32_max(s_addr + 96, rd, m3);
            tmem_ld_wait(ra);
            tmem_ld_wait(rb);
            tmem_ld_wait(rc);
            tmem_ld_wait(rd);
            tmem_ld_wait(m0);
            tmem_ld_wait(m1);
            tmem_ld_wait(m2);
            tmem_ld_wait(m3);
            const float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * LOG2E;
            const bool grow = mx > m_used + (RESCALE_THRESHOLD + P_SHIFT);
            if (__any_sync(0xffffffffu, grow)) {
              const float m_new = grow ? mx - P_SHIFT : m_used;
              const float factor = (m_new == m_used) ? 1.f : ex2(m_used - m_new);
              if (i > 0) {
                // O holds the PV of the tiles before: with two query tiles S_e
                // of this tile was issued after them, with one PV may still run.
                if constexpr (NQ == 1) {
                  ok = wait_warp(sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, kSitePvDone);
                  if (!ok) break;
                  tc_fence_after();
                }
#pragma unroll 1
                for (int c = 0; c < DH / 32; ++c) {
                  uint32_t ro[32];
                  tmem_ld32(o_base + c * 32, ro);
                  tmem_ld_wait(ro);
#pragma unroll
                  for (int x = 0; x < 32; ++x) ro[x] = __float_as_uint(__uint_as_float(ro[x]) * factor);
                  tmem_st32(o_base + c * 32, ro);
                }
                tmem_st_wait();
              }
              l *= factor;
              m_used = m_new;
            }
            const float mref = (m_used == -INFINITY) ? 0.f : m_used;
            const float2 l2e = make_float2(LOG2E, LOG2E), negm = make_float2(-mref, -mref);
            float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                             make_float2(0.f, 0.f)};
            {
              uint32_t pk[32];
              exp_pack(ra, pk, acc, l2e, negm);
              exp_pack(rb, pk + 16, acc, l2e, negm);
              tmem_st32(s_addr, pk);
            }
            {
              uint32_t pk[32];
              exp_pack(rc, pk, acc, l2e, negm);
              exp_pack(rd, pk + 16, acc, l2e, negm);
              tmem_st32(s_addr + 32, pk);
            }
            const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
            const float2 a = __fadd2_rn(a01, a23);
            l += a.x + a.y;
            tmem_st_wait();
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[sb]));
        }
        if (!ok) break;
        if constexpr (NQ == 1) {             // to the epilogue's warps
          ok = np < 2 || wait_warp(sh.stat_empty[np & 1], ((np >> 1) & 1) ^ 1, kSiteStatEmpty);
          if (!ok) break;
          sh.stat[np & 1][r] = make_float2(m_used, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.stat_full[np & 1]));
        } else {
          ok = epilogue(pc, m_used, l, np);
        }
        ++np;
      }
    }
  }
  if (lost_site != 0) record_error(p.status, kDevErrTimeoutBase + lost_site);
  if constexpr (CLUSTER) {
    // The cluster's parts: each CTA adds an equal share of the rows' 4-channel
    // vectors.
    const int cs = cluster_nctarank();
    __syncwarp();
    if (cs > 1) cluster_sync();
    if (warp >= 4 && cs > 1) {
      const int rank = cluster_ctarank(), head = static_cast<int>(blockIdx.x) / cs / p.units;
      const int j = head % p.H_kv, rows = sh.unit_rows, parts = sh.unit_parts;
      const uint32_t o_at = smem_u32(sP), st_at = o_at + p.rows * DH * 4;
      const int vecs = parts > 0 ? rows * (DH / 4) : 0;
      const int begin = vecs * rank / cs, all = vecs * (rank + 1) / cs;   // this CTA's
      // I vectors of a thread at once, A parts of each: the loads of a round trip
      // (clusters of two: 21.5 us for 12B-shaped local trees with one vector at a
      // time, 20.7 with four)
      auto add_up = [&](auto items, auto at_once) {
        constexpr int I = decltype(items)::value, A = decltype(at_once)::value;
        for (int i0 = begin + tid - 128; i0 < all; i0 += I * 256) {
          MergeAcc<1> acc[I];
          int c[I], r[I];
#pragma unroll
          for (int u = 0; u < I; ++u) {
            acc[u].o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int i = min(i0 + u * 256, all - 1);
            c[u] = i / rows;
            r[u] = i - c[u] * rows;
          }
          for (int x0 = 0; x0 < parts; x0 += A) {
            float2 st[I][A];
            float4 x[I][A][1];
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
              for (int k = 0; k < A; ++k)
                if (x0 + k < parts) {
                  st[u][k] = ld_cluster_f2(mapa_shared(st_at + r[u] * 8, x0 + k));
                  x[u][k][0] = ld_cluster_f4(mapa_shared(o_at + (c[u] * p.rows + r[u]) * 16, x0 + k));
                }
#pragma unroll
            for (int u = 0; u < I; ++u)
#pragma unroll
              for (int k = 0; k < A; ++k)
                if (x0 + k < parts) acc[u].add(st[u][k], x[u][k]);
          }
#pragma unroll
          for (int u = 0; u < I; ++u) {
            if (i0 + u * 256 >= all) break;
            const float inv = acc[u].l != 0.f ? 1.f / acc[u].l : 0.f;
            const size_t orow = static_cast<size_t>(sh.unit_row0 + (r[u] >> p.gshift)) * p.H + (j << p.gshift) +
                                (r[u] & ((1 << p.gshift) - 1));
            reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + orow * DH)[c[u]] = acc[u].packed(0, inv, p.o_f16);
          }
        }
      };
      using std::integral_constant;
      if (parts <= 2) add_up(integral_constant<int, 4>(), integral_constant<int, 2>());
      else add_up(integral_constant<int, 1>(), integral_constant<int, 4>());
    }
    __syncwarp();
    if (cs > 1) cluster_sync();   // no CTA leaves while another reads its shared memory
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Adds the parts of the units that several CTAs have worked on: the unit whose
// first part is attention CTA blockIdx.x's, by gridDim.y CTAs, which need not
// look at the other units (a list of all units' tasks, over CTAs of its own
// number, took 2 to 3 us more: 4B-shaped mixed batches 43.9 -> 40.7 us).  A task
// is up to 32 rows and some of their channels: lanes along the rows, which lie
// next to each other in a part, and where they are few along 4-channel vectors
// too, VV of them per lane.  A lane has its row's sums to itself, so a task is
// one warp's, or that of several where a unit has many parts.
constexpr int kMergeWarps = 8;

__device__ __forceinline__ Split load_split(const Split* from) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(from)), b = __ldcg(reinterpret_cast<const int4*>(from) + 1);
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Lanes along the rows of a unit of `all` rows: a power of two.
__host__ __device__ inline int merge_pad(int all) {
  int pad = 1;
  while (pad < all && pad < 32) pad *= 2;
  return pad;
}
__host__ __device__ inline int merge_warps(int parts) {   // of a task
  return parts >= 32 ? 8 : (parts >= 16 ? 4 : (parts >= 8 ? 2 : 1));
}

template <int DH, int VV>
__global__ void __launch_bounds__(32 * kMergeWarps, 3) paged_merge_kernel(const Params p) {
  pdl_enter();
  const bool lost = lost_work(p.status, kLostWait);   // parts may be missing
  __shared__ float2 sums[kMergeWarps][32];
  __shared__ float4 rows[kMergeWarps][VV][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Split u = load_split(p.split + blockIdx.x);
  if (__syncthreads_or(lost) || u.parts == 0) return;
  const int all = u.ntok << p.gshift;          // rows of the unit
  const int pad = merge_pad(all);
  const int vecs = 32 / pad * VV;              // vectors of a task
  const int chunks = (DH / 4 + vecs - 1) / vecs, total = (all + 31) / 32 * chunks;
  const int wp = merge_warps(u.parts);
  const int sub = warp & (wp - 1), per = kMergeWarps / wp;
  for (int t0 = blockIdx.y * per; t0 < total; t0 += gridDim.y * per) {
    const int task = t0 + warp / wp;
    const int r = task / chunks * 32 + (lane & (pad - 1)), v0 = task % chunks * vecs + lane / pad * VV;
    const bool mine = task < total && r < all && v0 < DH / 4;
    MergeAcc<VV> acc;
#pragma unroll
    for (int v = 0; v < VV; ++v) acc.o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) {
      // this warp's parts: sub, sub + wp, ...
      constexpr int AT_ONCE = 4;
      for (int i0 = sub; i0 < u.parts; i0 += AT_ONCE * wp) {
        float2 st[AT_ONCE];
        float4 x[AT_ONCE][VV];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
          const int i = i0 + k * wp;
          st[k] = make_float2(0.f, 0.f);
          if (i < u.parts) {
            const size_t slot = u.slot(i);
            st[k] = __ldcg(p.pstat + slot * p.rows + r);
#pragma unroll
            for (int v = 0; v < VV; ++v) x[k][v] = __ldcg(p.part + (slot * (DH / 4) + v0 + v) * p.rows + r);
          }
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
          if (i0 + k * wp < u.parts) acc.add(st[k], x[k]);
      }
    }
    if (wp > 1) {
      sums[warp][lane] = make_float2(acc.m, acc.l);
#pragma unroll
      for (int v = 0; v < VV; ++v) rows[warp][v][lane] = acc.o[v];
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < wp; ++k) {
          float4 x[VV];
#pragma unroll
          for (int v = 0; v < VV; ++v) x[v] = rows[warp + k][v][lane];
          acc.add(sums[warp + k][lane], x);
        }
      __syncthreads();
    }
    if (mine && sub == 0) {
      const float inv = acc.l != 0.f ? 1.f / acc.l : 0.f;
      const size_t orow = static_cast<size_t>(u.row0 + (r >> p.gshift)) * p.H + (u.j << p.gshift) + (r & ((1 << p.gshift) - 1));
      uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + orow * DH) + v0;
      uint2 w[VV];
#pragma unroll
      for (int v = 0; v < VV; ++v) w[v] = acc.packed(v, inv, p.o_f16);
      if constexpr (VV == 2) *reinterpret_cast<uint4*>(dst) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
      else dst[0] = w[0];
    }
  }
}

// Query tiles per unit: two where a unit of d_h = 128 can fill them.
int query_tiles(int T_max, int G, int d_h) { return d_h == 128 && static_cast<long long>(T_max) * G > BM ? 2 : 1; }

// Rows of a part in the workspace.
int part_rows(int T_max, int G, int d_h) {
  return static_cast<int>(std::min<long long>(static_cast<long long>(T_max) * G, query_tiles(T_max, G, d_h) * BM));
}

struct Layout {
  size_t stat, part, split, total;
};
Layout layout(int T_max, int H, int H_kv, int d_h) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = static_cast<size_t>(kSlots) * part_rows(T_max, H / H_kv, d_h);
  Layout l;
  l.stat = 0;
  l.part = up(rows * sizeof(float2));
  l.split = l.part + up(rows * d_h * 4);
  l.total = l.split + up(kMaxCtas * sizeof(Split));
  return l;
}

template <int DH, int NQ, int MODE>
cudaError_t prepare_cfg() {
  using C = Cfg<DH, NQ>;
  int regs = 0;
  const void* kern = reinterpret_cast<const void*>(paged_attn_kernel<DH, NQ, MODE>);
  if (cudaError_t e = prepare_kernel(kern, C::SMEM, &regs)) return e;
  // The warpgroups' register increase waits for the registers the control
  // warps give up: launch only when the split fits.
  return regs * C::THREADS < C::REGS_SPLIT ? cudaErrorInvalidConfiguration : cudaSuccess;
}

template <int DH, int NQ, int MODE>
cudaError_t launch_cfg(const CUtensorMap& tq, const CUtensorMap& tq32, const CUtensorMap& tk, const CUtensorMap& tv,
                       const Params& p, cudaStream_t stream) {
  using C = Cfg<DH, NQ>;
  if (cudaError_t e = prepare_cfg<DH, NQ, MODE>()) return e;
  const int ctas = std::min(num_sms(), kMaxCtas);
  if (cudaError_t e = launch_pdl(paged_attn_kernel<DH, NQ, MODE>, dim3(ctas), dim3(C::THREADS), C::SMEM, stream, tq,
                                 tq32, tk, tv, p))
    return e;
  // CTAs per unit: one round of its tasks, as far as the host can tell, where units
  // have many parts (a token over 130000 slots, one kv head of d_h = 256: 38 us with
  // four CTAs, 35 with eight; a tree of 7 over 60000 44 with eight, 34 with 32); at
  // most eight where there are many units.
  const long long units = static_cast<long long>(p.batch.B) * p.H_kv * paged_units(p.batch.T_max, p.ts);
  const int wp = merge_warps(static_cast<int>(4 * ctas / std::min<long long>(units, ctas)));   // (uneven units: of four times the mean)
  const int vecs = 32 / merge_pad(p.rows) * (p.rows <= 8 ? 1 : 2);   // of a task
  const int tasks = (p.rows + 31) / 32 * ((DH / 4 + vecs - 1) / vecs);
  const dim3 grid(ctas, std::min((tasks * wp + kMergeWarps - 1) / kMergeWarps, wp > 1 ? 32 : 8)), block(32 * kMergeWarps);
  return p.rows <= 8 ? launch_pdl(paged_merge_kernel<DH, 1>, grid, block, 0, stream, p)
                     : launch_pdl(paged_merge_kernel<DH, 2>, grid, block, 0, stream, p);
}

// Clusters of `size` CTAs that the device holds at once, asked once per device.
template <int DH>
int clusters_at_once(int size) {
  constexpr int kDevices = 64;
  static std::mutex mu;
  static int known[kDevices][kMaxCluster + 1];   // plus one; 0: not asked
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  int& k = known[dev][size];
  if (k == 0) {
    // (more than 8 CTAs: as large a cluster as the device allows)
    cudaFuncSetAttribute(paged_attn_kernel<DH, 1, kClusterUnit>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(Cfg<DH, 1>::THREADS);
    cfg.dynamicSmemBytes = Cfg<DH, 1>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, paged_attn_kernel<DH, 1, kClusterUnit>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    k = n + 1;
  }
  return k - 1;
}

// CTAs of a unit's cluster, or 0: equal shares.  What a unit's tiles can be at
// most is known here from the window and the page table's width; the equal
// shares take fewer tiles per CTA and a merge, which costs kMergeTiles of them (a
// tree of 7 over 16000 slots, one kv head of d_h = 256, 8 tiles per CTA: 20 us by
// clusters, 24 shared out).  A table wider than the slots are filled looks like
// longer units: a tree of 7 over 5003 slots takes 13 us by clusters while the table
// has up to 8192, and 21 to 22 us shared out from 16384 on.
template <int DH>
int cluster_size(const Params& p) {
  const PagedBatch& b = p.batch;
  const long long units = static_cast<long long>(b.B) * p.H_kv * p.units;
  long long most = (static_cast<long long>(b.max_pages) << b.page_shift) / BN + 1;
  if (p.window > 0) {
    const int reach = b.parents != nullptr ? b.T_max : std::min(b.T_max, 1 << p.ts);
    most = std::min(most, (static_cast<long long>(p.window) + reach) / BN + 2);
  }
  // What equal shares would take per CTA: of an uneven batch at most so many
  // units have tokens, and where only the table bounds the lengths of several
  // sequences, half of it is taken to be filled (8 steps over 100 to 6000 slots,
  // 12B-shaped: 44 us by clusters, 34 shared out; over 3000 each 35 and 40; trees of
  // 7 over 500, 2000, 7000 and 16000, 4B-shaped: 39 and 31).
  const long long filled = std::min(units, ((b.M >> p.ts) + static_cast<long long>(b.B)) * p.H_kv);
  const bool open = b.B > 1 && p.window == 0;
  const int sms = num_sms();
  if (units > sms || prepare_cfg<DH, 1, kClusterUnit>() != cudaSuccess) return 0;
  for (int size = static_cast<int>(std::min<long long>(kMaxCluster, std::min(most, sms / units))); size >= 1; --size) {
    if ((most + size - 1) / size > filled * most / (open ? 2 * sms : sms) + kMergeTiles) return 0;
    if (units <= clusters_at_once<DH>(size)) return size;
  }
  return 0;
}

// One query tile per unit: by clusters where that is faster; *done says so.
template <int DH>
cudaError_t launch_clusters(const CUtensorMap& tq, const CUtensorMap& tq32, const CUtensorMap& tk,
                            const CUtensorMap& tv, const Params& p, cudaStream_t stream, bool* done) {
  using C = Cfg<DH, 1>;
  const int size = cluster_size<DH>(p);
  *done = size > 0;
  if (size == 0) return cudaSuccess;
  return launch_pdl_cluster(paged_attn_kernel<DH, 1, kClusterUnit>, dim3(p.batch.B * p.H_kv * p.units * size),
                            dim3(C::THREADS), C::SMEM, size, stream, tq, tq32, tk, tv, p);
}

}  // namespace

size_t paged_attention_ws_bytes(int T_max, int H, int H_kv, int d_h) {
  return layout(T_max, H, H_kv, d_h).total;
}

cudaError_t launch_paged_attention(const PagedBatch& given, const void* Q, const void* K_pages,
                                   const void* V_pages, void* O, int o_dtype, int H, int H_kv,
                                   int d_h, int window, void* ws, cudaStream_t stream, int* status) {
  PagedBatch batch = given;
  batch.T_max = std::min(batch.T_max, batch.M);   // (no sequence has more; the workspace is enough for fewer)
  if (window > kMaxSlots) window = 0;             // (hides nothing; the masks' differences stay in 32 bits)
  const int G = H / H_kv, nq = query_tiles(batch.T_max, G, d_h);
  const Layout lay = layout(batch.T_max, H, H_kv, d_h);
  uint8_t* w = static_cast<uint8_t*>(ws);
  Params p;
  p.batch = batch;
  p.pstat = reinterpret_cast<float2*>(w + lay.stat);
  p.part = reinterpret_cast<float4*>(w + lay.part);
  p.split = reinterpret_cast<Split*>(w + lay.split);
  p.O = O;
  p.o_f16 = o_dtype == kF16 ? 1 : 0;
  p.H = H;
  p.H_kv = H_kv;
  p.gshift = G == 4 ? 2 : (G == 2 ? 1 : 0);
  p.window = window;
  p.ts = kTileShift + (nq - 1) - p.gshift;
  p.tokbox = std::min(BM / G, batch.T_max);
  p.rows = part_rows(batch.T_max, G, d_h);
  p.qsmall = nq == 1 && p.tokbox * G <= 32 ? 1 : 0;
  p.zero = 0;
  p.units = 1;
  p.status = status;
  // Q [M, H, d_h]: box {64 channels, G heads, tokens}; rows behind M read as zeros.
  CUtensorMap tq, tq32, tk, tv;   // tq32: units of few tokens, 32 rows at most
  const uint64_t row = static_cast<uint64_t>(d_h) * 2;
  const uint64_t qdims[3] = {static_cast<uint64_t>(d_h), static_cast<uint64_t>(H), static_cast<uint64_t>(batch.M)};
  const uint64_t qstr[2] = {row, static_cast<uint64_t>(H) * row};
  const uint32_t qbox[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(p.tokbox)};
  const uint32_t qbox32[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(std::min(p.tokbox, 32 / G))};
  // the pools as rows of slots: box {64 channels, 1 head, the slots of a page}
  const uint64_t kdims[3] = {static_cast<uint64_t>(d_h), static_cast<uint64_t>(H_kv),
                             static_cast<uint64_t>(batch.n_pages) << batch.page_shift};
  const uint64_t kstr[2] = {row, static_cast<uint64_t>(H_kv) * row};
  const uint32_t kbox[3] = {64, 1, static_cast<uint32_t>(std::min(1 << batch.page_shift, BN))};
  // V: box {64 channels, slots of a page, all 64-channel chunks, 1 head}
  p.vshift = std::min(batch.page_shift, d_h == 128 ? 6 : 5);
  const uint64_t vdims[4] = {64, kdims[2], static_cast<uint64_t>(d_h / 64), static_cast<uint64_t>(H_kv)};
  const uint64_t vstr[3] = {static_cast<uint64_t>(H_kv) * row, 128, row};
  const uint32_t vbox[4] = {64, 1u << p.vshift, static_cast<uint32_t>(d_h / 64), 1};
  if (!encode_tiled(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, Q, qdims, qstr, qbox) ||
      (qbox32[2] != qbox[2] && !encode_tiled(&tq32, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, Q, qdims, qstr, qbox32)) ||
      !encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, K_pages, kdims, kstr, kbox) ||
      !encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, V_pages, vdims, vstr, vbox))
    return cudaErrorInvalidValue;
  if (qbox32[2] == qbox[2]) tq32 = tq;
  // Clusters work on units of one query tile.
  Params one = p;
  one.ts = kTileShift - p.gshift;
  one.rows = static_cast<int>(std::min<long long>(static_cast<long long>(batch.T_max) * G, BM));
  one.units = paged_units(batch.T_max, one.ts);
  bool done = false;
  const cudaError_t e = d_h == 128 ? launch_clusters<128>(tq, tq32, tk, tv, one, stream, &done)
                                   : launch_clusters<256>(tq, tq32, tk, tv, one, stream, &done);
  if (e != cudaSuccess || done) return e;
  if (d_h == 128)
    return nq == 2 ? launch_cfg<128, 2, kAnyUnits>(tq, tq32, tk, tv, p, stream)
                   : launch_cfg<128, 1, kOneUnit>(tq, tq32, tk, tv, p, stream);
  return batch.T_max <= 1 << p.ts ? launch_cfg<256, 1, kOneUnit>(tq, tq32, tk, tv, p, stream)
                                  : launch_cfg<256, 1, kAnyUnits>(tq, tq32, tk, tv, p, stream);
}

}  // namespace g3
