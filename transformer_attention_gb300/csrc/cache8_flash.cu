// Attention of many new tokens (a prompt or a chunk of one) over the 8-bit KV
// cache, on the tcgen05 tensor cores; what cache8_attn.cu computes for few.
//
// A CTA holds 128-row query tiles (TQ = 128 / G tokens x the G heads of kv
// head j) and walks the visible slots in tiles of 128, with S = Q K^T and O +=
// P V in fp16 with fp32 accumulators in TMEM.  The cache's bytes become the
// swizzled fp16 tiles that the MMAs read in four to sixteen converter warps:
// number x scale is an exact fp16 value (cache8.cuh), so the conversion costs
// no precision, and kind::f8f6f4 would need Q and P in 8 bits.  Per 128-slot
// tile and 128 channels that is 16384 two-number conversions, 270 clocks at the
// 60 per clock and SM measured for cvt.f16x2.e4m3x2, against about 1100 clocks
// of MMA for each query tile: d_h = 128 shares a conversion among two query
// tiles.  What bounds it is shared memory: a tile of d_h = 256 takes 64 KB of
// bytes in and out again, 128 KB of fp16 written and 192 KB read by the MMAs,
// 3500 clocks at 128 bytes each against 2050 of MMA; two query tiles of d_h =
// 128 320 KB, 2500 against 2050.  (Without the conversion's arithmetic and
// stores a prompt of 16384 tokens, d_h = 256, takes 603 us instead of 818.)
// 1024 tokens over 32768 slots, 27B-shaped: 398 us, 1.36 PFLOP/s.
//
// Warps (d_h = 128, two query tiles e = 0, 1):
//   0      TMA of the Q tiles (and for d_h = 256 of V's bytes)
//   1      TMEM allocation and MMA issue
//   2      positions: per tile a bit for each slot that holds a token, the
//          range of the stored positions, and the tile's scales
//   3      TMA of the cache's bytes, 8 KB (64 slots x 128 channels) at a time
//   4-7    converters: K, then V of each tile
//   8-15   softmax of tile 0 and of tile 1, one thread per row
// One tile of d_h = 128: converters in 4-11, softmax in 12-15.
// d_h = 256 has one query tile, converters of its own for K (4-11) and V
// (12-19), softmax in 20-23.  Shared memory holds two 32 KB parts of K and two
// of V: whole tiles of 128 slots x 128 channels, or for d_h = 256 the two
// channel halves of one K tile and the two slot halves of one V tile.
// TMEM: S_0 0-127, S_1 128-255 (d_h = 256: S of even and odd tiles), O from
// 256; P (fp16 pairs) is written over the first 64 columns of its S.
//
// Slots hidden from the whole CTA become zeros in the conversion, so that
// what they hold (a NaN, say) cannot reach O through a zero probability.
// A unit is a query tile (pair) of one kv head and batch row.  Whole rounds of
// the SMs take a unit per CTA; the units left over, fewer than the SMs, are
// cut along their slots (plan8), into equal parts where several fit, else into
// a large part each and small ones that the remaining SMs take one after
// another; flash8_merge_kernel adds the parts.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <cstddef>

#include "attention_common.cuh"
#include "cache8.cuh"
#include "cache8_flash.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace g3 {

namespace {

using attn::ex2;

constexpr int BM = 128, BN = 128;
constexpr uint32_t CHUNK = 128 * 128;       // 128 rows x 64 channels (128 B), swizzled
constexpr uint32_t PART = 32768;
constexpr uint32_t O_COL = 256;
constexpr float LOG2E = 1.4426950408889634f;
// A row's reference stays P_SHIFT below a past maximum while the present one
// is less than RESCALE_THRESHOLD above that (log2 units): the probabilities
// that are rounded to fp16 reach 2^15, so that those below its normal range, off
// by 2^-25, are off by 2^-32 at most of the row's largest (a key far above
// thousands of others does not lose their sum).
constexpr float RESCALE_THRESHOLD = 8.0f, P_SHIFT = 7.0f;

enum : int {
  kSiteQ = 80, kSiteKFull, kSiteKEmpty, kSiteVFull, kSiteVEmpty, kSiteSFull, kSitePFull,
  kSitePvDone, kSiteMetaFull, kSiteMetaEmpty, kSiteOFinal, kSiteRawFull,
  kSiteRawEmpty
};

constexpr uint32_t RAW = 8192;              // bytes of a raw granule: 64 slots x 128 channels
constexpr int NMETA = 4;
constexpr int MAX_RAW = 8;

struct alignas(16) Meta {  // (use is read in pairs)
  uint32_t ok[4];          // slots of the tile that hold a token below the CTA's last slot
  uint32_t use[4];         // those of them in the windows' reach of some valid token
  __half2 ks[2], vs[2];    // scales of the two blocks in the tiles (tile_scale)
  int pmin, pmax;          // range of the positions of the ok slots
  uint32_t halves;         // blocks whose tiles hold halves: K's in bits 0 and 1, V's 2 and 3
  int seq, base;           // seq: each of them is at position base + its place in the tile
  int pos[BN];
};
static_assert(sizeof(Meta) % 16 == 0 && offsetof(Meta, use) % 8 == 0, "pairs of use");

struct Shared {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], pv_done[2],
      meta_full[NMETA], meta_empty[NMETA], raw_full[MAX_RAW], raw_empty[MAX_RAW], o_final[2], drain;
  Meta meta[NMETA];
  uint32_t tmem;
  int abort_flag;
};

// NQ_ query tiles per CTA: two for d_h = 128, which share the conversion of a
// tile's bytes, one where a call has no second: S is then double buffered, as
// with d_h = 256, and two warpgroups convert (32 query rows over 65536 slots
// of 8 kv heads 62 -> 58 us, 132 over 272 slots of 2 kv heads 19 -> 16 us).
template <int DH, int G, int NQ_>
struct Cfg {
  static constexpr int NQ = NQ_;
  static_assert(NQ == 1 || DH == 128, "TMEM columns");
  static constexpr int TQ = BM / G;                // tokens per query tile
  static constexpr int NCH = DH / 64;
  static constexpr int PARTS = DH / 128;           // parts of a K or V tile
  static constexpr uint32_t QT_BYTES = BM * DH * 2;
  // raw granules: d_h = 128 one ring for K and V in turn, d_h = 256 a ring for each
  static constexpr int RING = PARTS == 2 ? 2 : (NQ == 1 ? 8 : 4);
  static constexpr int N_RAW = PARTS * RING;
  static constexpr uint32_t SMEM = NQ * QT_BYTES + 4 * PART + N_RAW * RAW + sizeof(Shared);
  static_assert(SMEM <= 232448 && N_RAW <= MAX_RAW, "shared memory budget");
  // Converter warpgroups: one beside two of softmax, else two of K and (d_h =
  // 256) two of V, each for one granule of a part.  (d_h = 256 with one of
  // each: 0.9 us a part, which a prompt of 16384 tokens waited for: 937 us.)
  static constexpr int SPLIT = NQ == 2 ? 1 : 2;    // warpgroups of a part
  static constexpr int CONV = PARTS * SPLIT;
  static constexpr int THREADS = 128 * (1 + CONV + NQ);
  // Registers per thread: control and converter warpgroups give some of the
  // launch's to the softmax warpgroups.
  static constexpr int REGS_LAUNCH = PARTS == 1 ? 128 : 80;
  static constexpr int REGS_CTRL = PARTS == 1 ? 48 : 40, REGS_CONV = PARTS == 1 ? 80 : 56;
  static constexpr int REGS_SOFT = PARTS == 1 ? 192 : 216;
  static_assert(REGS_CTRL + CONV * REGS_CONV + NQ * REGS_SOFT <= (1 + CONV + NQ) * REGS_LAUNCH,
                "register split above the launch allocation");
};

struct Params {
  const uint8_t* K8;
  const uint8_t* V8;
  const float* K_scale;
  const float* V_scale;
  const int32_t* posc;
  const int32_t* qpos;
  const int32_t* pad_lens;
  const int32_t* first;       // [B, items] first visible slot of each item (local layers) or null
  float2* rowstat;            // [B, H_kv, T*G] (reference, 1 / sum) of every row, or null
  float2* pstat;              // [cut units, parts, NQ * 128] (reference, sum)
  float* part;                // [cut units, parts, NQ * 128, DH] unnormalised
  void* O;
  int o_f16, B, T, S, H, H_kv, nb, end, window, items;
  int whole, cut, parts;      // units in one piece, units cut, into how many parts
  float first_part;           // share of a cut unit's tiles in its first part
  uint32_t zero;              // 0, which the compiler does not know
  int* status;
};

__device__ __forceinline__ void prefetch_4d(const void* tmap, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

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

__device__ __forceinline__ float mask_max(uint32_t (&r)[32], uint32_t keep) {
  float a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    if (!((keep >> c) & 1u)) r[c] = 0xff800000u;
    if (!((keep >> (c + 1)) & 1u)) r[c + 1] = 0xff800000u;
    a = fmaxf(a, __uint_as_float(r[c]));
    b = fmaxf(b, __uint_as_float(r[c + 1]));
  }
  return fmaxf(a, b);
}

template <int DH, int G, int NQ>
__global__ void __launch_bounds__(Cfg<DH, G, NQ>::THREADS, 1)
    flash8_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Params p) {
  pdl_enter();
  using C = Cfg<DH, G, NQ>;
  const bool lost = lost_work(p.status, kLostWait);   // (under way until the first barrier)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // (the swizzled tiles need 1024-byte alignment; there is no other shared memory)
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::NQ * C::QT_BYTES;   // two parts
  uint8_t* sV = sK + 2 * PART;                // two parts
  uint8_t* sR = sV + 2 * PART;                // raw granules
  Shared& sh = *reinterpret_cast<Shared*>(sR + C::N_RAW * RAW);
  if ((smem_u32(smem) & 1023u) != 0) {        // (never, by the declaration above)
    if (tid == 0) record_error(p.status, kDevErrTimeoutBase + kSiteQ);
    return;
  }

  // CTAs: the whole units, the first parts of the cut ones, the other parts.
  // Units: the latest tokens of every batch row and kv head first, which have
  // the most slots on a causal prompt.  (A prompt of 4096 tokens, 27B-shaped, 119
  // us; 124 when this was chosen, against 150 with the items of a head next to
  // each other and the last ones cut.)
  const int head_units = p.whole + p.cut, rest = static_cast<int>(blockIdx.x) - head_units;
  const int unit = rest < 0 ? blockIdx.x : p.whole + rest % p.cut;
  const int pt = rest < 0 ? 0 : 1 + rest / p.cut;           // part
  const bool whole = unit < p.whole;
  const int bjs = p.B * p.H_kv, item = p.items - 1 - unit / bjs;
  const int bj = unit % bjs, j = bj % p.H_kv, b = bj / p.H_kv;
  const int t0 = item * C::NQ * C::TQ;
  const int valid = min(p.T, p.T - (p.pad_lens != nullptr ? __ldcg(p.pad_lens + b) : 0));
  const int t_end = min(t0 + C::NQ * C::TQ, valid);          // past the last valid token
  const int nq = C::NQ == 2 && t0 + C::TQ < p.T ? 2 : 1;     // query tiles with tokens
  const int hi = t_end > t0 ? p.end + t_end : 0;
  int lo = p.first != nullptr ? __ldcg(p.first + static_cast<size_t>(b) * p.items + item) : 0;
  lo = min(lo, hi) / kC8Block * kC8Block;
  int n_tiles = (hi - lo + BN - 1) / BN, first_tile = 0;
  if (!whole) {
    // part 0 has its share, the others the rest evenly
    const int n0 = min(n_tiles, static_cast<int>(ceilf(p.first_part * n_tiles)));
    const int left = n_tiles - n0, others = p.parts - 1;
    first_tile = pt == 0 ? 0 : n0 + left * (pt - 1) / others;
    n_tiles = pt == 0 ? n0 : left * pt / others - left * (pt - 1) / others;
  }
  const int s_base = lo + first_tile * BN;

  if (tid == 0) {
    mbar_init(smem_u32(&sh.q_full), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 4 * C::SPLIT);
      mbar_init(smem_u32(&sh.k_empty[s]), 1);
      mbar_init(smem_u32(&sh.v_full[s]), 4 * C::SPLIT);
      mbar_init(smem_u32(&sh.v_empty[s]), 1);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.p_full[s]), 4);
      mbar_init(smem_u32(&sh.pv_done[s]), 1);
      mbar_init(smem_u32(&sh.o_final[s]), 1);
    }
    for (int s = 0; s < C::N_RAW; ++s) {
      mbar_init(smem_u32(&sh.raw_full[s]), 1);
      mbar_init(smem_u32(&sh.raw_empty[s]), 4);
    }
    for (int s = 0; s < NMETA; ++s) {
      mbar_init(smem_u32(&sh.meta_full[s]), 1);
      mbar_init(smem_u32(&sh.meta_empty[s]), 4 * (nq + C::CONV));   // softmax and converter warps
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  const bool stop = __syncthreads_or(lost);
  tc_fence_after();
  const uint32_t tbase = sh.tmem;
  if (stop) {
    if (warp == 1) tmem_dealloc(tbase, 512);
    return;
  }
  auto wait_warp = [&](uint64_t& bar, int parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, &sh.abort_flag, p.status, site));
  };

  if (warp < 4) {
    regs_decrease<C::REGS_CTRL>();
    // Raw granule n of a stream (RING slots from slot r0 on): of K, granule
    // (channel half, slot half) of a tile, of V d_h = 256 (slot half, channel
    // half); d_h = 128 has K's and V's two slot halves in one stream.  For
    // d_h = 256, whose rings are shorter, granules are pulled into L2 AHEAD
    // turns before: its rings cover a copy from L2, not one from HBM.
    constexpr int AHEAD = C::PARTS == 1 ? 0 : 12;
    auto load_raw = [&](int r0, bool v, int n_granules) {
      auto coord = [&](int n, bool& vv, int& c, int& s) {
        const int hh = (n >> 1) & 1, gg = n & 1;   // part, granule of the part
        vv = C::PARTS == 1 ? hh : v;
        c = C::PARTS == 1 ? 0 : (v ? gg : hh) * 128;
        s = s_base + (n >> 2) * BN + (C::PARTS == 1 ? gg : (v ? hh : gg)) * 64;
      };
      bool vv;
      int c, s, n = 0;
      for (int k = 0; k < min(AHEAD, n_granules); ++k) {
        coord(k, vv, c, s);
        prefetch_4d(vv ? &tmV : &tmK, c, j, s, b);
      }
      for (; n < n_granules; ++n) {
        const int r = r0 + n % C::RING;
        if (!mbar_wait(smem_u32(&sh.raw_empty[r]), ((n / C::RING) & 1) ^ 1, &sh.abort_flag, p.status,
                       kSiteRawEmpty))
          break;
        coord(n, vv, c, s);
        const uint32_t bar = smem_u32(&sh.raw_full[r]);
        mbar_arrive_expect_tx(bar, RAW);
        tma_load_4d(smem_u32(sR + r * RAW), vv ? &tmV : &tmK, bar, c, j, s, b);
        if (AHEAD > 0 && n + AHEAD < n_granules) {
          coord(n + AHEAD, vv, c, s);
          prefetch_4d(vv ? &tmV : &tmK, c, j, s, b);
        }
      }
      for (int k = max(0, n - C::RING); k < n; ++k)
        mbar_wait_drain(smem_u32(&sh.raw_full[r0 + k % C::RING]), (k / C::RING) & 1);
    };
    if (warp == 0 && lane == 0 && n_tiles > 0) {
      // ---------------- Q
      const uint32_t qb = smem_u32(&sh.q_full);
      mbar_arrive_expect_tx(qb, nq * C::QT_BYTES);
      for (int e = 0; e < nq; ++e)
        for (int ch = 0; ch < C::NCH; ++ch)
          tma_load_4d(smem_u32(sQ + e * C::QT_BYTES + ch * CHUNK), &tmQ, qb, ch * 64, j * G,
                      t0 + e * C::TQ, b);
      if constexpr (C::PARTS == 2) load_raw(2, true, 4 * n_tiles);
      mbar_wait_drain(qb, 0);
    } else if (warp == 3 && lane == 0) {
      load_raw(0, false, 4 * n_tiles);
    } else if (warp == 1 && n_tiles > 0) {
      // ---------------- MMA issue (whole warp, one elected lane)
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc_qk = idesc_f16(BM, BN, /*f16*/ 0, 0, 0);
      constexpr uint32_t idesc_pv = idesc_f16(BM, DH, /*f16*/ 0, 0, /*B MN-major*/ 1);
      // Blocks whose tiles hold halves (tile_scale) are multiplied twice, the
      // second time onto the first: S of their 64 slots, their part of O.  (Here
      // rather than in the softmax, whose registers and instructions every tile
      // would pay for: 27B-shaped chunk 403 us, and 396 like this.)
      constexpr uint32_t idesc_qk1 = idesc_f16(BM, kC8Block, /*f16*/ 0, 0, 0);
      constexpr uint32_t KBLK = kC8Block * 128;               // a block's rows of a K chunk
      uint32_t halves = 0, halves_pv = 0;                     // of the tiles of S and of PV
      // S += Q K^T for channels [k0, k1) / 16 of the block's slots
      auto again_s = [&](uint32_t d, uint32_t qa, uint32_t ka, int k0, int k1) {
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
          if (!((halves >> blk) & 1u)) continue;
#pragma unroll 1
          for (int k = k0; k < k1; ++k) {
            const uint32_t off = (k >> 2) * CHUNK + (k & 3) * 32;
            mma_ss_lead(lead, d + blk * kC8Block, sdesc_sw128(qa + off, 16, 1024),
                        sdesc_sw128(ka + off + blk * KBLK, 16, 1024), idesc_qk1, 1u);
          }
        }
      };
      // O += P V for the block's slots, 16 at a time
      auto again_pv = [&](int blk, uint32_t d, uint32_t pa, uint32_t va, uint32_t lbo) {
        if (!((halves_pv >> (2 + blk)) & 1u)) return;
#pragma unroll 1
        for (int k = 0; k < 4; ++k)
          mma_ts_lead(lead, d, pa + (blk * 4 + k) * 8, sdesc_sw128(va + k * 2048, lbo, 1024), idesc_pv, 1u);
      };
      const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sK), v_addr = smem_u32(sV);
      bool ok = wait_warp(sh.q_full, 0, kSiteQ);
      if constexpr (C::NQ == 2) {
        auto issue_s = [&](int e, int i) {
          const uint32_t kb = k_addr + (i & 1) * PART;
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint32_t off = (k >> 2) * CHUNK + (k & 3) * 32;
            mma_ss_lead(lead, tbase + e * 128, sdesc_sw128(q_addr + e * C::QT_BYTES + off, 16, 1024),
                        sdesc_sw128(kb + off, 16, 1024), idesc_qk, k > 0 ? 1u : 0u);
          }
          if (halves & 3u) again_s(tbase + e * 128, q_addr + e * C::QT_BYTES, kb, 0, DH / 16);
          mma_commit_lead(lead, smem_u32(&sh.s_full[e]));
        };
        auto issue_pv = [&](int e, int i) -> bool {
          if (!wait_warp(sh.p_full[e], i & 1, kSitePFull)) return false;
          if (e == 0 && !wait_warp(sh.v_full[i & 1], (i >> 1) & 1, kSiteVFull)) return false;
          tc_fence_after();
          const uint32_t vb = v_addr + (i & 1) * PART;
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts_lead(lead, tbase + O_COL + e * 128, tbase + e * 128 + k * 8,
                        sdesc_sw128(vb + k * 2048, CHUNK, 1024), idesc_pv,
                        (i > 0 || k > 0) ? 1u : 0u);
          for (int blk = 0; halves_pv >= 4u && blk < 2; ++blk)
            again_pv(blk, tbase + O_COL + e * 128, tbase + e * 128, vb + blk * 4 * 2048, CHUNK);
          return true;
        };
        for (int i = 0; ok && i < n_tiles; ++i) {
          ok = wait_warp(sh.k_full[i & 1], (i >> 1) & 1, kSiteKFull);
          if (!ok) break;
          tc_fence_after();
          halves = sh.meta[i % NMETA].halves;   // (the converters have waited for it)
          for (int e = 0; ok && e < nq; ++e) {
            // S_e reuses the columns of P_e of the tile before: the tensor
            // pipe runs PV_e before it.
            if (i > 0) ok = issue_pv(e, i - 1);
            if (!ok) break;
            if (i > 0 && e == nq - 1) mma_commit_lead(lead, smem_u32(&sh.v_empty[(i - 1) & 1]));
            issue_s(e, i);
          }
          if (!ok) break;
          mma_commit_lead(lead, smem_u32(&sh.k_empty[i & 1]));
          halves_pv = halves;
        }
        for (int e = 0; ok && e < nq; ++e) {
          ok = issue_pv(e, n_tiles - 1);
          if (ok) mma_commit_lead(lead, smem_u32(&sh.o_final[e]));
        }
      } else if constexpr (C::PARTS == 1) {
        // one query tile: S of even and of odd tiles
        auto issue_pv = [&](int i) -> bool {
          if (!wait_warp(sh.p_full[i & 1], (i >> 1) & 1, kSitePFull)) return false;
          if (!wait_warp(sh.v_full[i & 1], (i >> 1) & 1, kSiteVFull)) return false;
          tc_fence_after();
          const uint32_t vb = v_addr + (i & 1) * PART;
#pragma unroll
          for (int k = 0; k < BN / 16; ++k)
            mma_ts_lead(lead, tbase + O_COL, tbase + (i & 1) * 128 + k * 8,
                        sdesc_sw128(vb + k * 2048, CHUNK, 1024), idesc_pv, (i > 0 || k > 0) ? 1u : 0u);
          for (int blk = 0; halves_pv >= 4u && blk < 2; ++blk)
            again_pv(blk, tbase + O_COL, tbase + (i & 1) * 128, vb + blk * 4 * 2048, CHUNK);
          mma_commit_lead(lead, smem_u32(&sh.v_empty[i & 1]));
          mma_commit_lead(lead, smem_u32(&sh.pv_done[i & 1]));
          return true;
        };
        for (int i = 0; ok && i < n_tiles; ++i) {
          ok = wait_warp(sh.k_full[i & 1], (i >> 1) & 1, kSiteKFull);
          if (!ok) break;
          tc_fence_after();
          halves = sh.meta[i % NMETA].halves;   // (the converters have waited for it)
          const uint32_t kb = k_addr + (i & 1) * PART;
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint32_t off = (k >> 2) * CHUNK + (k & 3) * 32;
            mma_ss_lead(lead, tbase + (i & 1) * 128, sdesc_sw128(q_addr + off, 16, 1024),
                        sdesc_sw128(kb + off, 16, 1024), idesc_qk, k > 0 ? 1u : 0u);
          }
          if (halves & 3u) again_s(tbase + (i & 1) * 128, q_addr, kb, 0, DH / 16);
          mma_commit_lead(lead, smem_u32(&sh.k_empty[i & 1]));
          mma_commit_lead(lead, smem_u32(&sh.s_full[i & 1]));
          if (i > 0) ok = issue_pv(i - 1);
          halves_pv = halves;
        }
        if (ok) ok = issue_pv(n_tiles - 1);
        if (ok) mma_commit_lead(lead, smem_u32(&sh.o_final[0]));
      } else {
        auto issue_pv = [&](int i) -> bool {
          if (!wait_warp(sh.p_full[i & 1], (i >> 1) & 1, kSitePFull)) return false;
          for (int h = 0; h < 2; ++h) {
            if (!wait_warp(sh.v_full[h], i & 1, kSiteVFull)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts_lead(lead, tbase + O_COL, tbase + (i & 1) * 128 + (h * 4 + k) * 8,
                          sdesc_sw128(v_addr + h * PART + k * 2048, CHUNK / 2, 1024), idesc_pv,
                          (i > 0 || h > 0 || k > 0) ? 1u : 0u);
            again_pv(h, tbase + O_COL, tbase + (i & 1) * 128, v_addr + h * PART, CHUNK / 2);
            mma_commit_lead(lead, smem_u32(&sh.v_empty[h]));
          }
          mma_commit_lead(lead, smem_u32(&sh.pv_done[i & 1]));
          return true;
        };
        for (int i = 0; ok && i < n_tiles; ++i) {
          // S of tile i is issued before PV of tile i - 1 and after PV of
          // tile i - 2, whose P its columns held.
          for (int h = 0; ok && h < 2; ++h) {
            ok = wait_warp(sh.k_full[h], i & 1, kSiteKFull);
            if (!ok) break;
            tc_fence_after();
            halves = sh.meta[i % NMETA].halves;   // (the converters have waited for it)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t off = (h * 2 + (k >> 2)) * CHUNK + (k & 3) * 32;
              mma_ss_lead(lead, tbase + (i & 1) * 128, sdesc_sw128(q_addr + off, 16, 1024),
                          sdesc_sw128(k_addr + off, 16, 1024), idesc_qk, (h > 0 || k > 0) ? 1u : 0u);
            }
            if (halves & 3u) again_s(tbase + (i & 1) * 128, q_addr, k_addr, h * 8, h * 8 + 8);
            mma_commit_lead(lead, smem_u32(&sh.k_empty[h]));
          }
          if (!ok) break;
          mma_commit_lead(lead, smem_u32(&sh.s_full[i & 1]));
          if (i > 0) ok = issue_pv(i - 1);
          halves_pv = halves;
        }
        if (ok) ok = issue_pv(n_tiles - 1);
        if (ok) mma_commit_lead(lead, smem_u32(&sh.o_final[0]));
      }
      mma_commit_lead(lead, smem_u32(&sh.drain));
      mbar_wait_drain(smem_u32(&sh.drain), 0);
    } else if (warp == 2) {
      // ---------------- positions and scales of each tile's slots
      // Which slots may count at all: in the windows' reach of any valid token.
      int plo = 0, phi = INT_MAX;
      if (p.window > 0) {
        int qn = INT_MAX, qx = INT_MIN;
        for (int t = t0 + lane; t < t_end; t += 32) {
          const int q = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t);
          qn = min(qn, q);
          qx = max(qx, q);
        }
        qn = __reduce_min_sync(0xffffffffu, qn);
        qx = __reduce_max_sync(0xffffffffu, qx);
        window_range(qn, qx, p.window, plo, phi);
      }
      const int32_t* posr = p.posc + static_cast<size_t>(b) * p.S;
      // lanes 0, 1: K's scales of the tile's blocks, 2, 3: V's
      const float* sc = (lane & 2 ? p.V_scale : p.K_scale) + static_cast<size_t>(b) * p.nb * p.H_kv + j;
      int nx[4];
      float ns = 0.f;
      auto fetch = [&](int i) {
        if (i >= n_tiles) return;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int s = s_base + i * BN + k * 32 + lane;
          nx[k] = s < hi ? __ldcg(posr + s) : -1;
        }
        if (lane < 4)
          ns = __ldcg(sc + static_cast<size_t>(min((s_base + i * BN) / kC8Block + (lane & 1), p.nb - 1)) *
                              p.H_kv);
      };
      fetch(0);
      for (int i = 0; i < n_tiles; ++i) {
        if (!wait_warp(sh.meta_empty[i % NMETA], ((i / NMETA) & 1) ^ 1, kSiteMetaEmpty)) break;
        Meta& m = sh.meta[i % NMETA];
        int mn = INT_MAX, mx = INT_MIN, bn = INT_MAX, bx = INT_MIN;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool okk = nx[k] >= 0;
          const uint32_t w = __ballot_sync(0xffffffffu, okk);
          const uint32_t u = __ballot_sync(0xffffffffu, nx[k] >= plo && nx[k] <= phi);
          if (lane == 0) {
            m.ok[k] = w;
            m.use[k] = u;
          }
          m.pos[k * 32 + lane] = nx[k];
          if (okk) {
            mn = min(mn, nx[k]);
            mx = max(mx, nx[k]);
            bn = min(bn, nx[k] - (k * 32 + lane));
            bx = max(bx, nx[k] - (k * 32 + lane));
          }
        }
        mn = __reduce_min_sync(0xffffffffu, mn);
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (p.window > 0) {
          bn = __reduce_min_sync(0xffffffffu, bn);
          bx = __reduce_max_sync(0xffffffffu, bx);
        }
        const uint32_t halves = __ballot_sync(0xffffffffu, lane < 4 && halved(ns));
        if (lane < 4) (lane & 2 ? m.vs : m.ks)[lane & 1] = tile_scale(ns);
        if (lane == 0) {
          m.halves = halves;
          m.pmin = mn;
          m.pmax = mx;
          m.seq = bn == bx;
          m.base = bn;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.meta_full[i % NMETA]));
        fetch(i + 1);
      }
    }
  } else if (warp < 4 + 4 * C::CONV) {
    // ---------------- converters
    regs_decrease<C::REGS_CONV>();
    const int ct = tid & 127;                  // thread of its warpgroup
    const int col = ct & 7, row0 = ct >> 3;    // 16-channel group, slots row0 + 16 k of a granule
    // Part q of the stream (d_h = 128: K, V of each tile in turn; d_h = 256:
    // warps 4-11 the channel halves of K, 12-19 the slot halves of V): two
    // granules to 32 KB of fp16, each warpgroup both or its own.  Wide parts
    // are 128 slots x 128 channels, half parts (V of d_h = 256) 64 slots x 256
    // channels.  All loads are in flight before the first conversion, and the
    // granules are free for the next copies by then.
    const bool v256 = C::PARTS == 2 && warp >= 12;
    const int r0 = v256 ? 2 : 0, g0 = C::SPLIT == 2 ? (warp >> 2 & 1) ^ 1 : 0;
    constexpr int NG = 2 / C::SPLIT;
    const int swap = swap8(col, row0) * 8;
#pragma unroll 1
    for (int q = 0; q < 2 * n_tiles; ++q) {
      const int i = q >> 1, hh = q & 1;
      const bool v = C::PARTS == 1 ? hh : v256;
      const int buf = C::PARTS == 1 ? (i & 1) : hh, use = C::PARTS == 1 ? (i >> 1) : i;
      if (hh == 0 && !wait_warp(sh.meta_full[i % NMETA], (i / NMETA) & 1, kSiteMetaFull)) break;
      const Meta& m = sh.meta[i % NMETA];
      // scales and counted slots of the granules' 64-slot blocks (a block
      // without any may have any scale)
      const __half2* msc = v ? m.vs : m.ks;
      __half2 sc[NG];
      uint2 u[NG];
      bool whole_block = true;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int blk = v256 ? hh : g0 + g;
        u[g] = *reinterpret_cast<const uint2*>(m.use + 2 * blk);
        sc[g] = (u[g].x | u[g].y) != 0 ? msc[blk] : __float2half2_rn(0.f);
        whole_block &= (u[g].x & u[g].y) == 0xffffffffu;
      }
      uint2 x[4 * NG][2];
      bool ok = true;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int n = 2 * q + g0 + g, r = r0 + n % C::RING;
        ok = ok && wait_warp(sh.raw_full[r], (n / C::RING) & 1, kSiteRawFull);
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = row0 + 16 * k;
          const uint8_t* src = sR + r * RAW + row * 128 + ((col ^ (row & 7)) << 4);
          x[4 * g + k][0] = *reinterpret_cast<const uint2*>(src + swap);
          x[4 * g + k][1] = *reinterpret_cast<const uint2*>(src + (swap ^ 8));
        }
      }
      if (!ok) break;
      // The copy that refills a granule may start once its barrier is arrived
      // on: the address takes every lane's loaded words in, so that the
      // arrival cannot overtake the loads (it did where nothing used them
      // before it: calls back to back gave wrong rows).
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t got = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          got |= (x[4 * g + k][0].x | x[4 * g + k][0].y) | (x[4 * g + k][1].x | x[4 * g + k][1].y);
        got = __reduce_or_sync(0xffffffffu, got) & p.zero;
        if (lane == 0)
          mbar_arrive(smem_u32(&sh.raw_empty[r0 + (2 * q + g0 + g) % C::RING]) + got);
      }
      ok = ok && wait_warp(v ? sh.v_empty[buf] : sh.k_empty[buf], (use & 1) ^ 1, kSiteKEmpty);
      if (!ok) break;
      if (!whole_block) {
#pragma unroll
        for (int k = 0; k < 4 * NG; ++k) {
          const uint32_t w = k & 2 ? u[k >> 2].y : u[k >> 2].x;
          if (!((w >> ((row0 + 16 * k) & 31)) & 1u)) x[k][0] = x[k][1] = make_uint2(0, 0);
        }
      }
      // a part's second granule: the other channel chunks of the same slots,
      // or the next 64 slots
      const uint32_t chunk = v256 ? CHUNK / 2 : CHUNK, g1 = v256 ? CHUNK : CHUNK / 2;
      uint8_t* base = (v ? sV : sK) + buf * PART + (col >> 2) * chunk + g0 * g1 + row0 * 128;
#pragma unroll
      for (int k = 0; k < 4 * NG; ++k)
        store16_values(x[k][0], x[k][1], sc[k >> 2], col, row0,
                       base + (k & 3) * 2048 + (k >> 2) * g1);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(v ? &sh.v_full[buf] : &sh.k_full[buf]));
        if (hh == 1) mbar_arrive(smem_u32(&sh.meta_empty[i % NMETA]));
      }
    }
  } else {
    // ---------------- softmax of query tile e, thread r owns row r
    regs_increase<C::REGS_SOFT>();
    const int e = C::NQ == 2 ? (warp - 4 - 4 * C::CONV) >> 2 : 0;
    if (e < nq) {
      const int q = warp & 3;                // TMEM lane quarter (= warp % 4)
      const int r = q * 32 + lane;
      const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
      const uint32_t o_base = tbase + lane_off + O_COL + e * 128;
      const int t = t0 + e * C::TQ + r / G, h = j * G + r % G;
      const bool row_valid = t < valid;
      const int lim = row_valid ? p.end + t : -1;            // last visible slot
      int plo = 0, phi = INT_MAX;
      if (p.window > 0 && row_valid) {
        const int qp = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t);
        window_range(qp, qp, p.window, plo, phi);
      }
      // over the warp's valid rows (the others are not stored)
      const int w_lim = __reduce_min_sync(0xffffffffu, row_valid ? lim : INT_MAX);
      const int w_plo = __reduce_max_sync(0xffffffffu, plo);
      const int w_phi = __reduce_min_sync(0xffffffffu, phi);
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      for (int i = 0; i < n_tiles; ++i) {
        const int sb = C::NQ == 2 ? e : (i & 1);
        const uint32_t s_addr = tbase + lane_off + sb * 128;
        ok = wait_warp(sh.meta_full[i % NMETA], (i / NMETA) & 1, kSiteMetaFull);
        if (!ok) break;
        const Meta& mt = sh.meta[i % NMETA];
        const int s_tile = s_base + i * BN;
        const int pmin = mt.pmin, pmax = mt.pmax;
        const bool win_ok = pmin >= w_plo && pmax <= w_phi;
        const bool whole = (mt.ok[0] & mt.ok[1] & mt.ok[2] & mt.ok[3]) == 0xffffffffu &&
                           s_tile + BN - 1 <= w_lim && win_ok;
        ok = wait_warp(sh.s_full[sb], C::NQ == 2 ? (i & 1) : ((i >> 1) & 1), kSiteSFull);
        if (!ok) break;
        tc_fence_after();
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
        if (!whole) {
          uint32_t keep[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = lim - (s_tile + 32 * k);       // last visible column of the 32
            keep[k] = mt.ok[k] & (c < 0 ? 0u : (c >= 31 ? 0xffffffffu : (2u << c) - 1u));
          }
          if (!win_ok && mt.seq) {
            const long long base = mt.base;
            const int c0 = static_cast<int>(min(max(plo - base, 0LL), 128LL));
            const int c1 = static_cast<int>(min(max(phi - base, -1LL), 127LL));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int a = c0 - 32 * k, z = c1 - 32 * k;   // columns [a, z] of the 32
              const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : 0xffffffffu << a);
              keep[k] &= from & (z < 0 ? 0u : (z >= 31 ? 0xffffffffu : (2u << z) - 1u));
            }
          } else if (!win_ok) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t w = 0;
#pragma unroll 8
              for (int c = 0; c < 32; ++c) {
                const int ps = mt.pos[k * 32 + c];
                w |= (ps >= plo && ps <= phi ? 1u : 0u) << c;
              }
              // (an index known at compile time keeps keep[] in registers)
              keep[0] &= k == 0 ? w : 0xffffffffu;
              keep[1] &= k == 1 ? w : 0xffffffffu;
              keep[2] &= k == 2 ? w : 0xffffffffu;
              keep[3] &= k == 3 ? w : 0xffffffffu;
            }
          }
          m0 = mask_max(ra, keep[0]);
          m1 = mask_max(rb, keep[1]);
          m2 = mask_max(rc, keep[2]);
          m3 = mask_max(rd, keep[3]);
        }
        const float mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * LOG2E;
        // (mx takes what was read of the tile's positions in, as above)
        __syncwarp();
        if (lane == 0)
          mbar_arrive(smem_u32(&sh.meta_empty[i % NMETA]) + (__float_as_uint(mx) & p.zero));
        const bool grow = mx > m_used + (RESCALE_THRESHOLD + P_SHIFT);
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? mx - P_SHIFT : m_used;
          const float factor = (m_new == m_used) ? 1.f : ex2(m_used - m_new);
          if (i > 0) {
            // O holds the PV of the tiles before: with two query tiles S_e of
            // this tile was issued after them, with one PV may still run.
            if constexpr (C::NQ == 1) {
              ok = wait_warp(sh.pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, kSitePvDone);
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
              uint32_t ro[32];
              tmem_ld32(o_base + c * 32, ro);
              tmem_ld_wait(ro);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                ro[k] = __float_as_uint(__uint_as_float(ro[k]) * factor);
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
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[C::NQ == 2 ? e : (i & 1)]));
      }
      // ---------------- epilogue: this row of O
      if (ok && n_tiles > 0) {
        ok = wait_warp(sh.o_final[e], 0, kSiteOFinal);
        tc_fence_after();
      }
      const size_t orow = (static_cast<size_t>(b) * p.T + t) * p.H + h;
      const size_t prow = (static_cast<size_t>(unit - p.whole) * p.parts + pt) * (C::NQ * BM) + e * BM + r;
      const bool have = row_valid && n_tiles > 0 && l != 0.f;
      if (ok && !whole)
        p.pstat[prow] = have ? make_float2(m_used, l) : make_float2(-INFINITY, 0.f);
      else if (ok && t < p.T && p.rowstat != nullptr)
        p.rowstat[((static_cast<size_t>(b) * p.H_kv + j) * p.T + t) * G + r % G] =
            row_stat(m_used, l, have);
      const float inv = have ? 1.f / l : 0.f;
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < DH / 32; ++c) {
          uint32_t ro[32];
          if (n_tiles > 0) {
            tmem_ld32(o_base + c * 32, ro);
            tmem_ld_wait(ro);
          }
          if (whole) {
            if (t < p.T)
              store_row32(static_cast<uint16_t*>(p.O) + orow * DH + c * 32, ro, inv, have, p.o_f16);
          } else {
            float4* d = reinterpret_cast<float4*>(p.part + prow * DH + c * 32);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              d[k] = have ? make_float4(__uint_as_float(ro[4 * k]), __uint_as_float(ro[4 * k + 1]),
                                        __uint_as_float(ro[4 * k + 2]),
                                        __uint_as_float(ro[4 * k + 3]))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        tc_fence_before();
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// The parts of the cut units: CTA (u, y) adds those of 8 rows of unit u, a
// warp each.
template <int DH, int G, int NQ>
__global__ void __launch_bounds__(256) flash8_merge_kernel(const Params p) {
  pdl_enter();
  using C = Cfg<DH, G, NQ>;
  const bool lost = lost_work(p.status, kLostWait);   // parts may be missing
  constexpr int ROWS = 8;
  const int unit = p.whole + blockIdx.x;
  const int bjs = p.B * p.H_kv, item = p.items - 1 - unit / bjs;
  const int bj = unit % bjs, j = bj % p.H_kv, b = bj / p.H_kv;
  for (int i = threadIdx.x / 32; i < ROWS; i += 8) {
    const int row = blockIdx.y * ROWS + i, lane = threadIdx.x & 31;   // of the query tiles
    const int e = row / BM, r = row % BM;
    const int t = item * C::NQ * C::TQ + e * C::TQ + r / G;
    if (t >= p.T) continue;
    auto at = [&](int c) -> size_t {
      return (static_cast<size_t>(blockIdx.x) * p.parts + c) * (C::NQ * BM) + row;
    };
    // (max, sum) of 32 parts at a time, one per lane, then their rows of O
    float M = -INFINITY, L = 0.f;
    float4 acc[DH / 128];
#pragma unroll
    for (int v = 0; v < DH / 128; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < p.parts; c0 += 32) {
      const int n = min(32, p.parts - c0);
      const float2 st = lane < n ? __ldcg(p.pstat + at(c0 + lane)) : make_float2(-INFINITY, 0.f);
      float m = st.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float mn = fmaxf(M, m), ref = mn == -INFINITY ? 0.f : mn;
      const float old = ex2(M - ref), f = ex2(st.x - ref);
      float l = f * st.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      L = fmaf(L, old, l);
      M = mn;
#pragma unroll
      for (int v = 0; v < DH / 128; ++v) {
        acc[v].x *= old;
        acc[v].y *= old;
        acc[v].z *= old;
        acc[v].w *= old;
      }
#pragma unroll 4
      for (int c = 0; c < n; ++c) {
        const float fc = __shfl_sync(0xffffffffu, f, c);
        const float4* src = reinterpret_cast<const float4*>(p.part + at(c0 + c) * DH);
#pragma unroll
        for (int v = 0; v < DH / 128; ++v) {
          const float4 o = __ldcg(src + v * 32 + lane);
          acc[v].x = fmaf(fc, o.x, acc[v].x);
          acc[v].y = fmaf(fc, o.y, acc[v].y);
          acc[v].z = fmaf(fc, o.z, acc[v].z);
          acc[v].w = fmaf(fc, o.w, acc[v].w);
        }
      }
    }
    if (lost) return;
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const size_t orow = (static_cast<size_t>(b) * p.T + t) * p.H + j * G + r % G;
#pragma unroll
    for (int v = 0; v < DH / 128; ++v) {
      const float x0 = acc[v].x * inv, x1 = acc[v].y * inv, x2 = acc[v].z * inv, x3 = acc[v].w * inv;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.O) + orow * DH + v * 128 + lane * 4) =
          p.o_f16 ? make_uint2(pack_half2(x0, x1), pack_half2(x2, x3))
                  : make_uint2(pack_bf162(x0, x1), pack_bf162(x2, x3));
    }
    if (lane == 0 && p.rowstat != nullptr)
      p.rowstat[((static_cast<size_t>(b) * p.H_kv + j) * p.T + t) * G + r % G] =
          row_stat(M, L, L != 0.f);
  }
}

// First slot of batch row b that a valid token of an item (span tokens from
// item * span) can see on a local layer, by its stored position; hi if none.
// Up to eight CTAs per item, a cluster, while they fit the SMs: CTA r looks
// through every C-th run of kFirstSlots slots (130000 slots: 20 us by one CTA
// for 8192 at a time, 7 by eight).
constexpr int kFirstSlots = 16384;

__global__ void __launch_bounds__(1024) first8_kernel(const int32_t* __restrict__ posc,
                                                      const int32_t* __restrict__ qpos,
                                                      const int32_t* __restrict__ pad_lens, int T,
                                                      int S, int end, int window, int span,
                                                      int items, int32_t* __restrict__ first) {
  pdl_enter();
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), C = cluster.num_blocks();
  __shared__ int found;
  const int item = blockIdx.x / C, b = blockIdx.y, tid = threadIdx.x;
  const int valid = min(T, T - (pad_lens != nullptr ? __ldcg(pad_lens + b) : 0));
  const int t0 = item * span, t_end = min(t0 + span, valid);
  const int hi = t_end > t0 ? end + t_end : 0;
  int qn = INT_MAX, qx = INT_MIN;
  for (int t = t0 + (tid & 31); t < t_end; t += 32) {
    const int q = __ldcg(qpos + static_cast<size_t>(b) * T + t);
    qn = min(qn, q);
    qx = max(qx, q);
  }
  qn = __reduce_min_sync(0xffffffffu, qn);
  qx = __reduce_max_sync(0xffffffffu, qx);
  int plo = 0, phi = INT_MAX;
  window_range(qn, qx, window, plo, phi);
  if (tid == 0) found = INT_MAX;
  __syncthreads();
  const int32_t* row = posc + static_cast<size_t>(b) * S;
  for (long long base = static_cast<long long>(rank) * kFirstSlots; base < hi;
       base += static_cast<long long>(C) * kFirstSlots) {
    int best = INT_MAX;
#pragma unroll
    for (int k = kFirstSlots / 1024 - 1; k >= 0; --k) {
      const int s = static_cast<int>(base) + k * 1024 + tid;
      const int ps = s < hi ? __ldcg(row + s) : -1;
      if (ps >= plo && ps <= phi) best = s;
    }
    best = __reduce_min_sync(0xffffffffu, best);
    if ((tid & 31) == 0 && best != INT_MAX) atomicMin(&found, best);
    __syncthreads();
    if (found != INT_MAX) break;
    __syncthreads();
  }
  if (C > 1) cluster.sync();
  if (rank == 0 && tid == 0) {
    int f = min(found, hi);
    for (int r = 1; r < C; ++r) f = min(f, *cluster.map_shared_rank(&found, r));
    first[static_cast<size_t>(b) * items + item] = f;
  }
  if (C > 1) cluster.sync();         // no CTA leaves before its minimum is read
}

template <int DH, int G, int NQ>
cudaError_t launch_cfg(const void* Q, const Params& p, cudaStream_t stream) {
  using C = Cfg<DH, G, NQ>;
  CUtensorMap tq, tk, tv;
  // Q' [B, T, H, d_h]: box {64 channels, the G heads of a kv head, TQ tokens, 1}
  const uint64_t dims[4] = {static_cast<uint64_t>(DH), static_cast<uint64_t>(p.H),
                            static_cast<uint64_t>(p.T), static_cast<uint64_t>(p.B)};
  const uint64_t str[3] = {static_cast<uint64_t>(DH) * 2, static_cast<uint64_t>(p.H) * DH * 2,
                           static_cast<uint64_t>(p.T) * p.H * DH * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(C::TQ), 1};
  if (!encode_tiled(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, Q, dims, str, box))
    return cudaErrorInvalidValue;
  // caches [B, S, H_kv, d_h] of bytes: box {128 channels, 1 head, 64 slots, 1 row}
  const uint64_t kdims[4] = {static_cast<uint64_t>(DH), static_cast<uint64_t>(p.H_kv),
                             static_cast<uint64_t>(p.S), static_cast<uint64_t>(p.B)};
  const uint64_t kstr[3] = {static_cast<uint64_t>(DH), static_cast<uint64_t>(p.H_kv) * DH,
                            static_cast<uint64_t>(p.S) * p.H_kv * DH};
  const uint32_t kbox[4] = {128, 1, 64, 1};
  if (!encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.K8, kdims, kstr, kbox) ||
      !encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.V8, kdims, kstr, kbox))
    return cudaErrorInvalidValue;
  auto kern = flash8_kernel<DH, G, NQ>;
  int regs = 0;
  if (cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM, &regs)) return e;
  // The softmax warpgroups' increases wait for what the others give up:
  // launch only when the split fits the CTA's allocation.
  if (regs < C::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  const long long ctas = p.whole + static_cast<long long>(p.cut) * p.parts;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  cudaError_t e =
      launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(C::THREADS), C::SMEM, stream, tq, tk, tv, p);
  if (e != cudaSuccess || p.cut == 0) return e;
  return launch_pdl(flash8_merge_kernel<DH, G, NQ>, dim3(p.cut, C::NQ * BM / 8), dim3(256), 0, stream, p);
}

// How many units stay whole, and the cut of the others (fewer than the SMs),
// where the parts' rounds end earliest: counted in KV tiles, with a start and
// an end of a CTA worth kStartTiles, the merge as much and a tile more for
// every kPartsPerTile parts, which pass through memory (256 units of 24 tiles:
// 103 us cut, 89 uncut; 128 of 256 tiles 404 and 429; 8 of 9 tiles 21 and 29).
// `least` is
// the tiles of the shortest unit: where several rounds of units are as uneven
// as on a causal prompt, the short last ones fill the gaps uncut.
constexpr int kStartTiles = 3, kPartsPerTile = 48;
constexpr int kMaxCutParts = 320;            // parts that the workspace has room for

struct Plan8 {
  int whole, cut, parts;
  float first_part;
};

Plan8 plan8(long long units, int tiles, int least, int sms) {
  const int rest = static_cast<int>(units % sms);
  Plan8 uncut = {static_cast<int>(units), 0, 1, 1.f};
  if (rest == 0 || (units > sms && least <= tiles / 2)) return uncut;
  const int one = tiles + kStartTiles;                      // a round of whole units
  int best = one, parts = 1;
  float first = 1.f;
  // equal parts, all in one round
  const int k = std::min(sms / rest, tiles);
  auto merge = [&](int n) { return kStartTiles + rest * n / kPartsPerTile; };
  const int even = (tiles + k - 1) / std::max(k, 1) + kStartTiles + merge(k);
  if (k >= 2 && even < best) {
    best = even;
    parts = k;
    first = 1.f / k;
  }
  // a large part each, the small ones in q rounds on the other SMs
  if (k < 2) {
    const int q = (rest + sms - rest - 1) / (sms - rest);
    const int small = std::max(1, (tiles - (q - 1) * kStartTiles) / (q + 1));
    const int end = std::max(tiles - small + kStartTiles, q * (small + kStartTiles)) + merge(2);
    if (small < tiles && end < best) {
      best = end;
      parts = 2;
      first = static_cast<float>(tiles - small) / static_cast<float>(tiles);
    }
  }
  if (parts == 1 || rest * parts > kMaxCutParts) return uncut;
  return {static_cast<int>(units - rest), rest, parts, first};
}

}  // namespace

int flash8_span(int d_h, int G) { return (d_h == 128 ? 2 : 1) * (BM / G); }

size_t flash8_part_rows(int B, int T, int S, int H, int H_kv, int d_h) {
  const int span = flash8_span(d_h, H / H_kv);
  const long long units = static_cast<long long>(B) * H_kv * ((T + span - 1) / span);
  const long long most = units * ((S + BN - 1) / BN);
  return static_cast<size_t>(std::min<long long>(kMaxCutParts, most)) * (d_h == 128 ? 2 : 1) * BM;
}

cudaError_t launch_flash8(const Flash8Args& a, cudaStream_t stream) {
  const int G = a.H / a.H_kv;
  const int span = flash8_span(a.d_h, G), items = (a.T + span - 1) / span;
  const int hi = a.end + a.T;
  if (a.window > 0) {
    int cl = 1;
    while (cl < 8 && static_cast<long long>(cl) * kFirstSlots < hi &&
           2LL * cl * items * a.B <= num_sms())
      cl *= 2;
    const dim3 grid(items * cl, a.B), block(1024);
    cudaError_t e =
        cl > 1 ? launch_pdl_cluster(first8_kernel, grid, block, 0, cl, stream, a.posc, a.qpos, a.pad_lens,
                                    a.T, a.S, a.end, a.window, span, items, a.first)
               : launch_pdl(first8_kernel, grid, block, 0, stream, a.posc, a.qpos, a.pad_lens, a.T, a.S,
                            a.end, a.window, span, items, a.first);
    if (e != cudaSuccess) return e;
  }
  const long long units = static_cast<long long>(a.B) * a.H_kv * items;
  if (units > (1 << 30)) return cudaErrorInvalidValue;
  // (a local item's slots: its window and its own tokens, from a block border)
  int tiles = (hi + BN - 1) / BN, least = (a.end + std::min(span, a.T) + BN - 1) / BN;
  if (a.window > 0) {
    tiles = static_cast<int>(std::min<long long>(
        tiles, (static_cast<long long>(a.window) + span + kC8Block + BN - 1) / BN));
    // (only the first tokens of a long local prompt see less)
    if (a.T > 4LL * a.window) least = tiles;
  }
  const Plan8 plan = plan8(units, tiles, least, num_sms());
  Params p;
  p.K8 = static_cast<const uint8_t*>(a.K8);
  p.V8 = static_cast<const uint8_t*>(a.V8);
  p.K_scale = a.K_scale;
  p.V_scale = a.V_scale;
  p.posc = a.posc;
  p.qpos = a.qpos;
  p.pad_lens = a.pad_lens;
  p.first = a.window > 0 ? a.first : nullptr;
  p.rowstat = a.rowstat;
  p.pstat = a.pstat;
  p.part = a.part;
  p.O = a.O;
  p.o_f16 = a.o_f16;
  p.B = a.B;
  p.T = a.T;
  p.S = a.S;
  p.H = a.H;
  p.H_kv = a.H_kv;
  p.nb = c8_blocks(a.S);
  p.end = a.end;
  p.window = a.window;
  p.items = items;
  p.whole = plan.whole;
  p.cut = plan.cut;
  p.parts = plan.parts;
  p.first_part = plan.first_part;
  p.zero = 0;
  p.status = a.status;
  // (a call with one query tile per kv head: its units stay one item each)
  const bool two = a.d_h == 128 && a.T > BM / G;
#define G3_FLASH8_CASE(DH_, G_, NQ_) \
  if (a.d_h == DH_ && G == G_ && two == (NQ_ == 2)) return launch_cfg<DH_, G_, NQ_>(a.Q, p, stream);
  G3_FLASH8_CASE(128, 1, 2)
  G3_FLASH8_CASE(128, 2, 2)
  G3_FLASH8_CASE(128, 4, 2)
  G3_FLASH8_CASE(128, 1, 1)
  G3_FLASH8_CASE(128, 2, 1)
  G3_FLASH8_CASE(128, 4, 1)
  G3_FLASH8_CASE(256, 1, 1)
  G3_FLASH8_CASE(256, 2, 1)
  G3_FLASH8_CASE(256, 4, 1)
#undef G3_FLASH8_CASE
  return cudaErrorInvalidValue;
}

}  // namespace g3
