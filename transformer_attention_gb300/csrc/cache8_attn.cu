// Attention of new tokens over the 8-bit KV cache (cache8.cuh), and the
// weight that each slot received.
//
//   O[t, h] = sum_s p_s v_s,  p = softmax over the visible slots of q . k_s
//   weight_sum[s] += sum over the row's valid tokens and heads of p_s
//
// Visible slots as in decode.cu: s <= end + t, a stored position >= 0 and, on
// a local layer, within the window of the query's position.
//
// decode8_kernel (few query rows: T * G <= 16 per kv head).  Every
// byte of the cache is read once and meets at most 16 query rows, so HBM
// bounds it: d_h = 128 needs 256 bytes per slot and kv head.  The two
// contractions run on mma.sync m16n8k16 with the slots (K) and the channels
// (V) on the 16-row side and the query rows on the 8-wide side.  One token over
// 131072 slots of 16 kv heads: 86 us, 6.3 TB/s; 9 to 16 rows double the
// fragments and reach about 3 TB/s (16 rows over 65536 slots, d_h = 128 and 8
// kv heads 44 us, d_h = 256 and 4 kv heads 46; 8 rows 35), bound by the latency
// of the ten warps that fit an SM.  At one byte per number the fp32 CUDA cores
// would need 4 FMAs per byte for 4 rows, about their whole rate at the HBM rate,
// while these MMAs take under a fifth of theirs (measured 1024 fp16 FMA per
// clock and SM).  A tcgen05 tile has 128
// rows for which there are no queries, and could take the e4m3 bytes as they
// are only if the probabilities were split into 8-bit parts; many rows go to
// the tcgen05 kernel (cache8_flash.cu).
//   - The bytes go from the swizzled TMA tile straight into MMA fragments:
//     the contraction over channels does not care for their order, so a
//     thread's 4 consecutive channels serve as its k columns {2c, 2c+1, 2c+8,
//     2c+9}, and Q's fragments are permuted alike.  V needs slots along k:
//     ldmatrix.trans on byte pairs and one byte permutation give the
//     fragments of 16 channels.
//   - e4m3 numbers are exact in fp16; scales multiply the logits (K) and the
//     fp32 accumulator (V) in fp32: the accumulator is kept in units of the
//     current block's V scale and changes unit in the multiplication that the
//     running maximum asks for anyway.
//   - For the V product the probabilities, at most 1 against the running
//     maximum, are rounded to fp16 times 2^15: off by 2^-11 relative each
//     (averaged over slots; below the fp16 or bf16 output's own rounding) down
//     to 2^-29, by 2^-40 absolute below that, so that a key far above
//     thousands of others does not lose their sum.  Sums and maxima are fp32.
// The slots of a (row, kv head) are split over CTAs: up to eight form a
// cluster that merges its parts through distributed shared memory, more leave
// them to a second launch (merge8_kernel).  For weight_sum a last launch
// (weigh8_kernel) adds up exp2(logit - max) / sum from the logits that the
// first one left in the workspace (4 bytes per query row and slot, against 2
// d_h for K' and V; reading K' again would cost d_h).  On a local layer the
// CTAs take the last window's worth of slots at once, and look through the
// positions of all earlier slots for ones that a query still sees (positions
// may have gaps) while the first copies are under way.
#include <algorithm>
#include <climits>

#include "cache8.cuh"
#include "cache8_flash.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace g3 {

namespace {

constexpr int kTile = kC8Block;      // slots per tile: one scale block
constexpr int kSWarps = 4;           // warps along a tile's slots, 16 each
constexpr int kMaxSplits = 256;
constexpr int kMaxCluster = 8;
constexpr int kFewRows = 16;         // query rows of a kv head that decode8_kernel takes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPUnit = 32768.f;    // what the fp16 probabilities are multiplied by

enum { kSiteFull = 70, kSiteEmpty = 71 };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void named_barrier(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT n-tiles of 8 query rows per warp, RG groups of warps along the rows.
// d_h = 256 with up to 16 rows takes two groups, whose V accumulators fit the
// registers (one group of two n-tiles spilled: 9 rows of 66000 slots, T = 4, G =
// 4, 132 us); each converts the cache's bytes for itself.
template <int DH, int NT, int RG>
struct Cfg {
  static constexpr int CWARPS = kSWarps * RG;           // consumer warps
  static constexpr int THREADS = (CWARPS + 1) * 32;
  static constexpr int NCH = DH / 128;                  // 128-byte column boxes of a row
  static constexpr int BOX = kTile * 128;
  static constexpr int TILE = 2 * NCH * BOX;            // K' and V of one tile
  // CTAs per SM, and ring stages: 64 KB of tiles per CTA for three, 96 for
  // two, 192 for one
  static constexpr int CTAS = RG == 2 ? 1 : (DH == 128 && NT == 1 ? 3 : 2);
  static constexpr int NST = DH == 256 ? 3 * RG : (CTAS == 3 ? 4 : 6);
  static constexpr int RING = NST * TILE;
  static constexpr int NC = DH / 16;                    // 16-channel chunks
  static constexpr int NN = NT * RG;                    // n-tiles of the CTA
  static constexpr int QF = NC * NN * 32 * 8;           // Q fragments
  static constexpr int ROWS = NN * 8;
  static constexpr int LDM = DH + 8;                    // merge record row, floats
  static constexpr int MERGE = kSWarps * ROWS * LDM * 4;
  static constexpr int SMEM = 1024 + RING + QF;
  static_assert(MERGE + ROWS * DH * 4 <= RING, "merge records must fit in the ring");
  static_assert((SMEM + 2048) * CTAS <= 228 * 1024, "CTAs per SM");
};

struct Params {
  const __half* Q;            // [B, T, H, DH], query scale applied
  const float* K_scale;       // [B, nb, H_kv]
  const float* V_scale;
  const int32_t* posc;        // [B, S]
  const int32_t* qpos;        // [B, T]
  const int32_t* pad_lens;    // [B] or null
  int2* swept;                // [B, nsplit] tiles of each CTA's early slots that were
                              // attended (local layers with weights), or null
  float2* stat;               // [B*T*H, parts] (max, sum); parts = nsplit, or 1 of a cluster
  float* part;                // [B*T*H, nsplit, DH] unnormalised, of parts > 1
  float* logits;              // [B, H_kv, T*G, S64] base-2 logits, or null
  void* O;
  int o_f16, B, T, S, H, H_kv, nb, end, window, nsplit, cluster, late;
  uint32_t zero;              // 0, which the compiler does not know
  int* status;
};

// Tiles [0, k0) of a batch row are its early ones, [k0, k1) the `late` last
// (all of them on a global layer); `per` of each for one of nsplit CTAs.
struct Tiles {
  int hi, k0, k1, per_early, per_late;
};
__device__ __forceinline__ Tiles tiles_of(int end, int T, int valid, int late, int nsplit) {
  Tiles t;
  t.hi = valid > 0 ? end + min(valid, T) : 0;
  t.k1 = (t.hi + kTile - 1) / kTile;
  t.k0 = max(0, t.k1 - late);
  t.per_early = (t.k0 + nsplit - 1) / nsplit;
  t.per_late = (t.k1 - t.k0 + nsplit - 1) / nsplit;
  return t;
}

__device__ __forceinline__ void store_o(void* O, int o_f16, size_t at, float v) {
  if (o_f16)
    static_cast<__half*>(O)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(O)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void store_o4(void* O, int o_f16, size_t at, const float4& v, float f) {
  const float x0 = v.x * f, x1 = v.y * f, x2 = v.z * f, x3 = v.w * f;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + at) =
      o_f16 ? make_uint2(pack_half2(x0, x1), pack_half2(x2, x3))
            : make_uint2(pack_bf162(x0, x1), pack_bf162(x2, x3));
}

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

template <int DH, int NT, int RG>
__global__ void __launch_bounds__(Cfg<DH, NT, RG>::THREADS, Cfg<DH, NT, RG>::CTAS)
    decode8_kernel(const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const Params p) {
  pdl_enter();
  using C = Cfg<DH, NT, RG>;
  constexpr int kConsumers = C::CWARPS * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint2* qf = reinterpret_cast<uint2*>(smem + C::RING);       // [NC][NT][32]
  __shared__ __align__(8) uint64_t full[C::NST], empty[C::NST];
  __shared__ int abort_flag;
  __shared__ int early[2];             // first and last early tile with a visible slot
  __shared__ float2 cstat[C::ROWS];    // this CTA's part, for its cluster
  __shared__ float2 mstat[kSWarps][C::ROWS];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int G = p.H / p.H_kv;
  const int R = p.T * G;
  const int valid = p.T - (p.pad_lens != nullptr ? __ldcg(p.pad_lens + b) : 0);

  if (tid == 0) {
#pragma unroll
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), C::CWARPS);
    }
    abort_flag = 0;
    early[0] = INT_MAX;
    early[1] = -1;
    fence_barrier_init();
  }
  const Tiles tl = tiles_of(p.end, p.T, valid, p.late, p.nsplit);
  const int hi = tl.hi;
  const int late0 = min(tl.k1, tl.k0 + split * tl.per_late);
  const int n_late = min(tl.k1, late0 + tl.per_late) - late0;
  __syncthreads();
  // Tile i of this CTA: its late ones, then the early ones that it found.
  int early0 = 0, n_tiles = n_late;
  auto tile_at = [&](int i) { return i < n_late ? late0 + i : early0 + (i - n_late); };
  auto take_early = [&]() {
    if (early[1] >= 0) {
      early0 = early[0];
      n_tiles = n_late + early[1] - early0 + 1;
    }
  };

  if (warp == C::CWARPS) {
    // ---------------- producer: K'/V tiles of 64 slots into the ring
    int issued = 0;
    auto issue = [&](int upto) {
      for (; issued < upto; ++issued) {
        const int st = issued % C::NST;
        if (issued >= C::NST && !mbar_wait(smem_u32(&empty[st]), ((issued / C::NST) - 1) & 1,
                                           &abort_flag, p.status, kSiteEmpty))
          return;
        const uint32_t bar = smem_u32(&full[st]);
        mbar_arrive_expect_tx(bar, C::TILE);
        uint8_t* kd = ring + st * C::TILE;
        uint8_t* vd = kd + C::NCH * C::BOX;
        const int s0 = tile_at(issued) * kTile;
#pragma unroll
        for (int ch = 0; ch < C::NCH; ++ch) {
          tma_load_4d(smem_u32(kd + ch * C::BOX), &tmK, bar, ch * 128, j, s0, b);
          tma_load_4d(smem_u32(vd + ch * C::BOX), &tmV, bar, ch * 128, j, s0, b);
        }
      }
    };
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      issue(p.window > 0 ? min(n_late, C::NST) : n_late);
    }
    if (p.window > 0) {
      __syncwarp();
      named_barrier(2, C::THREADS);
      take_early();
      if (lane == 0) issue(n_tiles);
    }
    // Every issued load lands before the CTA may exit.
    if (lane == 0)
      for (int i = max(0, issued - C::NST); i < issued; ++i)
        mbar_wait_drain(smem_u32(&full[i % C::NST]), (i / C::NST) & 1);
    __syncwarp();
    if (p.cluster) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ---------------- consumers
  // Q fragments (while the first copies are under way): k columns {2c, 2c+1,
  // 2c+8, 2c+9} of a 16-channel chunk are the channels 4c .. 4c+3, row n = lane / 4.
#pragma unroll 4
  for (int i = tid; i < C::NC * C::NN * 32; i += kConsumers) {
    const int l = i & 31, nt = (i >> 5) % C::NN, ch = (i >> 5) / C::NN;
    const int r = nt * 8 + (l >> 2);
    uint2 q = make_uint2(0, 0);
    if (r < R) {
      const int t = r / G, h = j * G + r % G;
      q = __ldcg(reinterpret_cast<const uint2*>(
          p.Q + ((static_cast<size_t>(b) * p.T + t) * p.H + h) * DH + ch * 16 + (l & 3) * 4));
    }
    qf[i] = q;
  }
  named_barrier(1, kConsumers);
  const int sw = warp % kSWarps, n0 = warp / kSWarps * NT;   // slots, first n-tile
  // Warp sw takes slots 16sw .. 16sw + 15 of every tile
  // Rows of this thread: (n0 + nt) * 8 + 2c + e; slots g and g + 8 of the warp's 16.
  int lim[NT][2], plo[NT][2], phi[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = (n0 + nt) * 8 + 2 * c + e;
      lim[nt][e] = -1;
      plo[nt][e] = 0;
      phi[nt][e] = INT_MAX;
      if (r < R && r / G < valid) {
        const int t = r / G;
        lim[nt][e] = p.end + t;
        if (p.window > 0) {
          const int qp = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t);
          window_range(qp, qp, p.window, plo[nt][e], phi[nt][e]);
        }
      }
    }
  if (p.window > 0) {
    // early slots that some query of the row sees
    int qn = INT_MAX, qx = INT_MIN;
    for (int t = 0; t < min(valid, p.T); ++t) {
      const int q = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t);
      qn = min(qn, q);
      qx = max(qx, q);
    }
    int lo, up, first = INT_MAX, last = -1;
    window_range(qn, qx, p.window, lo, up);
    const int32_t* row = p.posc + static_cast<size_t>(b) * p.S;
    const int e0 = min(tl.k0, split * tl.per_early) * kTile;
    const int e1 = min(tl.k0, (split + 1) * tl.per_early) * kTile;
    for (int s = e0 + tid; s < e1; s += 8 * kConsumers) {
      int ps[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        ps[k] = s + k * kConsumers < e1 ? __ldcg(row + s + k * kConsumers) : -1;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (ps[k] >= lo && ps[k] <= up) {
          first = min(first, (s + k * kConsumers) / kTile);
          last = (s + k * kConsumers) / kTile;
        }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last >= 0) {
      atomicMin(&early[0], first);
      atomicMax(&early[1], last);
    }
    __threadfence_block();
    named_barrier(2, C::THREADS);
    take_early();
    if (p.swept != nullptr && j == 0 && tid == 0)
      p.swept[static_cast<size_t>(b) * p.nsplit + split] =
          make_int2(early0, early0 + n_tiles - n_late);
  }
  float m[NT][2], l[NT][2], o[C::NC][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int ch = 0; ch < C::NC; ++ch)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[ch][nt][e] = 0.f;
  }
  float unit = 1.f;                  // V scale that o is in units of
  const float* ksp = p.K_scale + (static_cast<size_t>(b) * p.nb) * p.H_kv + j;
  const float* vsp = p.V_scale + (static_cast<size_t>(b) * p.nb) * p.H_kv + j;
  const int32_t* posr = p.posc + static_cast<size_t>(b) * p.S;
  const int so = sw * 16 + g;      // this thread's first slot within a tile

  // ldmatrix row addresses within a box: matrices (slots 0-7 | 8-15) x (two
  // 16-byte chunks), chunk XORed with the slot's low bits by the TMA swizzle.
  const int mrow = sw * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
  const int mch = lane >> 4;
  const uint32_t roff = mrow * 128, rxor = mrow & 7;

  // the next tile's positions and scales are fetched a tile ahead
  int pos0 = -1, pos1 = -1;
  float ks = 0.f, vs = 0.f;
  auto fetch = [&](int i) {
    pos0 = pos1 = -1;
    if (i < n_tiles) {
      const int k = tile_at(i), s = k * kTile + so;
      if (s < hi) pos0 = __ldcg(posr + s);
      if (s + 8 < hi) pos1 = __ldcg(posr + s + 8);
      ks = __ldcg(ksp + static_cast<size_t>(k) * p.H_kv);
      vs = __ldcg(vsp + static_cast<size_t>(k) * p.H_kv);
    }
  };
  fetch(0);
  for (int i = 0; i < n_tiles; ++i) {
    const int st = i % C::NST;
    const int s = tile_at(i) * kTile + so;
    const int ps0 = pos0, ps1 = pos1;
    const float kl = ks * kLog2e, vsc = vs;
    fetch(i + 1);
    // visible (row, slot) pairs, and per slot whether any row sees it
    bool vis[NT][4];
    bool any0 = false, any1 = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        vis[nt][e] = ps0 >= plo[nt][e] && ps0 <= phi[nt][e] && s <= lim[nt][e];
        vis[nt][2 + e] = ps1 >= plo[nt][e] && ps1 <= phi[nt][e] && s + 8 <= lim[nt][e];
        any0 |= vis[nt][e];
        any1 |= vis[nt][2 + e];
      }
    const unsigned b0 = __ballot_sync(0xffffffffu, any0), b1 = __ballot_sync(0xffffffffu, any1);
    const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&full[st]), (i / C::NST) & 1,
                                                      &abort_flag, p.status, kSiteFull));
    if (!ok) break;
    float* lg = nullptr;
    if (p.logits != nullptr)
      lg = p.logits +
           (static_cast<size_t>(b) * p.H_kv + j) * R * (static_cast<size_t>(p.nb) * kTile) + s;
    uint32_t loaded = 0;             // words of the tile's last load
    if ((b0 | b1) != 0) {
      const uint32_t kt = smem_u32(ring + st * C::TILE);
      // S^T (16 slots x 8 rows): two accumulators shorten the chain
      float acc[2][NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][nt][e] = acc[1][nt][e] = 0.f;
#pragma unroll
      for (int cp = 0; cp < C::NC / 2; ++cp) {
        uint32_t r[4];
        const int ch = cp * 2 + mch;
        ldsm4(kt + (cp >> 2) * C::BOX + roff + (((ch & 7) ^ rxor) << 4), r);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a0 = c8_half2(r[2 * u]), a2 = c8_half2_hi(r[2 * u]);
          const uint32_t a1 = c8_half2(r[2 * u + 1]), a3 = c8_half2_hi(r[2 * u + 1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q = qf[((cp * 2 + u) * C::NN + n0 + nt) * 32 + lane];
            mma16816(acc[u][nt], a0, a1, a2, a3, q.x, q.y);
          }
        }
      }
      // online softmax in base 2; o changes its unit to this block's V scale
      uint32_t pb[NT][2];
      float f[NT][2];
      const float du = unit / vsc;
      bool same = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = vis[nt][e] ? (acc[0][nt][e] + acc[1][nt][e]) * kl : -INFINITY;
        if (lg != nullptr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = (n0 + nt) * 8 + 2 * c + (e & 1);
            if (row < R)
              lg[static_cast<size_t>(row) * (static_cast<size_t>(p.nb) * kTile) + (e >> 1) * 8] =
                  x[e];
          }
        }
        float pr[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[e], x[2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][e], mx);
          const float ref = mn == -INFINITY ? 0.f : mn;
          const float al = ex2(m[nt][e] - ref);     // 0 before the first visible slot
          m[nt][e] = mn;
          pr[e] = ex2(x[e] - ref);
          pr[2 + e] = ex2(x[2 + e] - ref);
          l[nt][e] = fmaf(l[nt][e], al, pr[e] + pr[2 + e]);
          f[nt][e] = al * du;
          same &= f[nt][e] == 1.f;
        }
        pb[nt][0] = transpose8x8(pack_half2(pr[0] * kPUnit, pr[1] * kPUnit));
        pb[nt][1] = transpose8x8(pack_half2(pr[2] * kPUnit, pr[3] * kPUnit));
      }
      unit = vsc;
      if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int ch = 0; ch < C::NC; ++ch)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[ch][nt][e] *= f[nt][e & 1];
      }
      // slots that no row sees count as zero whatever they hold (a NaN there
      // would survive its zero probability)
      uint32_t v0 = 0xffffffffu, v1 = 0xffffffffu;
      {
        unsigned n0 = b0 | (b0 >> 1), n1 = b1 | (b1 >> 1);
        n0 = (n0 | (n0 >> 2)) & 0x11111111u;
        n1 = (n1 | (n1 >> 2)) & 0x11111111u;
        if (n0 != 0x11111111u || n1 != 0x11111111u) {
          v0 = ((n0 >> (8 * c)) & 1u ? 0xFFFFu : 0u) | ((n0 >> (8 * c + 4)) & 1u ? 0xFFFF0000u : 0u);
          v1 = ((n1 >> (8 * c)) & 1u ? 0xFFFFu : 0u) | ((n1 >> (8 * c + 4)) & 1u ? 0xFFFF0000u : 0u);
        }
      }
      const uint32_t vt = kt + C::NCH * C::BOX;
#pragma unroll
      for (int cp = 0; cp < C::NC / 2; ++cp) {
        uint32_t r[4];
        const int ch = cp * 2 + mch;
        ldsm4_trans(vt + (cp >> 2) * C::BOX + roff + (((ch & 7) ^ rxor) << 4), r);
        if (cp == C::NC / 2 - 1) loaded = (r[0] | r[1]) | (r[2] | r[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // bytes (slot 2c: channels 2g, 2g+1; slot 2c+1: the same) to
          // (channel 2g: slots 2c, 2c+1; channel 2g+1: the same)
          const uint32_t w0 = __byte_perm(r[2 * u] & v0, 0, 0x3120);
          const uint32_t w1 = __byte_perm(r[2 * u + 1] & v1, 0, 0x3120);
          const uint32_t a0 = c8_half2(w0), a1 = c8_half2_hi(w0);
          const uint32_t a2 = c8_half2(w1), a3 = c8_half2_hi(w1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(o[cp * 2 + u][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
    } else if (lg != nullptr) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = (n0 + nt) * 8 + 2 * c + (e & 1);
          if (row < R)
            lg[static_cast<size_t>(row) * (static_cast<size_t>(p.nb) * kTile) + (e >> 1) * 8] =
                -INFINITY;
        }
    }
    // The next copy into the stage may start once this arrives: its address
    // takes the last load's words in, so that it cannot overtake the loads.
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty[st]) + (loaded & p.zero));
  }

  // ---------------- merge the warps along the slots (records in the ring, which no copy
  // writes any more once every warp is past its last tile)
  named_barrier(1, kConsumers);
  float* mg = reinterpret_cast<float*>(ring);
  float* cacc = reinterpret_cast<float*>(ring + C::MERGE);     // [ROWS][DH]
  unit *= 1.f / kPUnit;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[nt][e];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      const int row = (n0 + nt) * 8 + 2 * c + e;
      if (g == 0) mstat[sw][row] = make_float2(m[nt][e], s);
#pragma unroll
      for (int ch = 0; ch < C::NC; ++ch)
        *reinterpret_cast<float2*>(mg + (sw * C::ROWS + row) * C::LDM + ch * 16 + 2 * g) =
            make_float2(o[ch][nt][e] * unit, o[ch][nt][2 + e] * unit);
    }
  named_barrier(1, kConsumers);
  for (int idx = tid; idx < R * (DH / 4); idx += kConsumers) {
    const int r = idx / (DH / 4), ch = idx % (DH / 4) * 4;
    float2 ms[kSWarps];
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w) {
      ms[w] = mstat[w][r];
      M = fmaxf(M, ms[w].x);
    }
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < kSWarps; ++w) {
        const float fw = ex2(ms[w].x - M);
        L += fw * ms[w].y;
        // (a warp that saw nothing holds zeros)
        const float4 v = *reinterpret_cast<const float4*>(mg + (w * C::ROWS + r) * C::LDM + ch);
        acc.x += fw * v.x;
        acc.y += fw * v.y;
        acc.z += fw * v.z;
        acc.w += fw * v.w;
      }
    }
    const int t = r / G, h = j * G + r % G;
    const size_t orow = (static_cast<size_t>(b) * p.T + t) * p.H + h;
    if (p.cluster) {
      if (ch == 0) cstat[r] = make_float2(M, L);
      *reinterpret_cast<float4*>(cacc + r * DH + ch) = acc;
      continue;
    }
    if (ch == 0 && p.stat != nullptr) p.stat[orow * p.nsplit + split] = make_float2(M, L);
    if (p.nsplit == 1)
      store_o4(p.O, p.o_f16, orow * DH + ch, acc, L != 0.f ? 1.f / L : 0.f);
    else
      *reinterpret_cast<float4*>(p.part + (orow * p.nsplit + split) * DH + ch) = acc;
  }
  if (p.cluster) {
    // The cluster's parts, read through distributed shared memory; each CTA
    // writes its share of the rows' channels.
    __syncwarp();
    cluster_sync();
    const uint32_t st = smem_u32(cstat), ac = smem_u32(cacc);
    for (int idx = split * kConsumers + tid; idx < R * (DH / 4);
         idx += p.nsplit * kConsumers) {
      const int r = idx / (DH / 4), ch = idx % (DH / 4) * 4;
      float2 ms[8];
      float4 v[8];
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w)
        if (w < p.nsplit) {
          ms[w] = ld_cluster_f2(mapa_shared(st + r * 8, w));
          v[w] = ld_cluster_f4(mapa_shared(ac + (r * DH + ch) * 4, w));
          M = fmaxf(M, ms[w].x);
        }
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < 8; ++w)
          if (w < p.nsplit) {
            const float fw = ex2(ms[w].x - M);
            L += fw * ms[w].y;
            acc.x += fw * v[w].x;
            acc.y += fw * v[w].y;
            acc.z += fw * v[w].z;
            acc.w += fw * v[w].w;
          }
      }
      const size_t orow = (static_cast<size_t>(b) * p.T + r / G) * p.H + j * G + r % G;
      if (ch == 0 && p.stat != nullptr) p.stat[orow] = make_float2(M, L);
      store_o4(p.O, p.o_f16, orow * DH + ch, acc, L != 0.f ? 1.f / L : 0.f);
    }
    __syncwarp();
    cluster_sync();     // no CTA leaves while another reads its shared memory
  }
}

// ---------------------------------------------------------------- later launches
// Merge of the parts of one query row per CTA; its (max, sum) to fstat, if
// given.
struct MergeParams {
  const float2* stat;
  const float* part;
  float2* fstat;
  void* O;
  int o_f16, parts;
};

template <int DH>
__global__ void __launch_bounds__(DH) merge8_kernel(const MergeParams p) {
  pdl_enter();
  __shared__ float fw[kMaxSplits];
  __shared__ float red[2][DH / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t row = blockIdx.x;
  const float2* st = p.stat + row * p.parts;
  float2 mine[kMaxSplits / DH];
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / DH; ++i) {
    mine[i] = tid + i * DH < p.parts ? __ldcg(st + tid + i * DH) : make_float2(-INFINITY, 0.f);
    M = fmaxf(M, mine[i].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < DH / 32; ++i) M = fmaxf(M, red[0][i]);
#pragma unroll
  for (int i = 0; i < kMaxSplits / DH; ++i) {
    const float f = M == -INFINITY ? 0.f : ex2(mine[i].x - M);
    fw[tid + i * DH] = f;
    L = fmaf(f, mine[i].y, L);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[1][warp] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int i = 0; i < DH / 32; ++i) L += red[1][i];
  const float* base = p.part + row * p.parts * DH + tid;
  float acc = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.parts; ++i) acc = fmaf(fw[i], __ldcg(base + static_cast<size_t>(i) * DH), acc);
  store_o(p.O, p.o_f16, row * DH + tid, L != 0.f ? acc / L : 0.f);
  if (tid == 0 && p.fstat != nullptr) p.fstat[row] = make_float2(M, L);
}

// Weights of 512 / RW slots of one batch row per CTA, every query row's logits
// once, two slots per thread; RW groups of threads take every RW-th row (4
// where a call has more than 16, which would otherwise come one batch after
// another).
struct WeighParams {
  const float2* stat;         // [B*T*H] (max, sum)
  const float* logits;
  float* weight_sum;
  const int2* swept;          // as in Params
  const int32_t* pad_lens;
  int T, S, H, H_kv, nb, end, nsplit, late, wchunks;
  const int* status;
  int lost;
};

template <int RW>
__global__ void __launch_bounds__(256) weigh8_kernel(const WeighParams p) {
  pdl_enter();
  constexpr int GT = 256 / RW, WROWS = 16 * RW;       // threads of a group, rows at a time
  __shared__ float2 rs[2][WROWS];
  __shared__ int last[2][WROWS];
  __shared__ float2 wacc[RW > 1 ? RW - 1 : 1][GT];
  const bool stop = lost_work(p.status, p.lost);      // logits may be missing
  const int tid = threadIdx.x, rg = tid / GT;
  const int b = blockIdx.x / p.wchunks, s = (blockIdx.x % p.wchunks) * (2 * GT) + 2 * (tid % GT);
  // Rows in the order of the logits: kv head, token, head of the group.
  const int rows = p.T * p.H, G = p.H / p.H_kv, R = p.T * G;
  const size_t S64 = static_cast<size_t>(p.nb) * kTile;
  const int valid = p.T - (p.pad_lens != nullptr ? __ldcg(p.pad_lens + b) : 0);
  // Did the first launch attend this slot's tile?
  const Tiles tl = tiles_of(p.end, p.T, valid, p.late, p.nsplit);
  const int k = s / kTile;
  bool seen = s < tl.hi;
  if (seen && k < tl.k0) {
    const int2 e = __ldcg(p.swept + static_cast<size_t>(b) * p.nsplit + k / tl.per_early);
    seen = k >= e.x && k < e.y;
  }
  const float* lg = p.logits + static_cast<size_t>(b) * rows * S64 + s;
  float* out = p.weight_sum + static_cast<size_t>(b) * p.S;
  float2 old = make_float2(0.f, 0.f), acc = make_float2(0.f, 0.f);
  if (seen && rg == 0) {
    old.x = __ldcg(out + s);
    if (s + 1 < p.S) old.y = __ldcg(out + s + 1);
  }
  for (int r0 = 0, par = 0; r0 < rows; r0 += WROWS, par ^= 1) {
    const int n = min(WROWS, rows - r0);
    // The rows' logits (of one tile; loaded without asking whether they
    // count) are under way while the rows' (max, 1 / sum) come, and the last
    // slot whose logit the first launch wrote (a valid token's own).
    float2 x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = seen && RW * i + rg < n
                 ? __ldcg(reinterpret_cast<const float2*>(lg + (r0 + RW * i + rg) * S64))
                 : make_float2(0.f, 0.f);
    if (tid < WROWS) {
      float2 st = make_float2(0.f, 0.f);
      int lim = -1;
      if (tid < n) {
        const int j = (r0 + tid) / R, e = (r0 + tid) % R, t = e / G;
        st = __ldcg(p.stat + (static_cast<size_t>(b) * p.T + t) * p.H + j * G + e % G);
        lim = t < valid ? p.end + t : -1;
      }
      rs[par][tid] = make_float2(st.x == -INFINITY ? 0.f : st.x, st.y != 0.f ? 1.f / st.y : 0.f);
      last[par][tid] = lim;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 st = rs[par][RW * i + rg];
      const int lim = last[par][RW * i + rg];
      const float e0 = ex2(x[i].x - st.x), e1 = ex2(x[i].y - st.x);
      acc.x = fmaf(s <= lim ? e0 : 0.f, st.y, acc.x);
      acc.y = fmaf(s + 1 <= lim ? e1 : 0.f, st.y, acc.y);
    }
  }
  if constexpr (RW > 1) {
    if (rg > 0) wacc[rg - 1][tid % GT] = acc;
    __syncthreads();
    if (rg == 0) {
#pragma unroll
      for (int i = 0; i < RW - 1; ++i) {
        acc.x += wacc[i][tid].x;
        acc.y += wacc[i][tid].y;
      }
    }
  }
  if (seen && rg == 0 && !stop) {
    if (acc.x != 0.f) out[s] = old.x + acc.x;
    if (acc.y != 0.f) out[s + 1] = old.y + acc.y;
  }
}

// ---------------------------------------------------------------- planning
// Few rows (decode8_kernel), whose slots are split over a bounded number of
// CTAs, or many (launch_flash8).
bool few_rows(int T, int G) { return static_cast<long long>(T) * G <= kFewRows; }

int max_splits(int B, int S, int H_kv) {
  const long long units = static_cast<long long>(B) * H_kv;
  return static_cast<int>(std::min<long long>(
      {kMaxSplits, std::max<long long>(1, 1024 / units), c8_blocks(S)}));
}

// Splits of few rows, bound by HBM: counted in the time a tile takes at the
// full rate of HBM (2.6 ns for d_h = 128, 5.1 for 256), the tiles all
// together, or those of one CTA at the pace of one among `full` (the CTAs
// that saturate HBM), whichever is longer, about 2 us per round of CTAs, and
// for a merging launch 3.5 us and 50 ns per split, which up to eight CTAs of a
// cluster save.  12B-shaped batch of 16 over 7777 slots, d_h = 256: 896 CTAs
// in three rounds 88 us, 256 CTAs in one 82 us.
struct Split {
  int n;
  bool cluster;
};
Split splits_few(long long units, int most, int tiles, int d_h, int ctas_per_sm) {
  const int slots = ctas_per_sm * num_sms(), us = d_h == 256 ? 200 : 400;
  const int full = d_h == 256 && ctas_per_sm > 1 ? 224 : slots;
  Split best_of = {1, false};
  long long best = LLONG_MAX;
  for (int n = 1; n <= std::max(std::min(most, tiles), kMaxCluster); ++n) {
    const bool cluster = n == 2 || n == 4 || n == kMaxCluster;
    if (!cluster && n > std::min(most, tiles)) continue;
    const long long waves = (units * n + slots - 1) / slots, per = (tiles + n - 1) / n;
    const long long cost = std::max(units * tiles, waves * per * full) + waves * 2 * us +
                           (n > 1 && !cluster ? 7 * us / 2 + n * us / 20 : 0);
    if (cost < best) {
      best = cost;
      best_of = {n, cluster};
    }
  }
  return best_of;
}

struct Layout {
  int2* swept;          // few: [B, splits]
  int32_t* first;       // many: [B, items]
  float2* stat;         // few: [B*T*H, splits], many: parts of cut units
  float* part;
  float* logits;        // few rows with weights, and the merged (max, sum)
  float2* fstat;
  float2* rowstat;      // many rows with weights
  float* wpart;
  size_t bytes;
};

Layout layout(void* ws, int B, int T, int S, int H, int H_kv, int d_h, bool weights) {
  const bool few = few_rows(T, H / H_kv);
  uint8_t* w = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](bool wanted, size_t n) {
    uint8_t* q = w + at;
    at += wanted ? (n + 255) / 256 * 256 : 0;
    return q;
  };
  const size_t rows = static_cast<size_t>(B) * T * H;
  const int splits = max_splits(B, S, H_kv), span = flash8_span(d_h, H / H_kv);
  const size_t items = (static_cast<size_t>(T) + span - 1) / span;
  const size_t parts = few ? rows * splits : flash8_part_rows(B, T, S, H, H_kv, d_h);
  Layout L;
  L.swept = reinterpret_cast<int2*>(
      take(few && weights, static_cast<size_t>(B) * std::max(splits, kMaxCluster) * 8));
  L.first = reinterpret_cast<int32_t*>(take(!few, B * items * 4));
  L.stat = reinterpret_cast<float2*>(take(true, parts * 8));
  L.part = reinterpret_cast<float*>(take(!few || splits > 1, parts * d_h * 4));
  L.logits = reinterpret_cast<float*>(take(few && weights, rows * c8_blocks(S) * kTile * 4));
  L.fstat = reinterpret_cast<float2*>(take(few && weights, rows * 8));
  L.rowstat = reinterpret_cast<float2*>(take(!few && weights, rows * 8));
  L.wpart = reinterpret_cast<float*>(take(!few && weights, weights8_part_floats() * 4));
  L.bytes = at;
  return L;
}

// CTAs of decode8_kernel per SM for T * G = rows.
int few_ctas(int d_h, int rows) {
  if (d_h == 256) return rows <= 8 ? Cfg<256, 1, 1>::CTAS : Cfg<256, 1, 2>::CTAS;
  return rows <= 8 ? Cfg<128, 1, 1>::CTAS : Cfg<128, 2, 1>::CTAS;
}

template <int DH, int NT, int RG>
cudaError_t launch_cfg(const CUtensorMap& tk, const CUtensorMap& tv, const Params& p, dim3 grid,
                       cudaStream_t stream) {
  using C = Cfg<DH, NT, RG>;
  auto kern = decode8_kernel<DH, NT, RG>;
  if (cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM))
    return e;
  if (p.cluster)
    return launch_pdl_cluster(kern, grid, dim3(C::THREADS), C::SMEM, p.nsplit, stream, tk, tv,
                              p);
  return launch_pdl(kern, grid, dim3(C::THREADS), C::SMEM, stream, tk, tv, p);
}

}  // namespace

size_t cached8_attention_ws_bytes(int B, int T, int S, int H, int H_kv, int d_h, bool weights) {
  return layout(nullptr, B, T, S, H, H_kv, d_h, weights).bytes;
}

cudaError_t launch_cached8_attention(const void* Q, const void* K8, const void* V8,
                                     const float* K_scale, const float* V_scale,
                                     const int32_t* pos_cache, const int32_t* qpos,
                                     const int32_t* pad_lens, void* O, int o_dtype,
                                     float* weight_sum, int B, int T, int S, int end, int H,
                                     int H_kv, int d_h, int window, void* ws, cudaStream_t stream,
                                     int* status, int lost) {
  const Layout lay = layout(ws, B, T, S, H, H_kv, d_h, weight_sum != nullptr);
  const int hi = end + T, nb = c8_blocks(S), o_f16 = o_dtype == kF16 ? 1 : 0;
  cudaError_t e;

  if (!few_rows(T, H / H_kv)) {
    Flash8Args a;
    a.Q = Q;
    a.K8 = K8;
    a.V8 = V8;
    a.K_scale = K_scale;
    a.V_scale = V_scale;
    a.posc = pos_cache;
    a.qpos = qpos;
    a.pad_lens = pad_lens;
    a.first = lay.first;
    a.rowstat = weight_sum != nullptr ? lay.rowstat : nullptr;
    a.pstat = lay.stat;
    a.part = lay.part;
    a.O = O;
    a.o_f16 = o_f16;
    a.B = B;
    a.T = T;
    a.S = S;
    a.end = end;
    a.H = H;
    a.H_kv = H_kv;
    a.d_h = d_h;
    a.window = window;
    a.status = status;
    a.lost = lost;
    e = launch_flash8(a, stream);
    if (e != cudaSuccess || weight_sum == nullptr) return e;
    return launch_weights8(a, lay.wpart, weight_sum, stream);
  }

  const long long est = window > 0 ? std::min<long long>(hi, static_cast<long long>(window) + T)
                                   : static_cast<long long>(hi);
  const int tiles = static_cast<int>((est + kTile - 1) / kTile) + (window > 0 ? 1 : 0);
  const Split sp = splits_few(static_cast<long long>(B) * H_kv, max_splits(B, S, H_kv), tiles, d_h,
                              few_ctas(d_h, T * (H / H_kv)));
  const int nsplit = sp.n, parts = sp.cluster ? 1 : nsplit;
  // caches [B, S, H_kv, d_h] of bytes: box {128 channels, 1 head, 64 slots, 1 row}
  CUtensorMap tk, tv;
  const uint64_t dims[4] = {static_cast<uint64_t>(d_h), static_cast<uint64_t>(H_kv),
                            static_cast<uint64_t>(S), static_cast<uint64_t>(B)};
  const uint64_t str[3] = {static_cast<uint64_t>(d_h), static_cast<uint64_t>(H_kv) * d_h,
                           static_cast<uint64_t>(S) * H_kv * d_h};
  const uint32_t box[4] = {128, 1, kTile, 1};
  if (!encode_tiled(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, K8, dims, str, box) ||
      !encode_tiled(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, V8, dims, str, box))
    return cudaErrorInvalidValue;

  Params p;
  p.Q = static_cast<const __half*>(Q);
  p.K_scale = K_scale;
  p.V_scale = V_scale;
  p.posc = pos_cache;
  p.qpos = qpos;
  p.pad_lens = pad_lens;
  p.swept = window > 0 && weight_sum != nullptr ? lay.swept : nullptr;
  p.stat = parts > 1 || weight_sum != nullptr ? lay.stat : nullptr;
  p.part = lay.part;
  p.logits = weight_sum != nullptr ? lay.logits : nullptr;
  p.O = O;
  p.o_f16 = o_f16;
  p.B = B;
  p.T = T;
  p.S = S;
  p.H = H;
  p.H_kv = H_kv;
  p.nb = nb;
  p.end = end;
  p.window = window;
  p.nsplit = nsplit;
  p.cluster = sp.cluster ? 1 : 0;
  // (the last slots that positions without gaps let a window's tokens see)
  p.late = window > 0 ? tiles : INT_MAX;
  p.zero = 0;
  p.status = status;
  const dim3 grid(nsplit, H_kv, B);
  const bool one = T * (H / H_kv) <= 8;
  if (d_h == 256)
    e = one ? launch_cfg<256, 1, 1>(tk, tv, p, grid, stream)
            : launch_cfg<256, 1, 2>(tk, tv, p, grid, stream);
  else
    e = one ? launch_cfg<128, 1, 1>(tk, tv, p, grid, stream)
            : launch_cfg<128, 2, 1>(tk, tv, p, grid, stream);
  if (e != cudaSuccess) return e;

  if (parts > 1) {
    MergeParams q;
    q.stat = lay.stat;
    q.part = lay.part;
    q.fstat = weight_sum != nullptr ? lay.fstat : nullptr;
    q.O = O;
    q.o_f16 = o_f16;
    q.parts = parts;
    e = d_h == 256 ? launch_pdl(merge8_kernel<256>, dim3(B * T * H), dim3(256), 0, stream, q)
                   : launch_pdl(merge8_kernel<128>, dim3(B * T * H), dim3(128), 0, stream, q);
    if (e != cudaSuccess) return e;
  }
  if (weight_sum == nullptr) return cudaSuccess;
  const bool many = T * H > 16;
  WeighParams q;
  q.stat = parts > 1 ? lay.fstat : lay.stat;
  q.logits = lay.logits;
  q.weight_sum = weight_sum;
  q.swept = lay.swept;
  q.pad_lens = pad_lens;
  q.T = T;
  q.S = S;
  q.H = H;
  q.H_kv = H_kv;
  q.nb = nb;
  q.end = end;
  q.nsplit = nsplit;
  q.late = p.late;
  q.status = status;
  q.lost = lost;
  q.wchunks = (hi + (many ? 128 : 512) - 1) / (many ? 128 : 512);
  const long long ctas = static_cast<long long>(B) * q.wchunks;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(many ? weigh8_kernel<4> : weigh8_kernel<1>, dim3(static_cast<unsigned>(ctas)),
                    dim3(256), 0, stream, q);
}

}  // namespace g3
