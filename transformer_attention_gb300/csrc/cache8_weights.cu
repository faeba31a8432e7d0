// The weight that each slot of the 8-bit cache received from many query rows
// (a prompt or a chunk), after the attention has left every row's reference
// (near its maximum) and sum: weight_sum[s] += sum over rows of exp2(l_s -
// reference) / sum.  The logits are computed again from K (half the attention's
// products and no V) because keeping them would take 4 bytes per query row and
// slot.
//
// The product is transposed, S^T = K Q^T with 128 slots on the tensor core's
// 128 rows: a thread owns a slot and sums over the query rows in its own
// registers.  A CTA owns 128 slots of a batch row and a run of (kv head, row
// tile) pairs; it converts K once per head (cache8_flash.cuh) and streams Q
// tiles by TMA.  Each tile's 128 terms are summed on their own and then added,
// always in the same order; several CTAs on one slot tile write parts that a
// last launch adds.  Bound by the way of a Q tile through the pipeline, copy,
// MMA and sums, not by any one of them: 24 us for 515 tokens, 16 heads, window
// 1024, whose products take 5, and 429 us for 1024 tokens over 32768 slots,
// 27B-shaped, whose products take 143 (without exponentials, row statistics
// and MMA 260).  Four warpgroups of sums bring the long call to 390 us, two slot
// tiles per CTA to 370; either costs short ones 2 us.
//
// Warps: 0 TMA of Q, 1 MMA issue, 4-7 converters, 8-11 and 12-15 the sums of
// even and odd tiles.  TMEM: four S^T buffers of 128 columns.
#include <algorithm>
#include <climits>

#include "attention_common.cuh"
#include "cache8.cuh"
#include "cache8_flash.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace g3 {

namespace {

using attn::ex2;

constexpr int THREADS = 512;
constexpr int BM = 128, BN = 128;
constexpr uint32_t CHUNK = 128 * 128;
constexpr uint32_t PART = 32768;
constexpr float LOG2E = 1.4426950408889634f;
constexpr int NS = 4;                        // S^T buffers

enum : int {
  kSiteQFull = 100, kSiteQEmpty, kSiteKFull, kSiteKEmpty, kSiteSFull, kSiteSEmpty
};

template <int DH, int G>
struct Cfg {
  static constexpr int TQ = BN / G;                      // tokens per row tile
  static constexpr int NCH = DH / 64;
  static constexpr int PARTS = DH / 128;
  static constexpr uint32_t QT_BYTES = BN * DH * 2;
  static constexpr int KB = 2 / PARTS;                   // K tiles held
  static constexpr int QB = 4 / PARTS;                   // Q tiles held
  static constexpr uint32_t SMEM = KB * PARTS * PART + QB * QT_BYTES + 1024;
  static_assert(SMEM + 8192 <= 232448, "shared memory budget");
};

struct Params {
  const uint8_t* K8;
  const float* K_scale;
  const int32_t* posc;
  const int32_t* qpos;
  const int32_t* pad_lens;
  const float2* rowstat;      // [B, H_kv, T*G] (reference, 1 / sum), (inf, 0) for a row of no weight
  float* weight_sum;          // [B, S]
  float* wpart;               // [usplit, B, tiles * 128] when usplit > 1
  int B, T, S, H, H_kv, nb, end, window, usplit, tiles;
  int* status;
  int lost;
};

template <int DH, int G>
__global__ void __launch_bounds__(THREADS, 1)
    weights8_kernel(const __grid_constant__ CUtensorMap tmQ, const Params p) {
  pdl_enter();
  using C = Cfg<DH, G>;
  const bool lost = lost_work(p.status, p.lost);      // (under way until the first barrier)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;
  uint8_t* sQ = smem + C::KB * C::PARTS * PART;
  __shared__ __align__(8) uint64_t q_full[C::QB], q_empty[C::QB], k_full[C::KB], k_empty[C::KB],
      s_full[NS], s_empty[NS], drain;
  __shared__ __align__(16) float2 rs[2][2][BN];   // [warpgroup][tile parity] row statistics
  __shared__ int sq[2][2][BN];               // query positions of the tile's tokens
  __shared__ float other[BM];
  __shared__ int pr[4];                      // min / max position, first / last token
  __shared__ int any_halves;                 // does a K tile hold halves (tile_scale)?
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_flag;

  // the latest slots first: on a local layer the early tiles have no work
  const int us = blockIdx.x % p.usplit, b = (blockIdx.x / p.usplit) % p.B;
  const int st = p.tiles - 1 - static_cast<int>(blockIdx.x) / p.usplit / p.B;
  const int valid = min(p.T, p.T - (p.pad_lens != nullptr ? __ldcg(p.pad_lens + b) : 0));
  const int s_tile = st * BM, hi = valid > 0 ? p.end + valid : 0;

  if (tid == 0) {
    for (int s = 0; s < C::QB; ++s) {
      mbar_init(smem_u32(&q_full[s]), 1);
      mbar_init(smem_u32(&q_empty[s]), 1);
    }
    for (int s = 0; s < C::KB; ++s) {
      mbar_init(smem_u32(&k_full[s]), 4);
      mbar_init(smem_u32(&k_empty[s]), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&s_full[s]), 1);
      mbar_init(smem_u32(&s_empty[s]), 4);
    }
    mbar_init(smem_u32(&drain), 1);
    abort_flag = 0;
    pr[0] = INT_MAX;
    pr[1] = -1;
    pr[2] = INT_MAX;
    pr[3] = -1;
    any_halves = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_sh), 512);
    tmem_relinquish();
  }
  if (__syncthreads_or(lost)) {
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_sh, 512);
    return;
  }
  if (warp < 4) {
    const int s = s_tile + tid;
    const int ps = s < hi ? __ldcg(p.posc + static_cast<size_t>(b) * p.S + s) : -1;
    const int mn = __reduce_min_sync(0xffffffffu, ps >= 0 ? ps : INT_MAX);
    const int mx = __reduce_max_sync(0xffffffffu, ps);
    if (lane == 0 && mx >= 0) {
      atomicMin(&pr[0], mn);
      atomicMax(&pr[1], mx);
    }
  } else {
    // the scales of the tile's blocks, heads next to each other
    const int n = (min(s_tile / kC8Block + 2, p.nb) - s_tile / kC8Block) * p.H_kv;
    const float* sc = p.K_scale + (static_cast<size_t>(b) * p.nb + s_tile / kC8Block) * p.H_kv;
    for (int i = tid - 128; i < n; i += THREADS - 128)
      if (halved(__ldcg(sc + i))) any_halves = 1;
  }
  __syncthreads();
  // The tokens that may see a slot of the tile.
  const int pmin = pr[0], pmax = pr[1];
  int tmin = INT_MAX, tmax = -1;
  if (pmax >= 0) {
    for (int t = max(0, s_tile - p.end) + tid; t < valid; t += THREADS) {
      bool see = true;
      if (p.window > 0) {
        const int q = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t);
        int plo, phi;
        window_range(q, q, p.window, plo, phi);
        see = plo <= pmax && phi >= pmin;
      }
      if (see) {
        tmin = min(tmin, t);
        tmax = max(tmax, t);
      }
    }
  }
  tmin = __reduce_min_sync(0xffffffffu, tmin);
  tmax = __reduce_max_sync(0xffffffffu, tmax);
  if (lane == 0 && tmax >= 0) {
    atomicMin(&pr[2], tmin);
    atomicMax(&pr[3], tmax);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_sh;
  // This CTA's run of units (kv head, row tile).
  const int rt0 = pr[3] >= 0 ? pr[2] / C::TQ : 0;
  const int nrt = pr[3] >= 0 ? pr[3] / C::TQ - rt0 + 1 : 0;
  const long long units = static_cast<long long>(p.H_kv) * nrt;
  const int u0 = static_cast<int>(units * us / p.usplit);
  const int u1 = static_cast<int>(units * (us + 1) / p.usplit);
  const int n_units = u1 - u0;
  auto head_of = [&](int u) { return u / nrt; };
  auto tile_of = [&](int u) { return rt0 + u % nrt; };
  auto wait_warp = [&](uint64_t& bar, int parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar), parity, &abort_flag, p.status, site));
  };

  float total = 0.f;
  if (warp == 0) {
    if (lane == 0) {
      // ---------------- Q tiles
      int issued = 0;
      for (int n = 0; n < n_units; ++n) {
        const int qb = n % C::QB, u = u0 + n;
        if (!mbar_wait(smem_u32(&q_empty[qb]), ((n / C::QB) & 1) ^ 1, &abort_flag, p.status,
                       kSiteQEmpty))
          break;
        const uint32_t bar = smem_u32(&q_full[qb]);
        mbar_arrive_expect_tx(bar, C::QT_BYTES);
        for (int ch = 0; ch < C::NCH; ++ch)
          tma_load_4d(smem_u32(sQ + qb * C::QT_BYTES + ch * CHUNK), &tmQ, bar, ch * 64,
                      head_of(u) * G, tile_of(u) * C::TQ, b);
        ++issued;
      }
      for (int n = max(0, issued - C::QB); n < issued; ++n)
        mbar_wait_drain(smem_u32(&q_full[n % C::QB]), (n / C::QB) & 1);
    }
  } else if (warp == 1) {
    // ---------------- MMA issue
    if (n_units > 0) {
      const uint32_t lead = elect_one();
      constexpr uint32_t idesc = idesc_f16(BM, BN, /*f16*/ 0, 0, 0);
      int hh = -1;
      for (int n = 0; n < n_units; ++n) {
        const int u = u0 + n, qb = n % C::QB, sb = n % NS;
        if (n == 0 || head_of(u) != head_of(u - 1)) {
          ++hh;
          if (!wait_warp(k_full[hh % C::KB], (hh / C::KB) & 1, kSiteKFull)) break;
        }
        if (!wait_warp(q_full[qb], (n / C::QB) & 1, kSiteQFull)) break;
        if (!wait_warp(s_empty[sb], ((n / NS) & 1) ^ 1, kSiteSEmpty)) break;
        tc_fence_after();
        const uint32_t ka = smem_u32(sK) + (hh % C::KB) * C::PARTS * PART;
        const uint32_t qa = smem_u32(sQ) + qb * C::QT_BYTES;
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint32_t off = (k >> 2) * CHUNK + (k & 3) * 32;
          mma_ss_lead(lead, tbase + sb * BN, sdesc_sw128(ka + off, 16, 1024),
                      sdesc_sw128(qa + off, 16, 1024), idesc, k > 0 ? 1u : 0u);
        }
        mma_commit_lead(lead, smem_u32(&q_empty[qb]));
        mma_commit_lead(lead, smem_u32(&s_full[sb]));
        if (n + 1 < n_units && head_of(u + 1) != head_of(u))
          mma_commit_lead(lead, smem_u32(&k_empty[hh % C::KB]));
      }
      mma_commit_lead(lead, smem_u32(&drain));
      mbar_wait_drain(smem_u32(&drain), 0);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------- converters: the tile's K, once per head
    const int ct = tid - 128;
    const uint8_t* num = p.K8 + static_cast<size_t>(b) * p.S * p.H_kv * DH + (ct % 8) * 16;
    const float* sc = p.K_scale + static_cast<size_t>(b) * p.nb * p.H_kv;
    const int32_t* posr = p.posc + static_cast<size_t>(b) * p.S;
    if (n_units > 0) {
      const int h_first = head_of(u0), n_parts = (head_of(u1 - 1) - h_first + 1) * C::PARTS;
      const int row0 = ct / 8, blk = s_tile / kC8Block;
      uint32_t ok = 0;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int s = s_tile + row0 + it * 16;
        ok |= (s < hi && __ldcg(posr + s) >= 0 ? 1u : 0u) << it;
      }
      // a part: 128 slots x 128 channels, 128 bytes per thread
      uint2 x[8][2];
      const int swap = swap8(ct % 8, row0);
      float sc0 = 0.f, sc1 = 0.f;
      auto fetch = [&](int q) {
        const int h = h_first + q / C::PARTS;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          x[it][0] = x[it][1] = make_uint2(0, 0);
          if ((ok >> it) & 1u) {
            const uint2* src = reinterpret_cast<const uint2*>(
                num + static_cast<size_t>(s_tile + row0 + it * 16) * p.H_kv * DH + h * DH +
                (q % C::PARTS) * 128);
            x[it][0] = __ldcg(src + swap);
            x[it][1] = __ldcg(src + 1 - swap);
          }
        }
        sc0 = __ldcg(sc + static_cast<size_t>(blk) * p.H_kv + h);
        sc1 = __ldcg(sc + static_cast<size_t>(min(blk + 1, p.nb - 1)) * p.H_kv + h);
      };
      fetch(0);
      for (int q = 0; q < n_parts; ++q) {
        const int hh = q / C::PARTS, part = q % C::PARTS, kb = hh % C::KB;
        if (part == 0 && !wait_warp(k_empty[kb], ((hh / C::KB) & 1) ^ 1, kSiteKEmpty)) break;
        uint8_t* dst = sK + (kb * C::PARTS + part) * PART + ((ct % 8) >> 2) * CHUNK;
        // (finite where a block holds no token: the bytes are zeros there)
        const __half2 h0 = tile_scale(fminf(fabsf(sc0), 256.f)), h1 = tile_scale(fminf(fabsf(sc1), 256.f));
#pragma unroll
        for (int it = 0; it < 8; ++it)
          store16_values(x[it][0], x[it][1], it >= 4 ? h1 : h0, ct % 8, row0 + it * 16,
                         dst + (row0 + it * 16) * 128);
        if (part == C::PARTS - 1)
          publish8(k_full[kb], lane);
        else
          fence_proxy_async_smem();
        if (q + 1 < n_parts) fetch(q + 1);
      }
    }
  } else if (warp >= 8) {
    // ---------------- sums: warpgroup wg takes every other tile, thread = slot
    const int wg = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int s = s_tile + r;
    const int ps = s < hi ? __ldcg(p.posc + static_cast<size_t>(b) * p.S + s) : -1;
    // query positions that see this slot on a local layer (negative ones too:
    // only a stored position below 0 means that there is no token)
    int qlo = INT_MIN, qhi = INT_MAX;
    if (p.window > 0 && ps >= 0) {
      qlo = ps - (p.window - 1);
      qhi = ps > INT_MAX - (p.window - 1) ? INT_MAX : ps + (p.window - 1);
    }
    const size_t rows = static_cast<size_t>(p.T) * G;
    // the slot's K scale of the unit's head: what its logits count (tile_scale)
    const float* sc = p.K_scale + (static_cast<size_t>(b) * p.nb + min(s / kC8Block, p.nb - 1)) * p.H_kv;
    float2 nx = make_float2(INFINITY, 0.f);
    const bool halves = any_halves != 0;
    int nq = 0;
    auto fetch = [&](int n) {
      if (n >= n_units) return;
      const int j = head_of(u0 + n), t0 = tile_of(u0 + n) * C::TQ;
      const size_t row = static_cast<size_t>(t0) * G + r;
      nx = row < rows ? __ldcg(p.rowstat + (static_cast<size_t>(b) * p.H_kv + j) * rows + row)
                      : make_float2(INFINITY, 0.f);
      if (p.window > 0 && r < C::TQ && t0 + r < p.T)
        nq = __ldcg(p.qpos + static_cast<size_t>(b) * p.T + t0 + r);
    };
    fetch(wg);
    bool ok = true;
    for (int n = wg; n < n_units; n += 2) {
      const int par = (n >> 1) & 1, sb = n % NS;
      rs[wg][par][r] = nx;
      if (r < C::TQ) sq[wg][par][r] = nq;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
      fetch(n + 2);
      // (a warp whose wait gave up still meets the barriers of the others)
      ok = ok && wait_warp(s_full[sb], (n / NS) & 1, kSiteSFull);
      if (!ok) continue;
      tc_fence_after();
      const int t0 = tile_of(u0 + n) * C::TQ;
      float by = LOG2E;
      if (halves) by = halved(__ldcg(sc + head_of(u0 + n))) ? 2.f * LOG2E : LOG2E;
      // columns [c0, c1) are valid tokens at or behind this slot
      const int n_tok = max(0, min(C::TQ, valid - t0));
      int c0 = max(0, min(C::TQ, s - p.end - t0)) * G, c1 = n_tok * G;
      bool runs = true;              // the columns that see the slot are a run
      if (p.window > 0) {
        const int q0 = sq[wg][par][0];
        bool step = true;            // tokens at positions q0, q0 + 1, ..
        for (int k = lane; k < n_tok; k += 32)
          step &= static_cast<unsigned>(sq[wg][par][k]) == static_cast<unsigned>(q0) + k;
        runs = __all_sync(0xffffffffu, step);
        if (runs && ps >= 0) {
          const long long a = static_cast<long long>(qlo) - q0, z = static_cast<long long>(qhi) - q0 + 1;
          c0 = max(c0, static_cast<int>(min(max(a, 0LL), static_cast<long long>(C::TQ))) * G);
          c1 = min(c1, static_cast<int>(min(max(z, 0LL), static_cast<long long>(C::TQ))) * G);
        }
      }
      // (a slot without a token: whatever it sums is dropped)
      if (ps < 0) {
        c0 = 0;
        c1 = BN;
      }
      const int w0 = __reduce_max_sync(0xffffffffu, c0), w1 = __reduce_min_sync(0xffffffffu, c1);
      const int any0 = __reduce_min_sync(0xffffffffu, ps < 0 ? BN : c0);
      const int any1 = __reduce_max_sync(0xffffffffu, ps < 0 ? 0 : c1);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4* st4 = reinterpret_cast<const float4*>(rs[wg][par]);
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        // (no column of the 32 counts for any slot of the warp)
        if (c + 32 <= any0 || c >= any1) continue;
        uint32_t x[32];
        tmem_ld32(tbase + lane_off + sb * BN + c, x);
        tmem_ld_wait(x);
        if (runs) {
          if (c < w0 || c + 32 > w1) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (c + k < c0 || c + k >= c1) x[k] = 0xff800000u;   // -inf
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int qp = sq[wg][par][(c + k) / G];
            const bool see = c + k >= c0 && c + k < c1 && qp >= qlo && qp <= qhi;
            if (!see) x[k] = 0xff800000u;   // -inf
          }
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float4 a = st4[(c + k) >> 1];       // rows k and k + 1
          const float e0 = ex2(fmaf(__uint_as_float(x[k]), by, -a.x));
          const float e1 = ex2(fmaf(__uint_as_float(x[k + 1]), by, -a.z));
          if (k & 2) {
            acc.z = fmaf(e0, a.y, acc.z);
            acc.w = fmaf(e1, a.w, acc.w);
          } else {
            acc.x = fmaf(e0, a.y, acc.x);
            acc.y = fmaf(e1, a.w, acc.y);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_empty[sb]));
      total += (acc.x + acc.y) + (acc.z + acc.w);
    }
    if (ps < 0) total = 0.f;
    if (wg == 1) other[r] = total;
  }
  __syncthreads();
  if (warp >= 8 && warp < 12) {
    const int r = tid - 256, s = s_tile + r;
    total += other[r];
    if (p.usplit > 1)
      p.wpart[(static_cast<size_t>(us) * p.B + b) * p.tiles * BM + s] = total;
    else if (s < hi && total != 0.f && !abort_flag) {
      float* w = p.weight_sum + static_cast<size_t>(b) * p.S + s;
      *w = __ldcg(w) + total;
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

__global__ void __launch_bounds__(256) wadd8_kernel(const float* __restrict__ wpart, int usplit,
                                                    int B, int ld, int hi, int S,
                                                    float* __restrict__ weight_sum,
                                                    const int* status, int lost) {
  pdl_enter();
  const bool stop = lost_work(status, lost);   // parts may be missing
  const int s = blockIdx.x * 256 + threadIdx.x, b = blockIdx.y;
  if (s >= hi) return;
  float a = 0.f;
  for (int k = 0; k < usplit; ++k) a += __ldcg(wpart + (static_cast<size_t>(k) * B + b) * ld + s);
  float* w = weight_sum + static_cast<size_t>(b) * S + s;
  if (a != 0.f && !stop) *w = __ldcg(w) + a;
}

template <int DH, int G>
cudaError_t launch_cfg(const void* Q, const Params& p, cudaStream_t stream) {
  using C = Cfg<DH, G>;
  CUtensorMap tq;
  const uint64_t dims[4] = {static_cast<uint64_t>(DH), static_cast<uint64_t>(p.H),
                            static_cast<uint64_t>(p.T), static_cast<uint64_t>(p.B)};
  const uint64_t str[3] = {static_cast<uint64_t>(DH) * 2, static_cast<uint64_t>(p.H) * DH * 2,
                           static_cast<uint64_t>(p.T) * p.H * DH * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(C::TQ), 1};
  if (!encode_tiled(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, Q, dims, str, box))
    return cudaErrorInvalidValue;
  auto kern = weights8_kernel<DH, G>;
  if (cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), C::SMEM)) return e;
  const long long ctas = static_cast<long long>(p.tiles) * p.B * p.usplit;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), C::SMEM, stream, tq, p);
}

// CTAs on one slot tile, while their parts fit the scratch: where the rounds
// of the SMs end earliest, counted in units, with the start and the end of a
// CTA worth kStart.  On a local layer without gaps only the slots of the
// window and the new tokens have work, and of the row tiles those that a
// window reaches.
constexpr int kStart = 8;

int split_units(const Flash8Args& a, int tiles) {
  const long long all = static_cast<long long>(tiles) * a.B;
  const int tq = BN / (a.H / a.H_kv);
  long long busy = tiles, nrt = (a.T + tq - 1) / tq;
  if (a.window > 0) {
    busy = std::min<long long>(busy, (static_cast<long long>(a.window) + a.T + BM - 1) / BM + 1);
    nrt = std::min<long long>(nrt, (static_cast<long long>(a.window) + BM + tq - 1) / tq + 1);
  }
  const long long units = nrt * a.H_kv, most = std::min({units, kWeights8MaxCtas / all, 64LL});
  const int sms = num_sms();
  long long best = LLONG_MAX;
  int split = 1;
  for (int n = 1; n <= most; ++n) {
    const long long rounds = (busy * a.B * n + sms - 1) / sms;
    const long long cost = rounds * (kStart + (units + n - 1) / n);
    if (cost < best) {
      best = cost;
      split = n;
    }
  }
  return split;
}

}  // namespace

cudaError_t launch_weights8(const Flash8Args& a, float* wpart, float* weight_sum,
                            cudaStream_t stream) {
  const int G = a.H / a.H_kv;
  cudaError_t e = cudaErrorInvalidValue;
  Params p;
  p.K8 = static_cast<const uint8_t*>(a.K8);
  p.K_scale = a.K_scale;
  p.posc = a.posc;
  p.qpos = a.qpos;
  p.pad_lens = a.pad_lens;
  p.rowstat = a.rowstat;
  p.weight_sum = weight_sum;
  p.wpart = wpart;
  p.B = a.B;
  p.T = a.T;
  p.S = a.S;
  p.H = a.H;
  p.H_kv = a.H_kv;
  p.nb = c8_blocks(a.S);
  p.end = a.end;
  p.window = a.window;
  p.status = a.status;
  p.lost = a.lost;
  p.tiles = (a.end + a.T + BM - 1) / BM;
  p.usplit = split_units(a, p.tiles);
#define G3_WEIGHTS8_CASE(DH_, G_) \
  if (a.d_h == DH_ && G == G_) e = launch_cfg<DH_, G_>(a.Q, p, stream);
  G3_WEIGHTS8_CASE(128, 1)
  G3_WEIGHTS8_CASE(128, 2)
  G3_WEIGHTS8_CASE(128, 4)
  G3_WEIGHTS8_CASE(256, 1)
  G3_WEIGHTS8_CASE(256, 2)
  G3_WEIGHTS8_CASE(256, 4)
#undef G3_WEIGHTS8_CASE
  if (e != cudaSuccess || p.usplit == 1) return e;
  return launch_pdl(wadd8_kernel, dim3((a.end + a.T + 255) / 256, a.B), dim3(256), 0, stream,
                    static_cast<const float*>(wpart), p.usplit, a.B, p.tiles * BM, a.end + a.T, a.S,
                    weight_sum, static_cast<const int*>(a.status), a.lost);
}

}  // namespace g3
