// The 8-bit KV cache's storage: write of new tokens, read-back as fp16, and
// eviction into another cache (numbers and scales: cache8.cuh).
//
// All three move each byte once and are bound by HBM; a call of one token or
// a small cache is bound by its launch and one or two memory round trips.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "cache8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace g3 {

namespace {

constexpr int kTile = kC8Block;
constexpr int kRowThreads = 256;

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kRowThreads / 32; ++i) v = fmaxf(v, red[i]);
  return v;
}

// Largest finite magnitude of eight fp16 values.
__device__ __forceinline__ float finite_max8(const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
    m = max(m, a < 0x7C00u ? a : 0u);
    m = max(m, b < 0x7C00u ? b : 0u);
  }
  return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
}

__device__ __forceinline__ uint2 pack8(const uint4& r, float inv) {
  const __half2* h = reinterpret_cast<const __half2*>(&r);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(h[i]);
    f[2 * i] = v.x * inv;
    f[2 * i + 1] = v.y * inv;
  }
  return make_uint2(c8_pack4(f[0], f[1], f[2], f[3]), c8_pack4(f[4], f[5], f[6], f[7]));
}

// ---------------------------------------------------------------- write
struct WriteParams {
  const __half* K_rows;
  const __half* V_rows;
  long ld;
  const int32_t* segment_pos;
  const int32_t* pad_lens;
  int T, S, end, H_kv, blk0, nblk, nb;   // nb: blocks of a cache row
  uint8_t* K8;
  uint8_t* V8;
  float* K_scale;
  float* V_scale;
  int32_t* posc;
  const int* status;          // or null
  int lost;
};

// One CTA per (block of 64 slots, kv head, K' or V, batch row): the block's
// new rows stay in registers between the search for their largest magnitude
// and the rounding, so each is read once.  Only a block that held tokens
// before and whose scale grows reads its older numbers (one block per row and
// call at most), and no other CTA touches them.  CHECK: nothing is written once
// an error of the mask `lost` was recorded (a form of its own: 251 us instead
// of 247 for a prompt of 65536 tokens with the read-back).
template <int DH, bool CHECK>
__global__ void __launch_bounds__(kRowThreads) cache8_write_kernel(const WriteParams p) {
  pdl_enter();
  constexpr int TPR = DH / 8;                  // threads per row, 8 channels each
  constexpr int RPP = kRowThreads / TPR;       // rows per pass
  constexpr int NP = kTile / RPP;
  __shared__ float red[kRowThreads / 32];
  const int tid = threadIdx.x;
  unsigned idx = blockIdx.x;
  const int hk = idx % (2 * p.H_kv);
  idx /= 2 * p.H_kv;
  const int blk = p.blk0 + idx % p.nblk, b = idx / p.nblk;
  const int j = hk >> 1;
  const bool isv = hk & 1;
  const __half* rows = isv ? p.V_rows : p.K_rows;
  uint8_t* num = isv ? p.V8 : p.K8;
  float* scale = (isv ? p.V_scale : p.K_scale) + (static_cast<size_t>(b) * p.nb + blk) * p.H_kv + j;
  const int valid = p.T - (p.pad_lens != nullptr ? __ldcg(p.pad_lens + b) : 0);
  const int s0 = blk * kTile, c = (tid % TPR) * 8;
  const bool held = s0 < p.end;                // the block holds earlier tokens
  const float old = held ? __ldcg(scale) : 0.f;
  const bool stop = CHECK && lost_work(p.status, p.lost);

  uint4 x[NP];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = s0 + i * RPP + tid / TPR - p.end;
    x[i] = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < valid && t < p.T)
      x[i] = __ldcg(reinterpret_cast<const uint4*>(
          rows + (static_cast<size_t>(b) * p.T + t) * p.ld + static_cast<size_t>(j) * DH + c));
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) mx = fmaxf(mx, finite_max8(x[i]));
  // (also: every thread has read the old scale, and all stop if one does)
  mx = block_max(CHECK && stop ? INFINITY : mx, red);
  if (CHECK && mx == INFINITY) return;
  const float s = fmaxf(old, c8_scale_for(mx));
  const float inv = 1.f / s;
  const size_t ldc = static_cast<size_t>(p.H_kv) * DH;
  uint8_t* dst = num + (static_cast<size_t>(b) * p.S + s0) * ldc + static_cast<size_t>(j) * DH + c;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int r = i * RPP + tid / TPR, t = s0 + r - p.end;
    uint2* d = reinterpret_cast<uint2*>(dst + static_cast<size_t>(r) * ldc);
    if (t >= 0 && t < p.T) {
      *d = pack8(x[i], inv);
    } else if (t < 0 && s != old) {
      const uint2 n = __ldcg(d);
      *d = make_uint2(c8_rescale4(n.x, old * inv), c8_rescale4(n.y, old * inv));
    }
  }
  if (tid == 0) *scale = s;
  if (hk == 0 && tid < kTile) {
    const int t = s0 + tid - p.end;
    if (t >= 0 && t < p.T)
      p.posc[static_cast<size_t>(b) * p.S + s0 + tid] =
          t < valid ? __ldcg(p.segment_pos + static_cast<size_t>(b) * p.T + t) : -1;
  }
}

// ---------------------------------------------------------------- read
// Slots [first, first + n) of K (blockIdx.y even) or V of one batch row as
// fp16 rows: 16 numbers per unit, four units per thread in flight.
constexpr int kReadUnits = 4;

__global__ void __launch_bounds__(256) cache8_read_kernel(
    const uint8_t* __restrict__ K8, const uint8_t* __restrict__ V8,
    const float* __restrict__ K_scale, const float* __restrict__ V_scale, int S, int nb, int first,
    int n, int H_kv, int d_h, unsigned chunks, __half* K_rows, __half* V_rows, long ld) {
  pdl_enter();
  const unsigned row_units = H_kv * d_h / 16, head_units = d_h / 16;
  const unsigned chunk = blockIdx.x % chunks, bk = blockIdx.x / chunks;   // (batch row, K or V)
  const bool isv = bk & 1;
  const size_t b = bk >> 1;
  const uint8_t* num = (isv ? V8 : K8) + (b * S + first) * static_cast<size_t>(H_kv) * d_h;
  const float* scale = (isv ? V_scale : K_scale) + b * nb * H_kv;
  __half* rows = (isv ? V_rows : K_rows) + b * n * ld;
  // (slots x units per slot passes 2^32 only beyond any one row's 2^40 bytes / 16;
  // 64-bit unit numbers, 32-bit within a chunk)
  const size_t total = static_cast<size_t>(n) * row_units;
  const size_t base = static_cast<size_t>(chunk) * (256 * kReadUnits);
  const unsigned t0 = static_cast<unsigned>(base / row_units);
  const unsigned u0 = static_cast<unsigned>(base - static_cast<size_t>(t0) * row_units);
  uint4 v[kReadUnits];
  float s[kReadUnits];
  unsigned t[kReadUnits], u[kReadUnits];
#pragma unroll
  for (int k = 0; k < kReadUnits; ++k) {
    const unsigned i = k * 256 + threadIdx.x;
    const unsigned q = (u0 + i) / row_units;
    t[k] = t0 + q;
    u[k] = u0 + i - q * row_units;
    if (base + i < total) {
      v[k] = __ldcg(reinterpret_cast<const uint4*>(num + (static_cast<size_t>(t[k]) * row_units + u[k]) * 16));
      s[k] = __ldcg(scale + static_cast<size_t>((first + t[k]) / kC8Block) * H_kv + u[k] / head_units);
    }
  }
#pragma unroll
  for (int k = 0; k < kReadUnits; ++k) {
    if (base + k * 256 + threadIdx.x >= total) break;
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 f = c8_float2(w[e >> 1] >> ((e & 1) * 16));
      f.x *= s[k];
      f.y *= s[k];
      // beyond fp16's largest (only 65504 itself rounds there): 65504; NaN passes
      f.x = f.x > 65504.f ? 65504.f : (f.x < -65504.f ? -65504.f : f.x);
      f.y = f.y > 65504.f ? 65504.f : (f.y < -65504.f ? -65504.f : f.y);
      o[e] = pack_half2(f.x, f.y);
    }
    uint4* d = reinterpret_cast<uint4*>(rows + static_cast<size_t>(t[k]) * ld + u[k] * 16);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------- evict
// Order of the candidates as unsigned keys: 0 for a slot without a token,
// ~0 for one of the last `recent` slots, in between the weight (NaN below
// every number, -0 as 0).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int s, int first_recent) {
  const uint32_t u = __float_as_uint(w + 0.f);
  uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
  k = w != w ? 1u : k;
  k = s >= first_recent ? 0xFFFFFFFFu : k;
  return pos < 0 ? 0u : k;
}

struct SelectParams {
  const float* w;
  const int32_t* pos;
  int S, end, first_recent, keep, S_dst;
  int32_t* kept;
  int32_t* pos_dst;
  float* w_dst;
};

constexpr int kSelThreads = 1024;
constexpr int kSelSlots = 4096;      // slots per CTA worth one more CTA in the cluster
constexpr int kSelMaxCluster = 8;
constexpr int kSelKeys = 40 * 1024;  // keys that a CTA keeps in shared memory
constexpr int kSelHist = 256 * 32;   // digit counts, each lane its own

// One cluster per batch row: the keep-th largest key by four rounds of 8-bit
// digit counts (each CTA counts its run of slots, the counts are summed over
// the cluster through distributed shared memory), then the slots above it,
// and the first of those equal to it, are written out in slot order.  Weights
// and positions are read once; the keys stay in shared memory between the
// rounds (a run longer than kSelKeys is read from L2 again).  Bound by the
// rounds' latency: 131072 slots 23 us on eight CTAs, 1000 slots 11 us on one;
// their bytes take 0.2 us.  (A search bit by bit, one count over the CTA for
// each, took 15 us for the 1000.)
template <bool KEPT>
__global__ void __launch_bounds__(kSelThreads) cache8_select_kernel(const SelectParams p) {
  pdl_enter();
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), C = cluster.num_blocks();
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Counts [digit][lane]: weights of one magnitude share their first digit,
  // and lanes adding to one word would wait for each other.
  extern __shared__ int hist[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(hist + kSelHist);
  __shared__ int tot[2][256];        // this CTA's counts, for its cluster
  __shared__ int sum[256], own[32];
  __shared__ int wsum[32];
  __shared__ int counts[2];
  __shared__ int found[2][2];        // by round parity: digit, keys above it
  const float* w = p.w + static_cast<size_t>(b) * p.S;
  const int32_t* pos = p.pos + static_cast<size_t>(b) * p.S;
  int run = (p.end + C - 1) / C;
  run = (run + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int lo = static_cast<int>(min(static_cast<long long>(p.end), static_cast<long long>(rank) * run));
  const int hi = static_cast<int>(min(static_cast<long long>(p.end), static_cast<long long>(lo) + run));
  // Warp w owns the slots w0 .. w1 of the CTA's run, 32 next to each other at
  // a time (a thread reads back only keys that it stored).
  const int seg = run / 32, w0 = lo + warp * seg, w1 = min(hi, w0 + seg);
  auto fresh_key = [&](int s) { return evict_key(__ldcg(w + s), __ldcg(pos + s), s, p.first_recent); };
  if constexpr (KEPT) {
    for (int base = w0 + lane; base < w1; base += 8 * 32) {
      uint32_t k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i] = base + 32 * i < w1 ? fresh_key(base + 32 * i) : 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (base + 32 * i < w1) keys[base + 32 * i - lo] = k[i];
    }
  }
  auto key_at = [&](int s) -> uint32_t {
    if constexpr (KEPT)
      return keys[s - lo];
    else
      return fresh_key(s);
  };

  uint32_t prefix = 0;
  int want = p.keep;                 // rank still to find among keys that match the prefix
  bool all = false;                  // fewer tokens than places: keep every one
  int own_gt = 0;                    // (thread 0) keys of this CTA above the prefix
  int own_eq = 0;
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    int* h = tot[round & 1];
#pragma unroll
    for (int i = 0; i < kSelHist / kSelThreads; ++i) hist[i * kSelThreads + tid] = 0;
    __syncthreads();
#pragma unroll 4
    for (int s = w0 + lane; s < w1; s += 32) {
      const uint32_t key = key_at(s);
      if (key != 0 && (round == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8))))
        atomicAdd(&hist[((key >> shift) & 255u) * 32 + lane], 1);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = warp * 8 + i, n = __reduce_add_sync(0xffffffffu, hist[d * 32 + lane]);
      if (lane == 0) h[d] = n;
    }
    cluster.sync();
    if (tid < 256) {
      int n = 0;
#pragma unroll
      for (int r = 0; r < kSelMaxCluster; ++r)
        if (r < C) n += cluster.map_shared_rank(h, r)[tid];
      sum[tid] = n;
    }
    __syncthreads();
    int* f = found[round & 1];
    if (warp == 0) {
      // lane l holds digits 255 - 8l .. 248 - 8l, largest first
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += sum[255 - 8 * lane - i];
      int before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const int total = __shfl_sync(0xffffffffu, before, 31);
      before -= mine;
      if (lane == 0) f[0] = -1;
      __syncwarp();
      if (total >= want && before < want && before + mine >= want) {
        int above = before;
        for (int i = 0; i < 8; ++i) {
          const int d = 255 - 8 * lane - i;
          if (above + sum[d] >= want) {
            f[0] = d;
            f[1] = above;
            break;
          }
          above += sum[d];
        }
      }
      // this CTA's own keys above the digit (or all its tokens), and on it
      __syncwarp();
      const int d = f[0];
      int gt = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = 255 - 8 * lane - i;
        if (k > d) gt += h[k];
      }
      gt = __reduce_add_sync(0xffffffffu, gt);
      own_gt += gt;
      own_eq = d >= 0 ? h[d] : 0;
    }
    __syncthreads();
    if (f[0] < 0) {                  // (only in round 0)
      all = true;
      break;
    }
    prefix |= static_cast<uint32_t>(f[0]) << shift;
    want -= f[1];
  }
  // A slot stays if its key is above `prefix`, or equals it and is among the
  // first `want` that do.
  const uint32_t thr = all ? 0u : prefix;
  if (all) want = 0;
  if (tid == 0) {
    counts[0] = own_gt;
    counts[1] = own_eq;
  }
  cluster.sync();
  int gt0 = 0, eq0 = 0, n_kept = 0, n_eq = 0;
#pragma unroll
  for (int r = 0; r < kSelMaxCluster; ++r) {
    if (r >= C) break;
    const int* q = cluster.map_shared_rank(counts, r);
    const int a = q[0], e = q[1];
    if (r < rank) {
      gt0 += a;
      eq0 += e;
    }
    n_kept += a;
    n_eq += e;
  }
  n_kept += min(n_eq, want);
  cluster.sync();                    // no CTA leaves while another reads its shared memory

  int32_t* kept = p.kept + static_cast<size_t>(b) * p.keep;
  int32_t* pos_dst = p.pos_dst + static_cast<size_t>(b) * p.S_dst;
  float* w_dst = p.w_dst + static_cast<size_t>(b) * p.S_dst;
  // counts of (above, equal) of each warp's slots, and before them
  int wg = 0, we = 0;
#pragma unroll 4
  for (int s = w0 + lane; s < w1; s += 32) {
    const uint32_t key = key_at(s);
    wg += key > thr;
    we += key == thr;
  }
  wg = __reduce_add_sync(0xffffffffu, wg);
  we = want > 0 ? __reduce_add_sync(0xffffffffu, we) : 0;
  if (lane == 0) {
    wsum[warp] = wg;
    own[warp] = we;
  }
  __syncthreads();
  gt0 += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0);
  eq0 += __reduce_add_sync(0xffffffffu, lane < warp ? own[lane] : 0);
  const unsigned below = (1u << lane) - 1u;
  for (int base = w0; base < w1; base += 4 * 32) {
    // (positions and weights of four steps at once, kept or not)
    float ws[4];
    int ps[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = min(base + 32 * i + lane, w1 - 1);
      ws[i] = __ldcg(w + s);
      ps[i] = __ldcg(pos + s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = base + 32 * i + lane;
      const uint32_t key = s < w1 ? key_at(s) : 0u;
      const bool g = s < w1 && key > thr, e = s < w1 && key == thr && want > 0;
      const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
      const int ng = gt0 + __popc(bg & below), ne = eq0 + __popc(be & below);
      if (g || (e && ne < want)) {
        const int d = ng + min(ne, want);
        kept[d] = s;
        pos_dst[d] = ps[i];
        w_dst[d] = ws[i];
      }
      gt0 += __popc(bg);
      eq0 += __popc(be);
    }
  }
  for (int d = n_kept + rank * kSelThreads + tid; d < p.keep; d += C * kSelThreads) {
    kept[d] = -1;
    pos_dst[d] = -1;
    w_dst[d] = 0.f;
  }
}

struct MoveParams {
  const uint8_t* K8;
  const uint8_t* V8;
  const float* K_scale;
  const float* V_scale;
  int S, H_kv, nb, keep, nblk, S_dst, nb_dst;
  const int32_t* kept;
  uint8_t* K8_dst;
  uint8_t* V8_dst;
  float* K_scale_dst;
  float* V_scale_dst;
};

// One CTA per block of 64 kept slots, batch row and U neighbouring (kv head, K
// or V) tiles, heads fastest so that the CTAs at work at one time read whole
// slots.  The numbers stay in registers between the search for the largest
// value and the move to the block's own scale; a chain of three memory round
// trips (which slots, their numbers, the stores) is paid once for U tiles.
// (One tile per CTA: 115 us for 268 MB each way, four: 105 us.)
template <int DH, int U>
__global__ void __launch_bounds__(kRowThreads) cache8_move_kernel(const MoveParams p) {
  pdl_enter();
  constexpr int TPR = DH / 16;                 // threads per row, 16 channels each
  constexpr int RPP = kRowThreads / TPR;
  constexpr int NP = kTile / RPP;
  __shared__ float red[U][kRowThreads / 32];
  const int tid = threadIdx.x, n_hk = 2 * p.H_kv, groups = (n_hk + U - 1) / U;
  unsigned idx = blockIdx.x;
  const int hk0 = idx % groups * U;
  idx /= groups;
  const int blk = idx % p.nblk, b = idx / p.nblk;
  const int c = (tid % TPR) * 16;
  const size_t ldc = static_cast<size_t>(p.H_kv) * DH;
  const size_t src0 = static_cast<size_t>(b) * p.S * ldc, sc0 = static_cast<size_t>(b) * p.nb * p.H_kv;

  int from[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int d = blk * kTile + i * RPP + tid / TPR;
    from[i] = d < p.keep ? __ldcg(p.kept + static_cast<size_t>(b) * p.keep + d) : -1;
  }
  uint4 n[U][NP];
  float sc[U][NP];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hk = hk0 + u, j = hk >> 1;
    const bool isv = hk & 1;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      n[u][i] = make_uint4(0, 0, 0, 0);
      sc[u][i] = 0.f;
      if (hk < n_hk && from[i] >= 0) {
        n[u][i] = __ldcg(reinterpret_cast<const uint4*>(
            (isv ? p.V8 : p.K8) + src0 + static_cast<size_t>(from[i]) * ldc + j * DH + c));
        sc[u][i] = __ldcg((isv ? p.V_scale : p.K_scale) + sc0 +
                         static_cast<size_t>(from[i] / kC8Block) * p.H_kv + j);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      // e4m3 magnitudes order like their codes; 0x7f is NaN
      const uint32_t w[4] = {n[u][i].x, n[u][i].y, n[u][i].z, n[u][i].w};
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t a = w[k] & 0x7F7F7F7Fu;
        a &= ~__vcmpeq4(a, 0x7F7F7F7Fu);
        m = __vmaxu4(m, a);
      }
      m = __vmaxu4(m, m >> 16);
      m = max(m & 0xFFu, (m >> 8) & 0xFFu);
      mx = fmaxf(mx, c8_float2(m).x * sc[u][i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[u][tid >> 5] = mx;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int hk = hk0 + u, j = hk >> 1;
    if (hk >= n_hk) break;
    const bool isv = hk & 1;
    float mx = red[u][0];
#pragma unroll
    for (int i = 1; i < kRowThreads / 32; ++i) mx = fmaxf(mx, red[u][i]);
    const float s = c8_scale_for(mx), inv = 1.f / s;
    uint8_t* dst = (isv ? p.V8_dst : p.K8_dst) + static_cast<size_t>(b) * p.S_dst * ldc + j * DH + c;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int d = blk * kTile + i * RPP + tid / TPR;
      if (d >= p.keep) continue;
      const float ratio = sc[u][i] * inv;
      uint4 v = n[u][i];
      if (ratio != 1.f)
        v = make_uint4(c8_rescale4(v.x, ratio), c8_rescale4(v.y, ratio), c8_rescale4(v.z, ratio),
                       c8_rescale4(v.w, ratio));
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(d) * ldc) = v;
    }
    if (tid == 0)
      (isv ? p.V_scale_dst : p.K_scale_dst)[(static_cast<size_t>(b) * p.nb_dst + blk) * p.H_kv + j] = s;
  }
}

}  // namespace

cudaError_t launch_cache8_write(const void* K_rows, const void* V_rows, long ld,
                                const int32_t* segment_pos, const int32_t* pad_lens, int B, int T,
                                int S, int end, int H_kv, int d_h, void* K8, void* V8,
                                float* K_scale, float* V_scale, int32_t* pos_cache,
                                cudaStream_t stream, const int* status, int lost) {
  WriteParams p;
  p.K_rows = static_cast<const __half*>(K_rows);
  p.V_rows = static_cast<const __half*>(V_rows);
  p.ld = ld;
  p.segment_pos = segment_pos;
  p.pad_lens = pad_lens;
  p.T = T;
  p.S = S;
  p.end = end;
  p.H_kv = H_kv;
  p.blk0 = end / kC8Block;
  p.nblk = (end + T - 1) / kC8Block - p.blk0 + 1;
  p.nb = c8_blocks(S);
  p.K8 = static_cast<uint8_t*>(K8);
  p.V8 = static_cast<uint8_t*>(V8);
  p.K_scale = K_scale;
  p.V_scale = V_scale;
  p.posc = pos_cache;
  p.status = status;
  p.lost = lost;
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(B) * p.nblk * H_kv * 2));
  const auto kern = d_h == 256
                        ? (status != nullptr ? cache8_write_kernel<256, true> : cache8_write_kernel<256, false>)
                        : (status != nullptr ? cache8_write_kernel<128, true> : cache8_write_kernel<128, false>);
  return launch_pdl(kern, grid, dim3(kRowThreads), 0, stream, p);
}

cudaError_t launch_cache8_read(const void* K8, const void* V8, const float* K_scale,
                               const float* V_scale, int B, int S, int first, int n, int H_kv,
                               int d_h, void* K_rows, void* V_rows, long ld, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const size_t units = static_cast<size_t>(n) * (H_kv * d_h / 16);
  const size_t chunks = (units + 256 * kReadUnits - 1) / (256 * kReadUnits);
  if (chunks * B * 2 > INT_MAX) return cudaErrorInvalidValue;
  return launch_pdl(cache8_read_kernel, dim3(static_cast<unsigned>(chunks * B * 2)), dim3(256), 0,
                    stream, static_cast<const uint8_t*>(K8), static_cast<const uint8_t*>(V8), K_scale,
                    V_scale, S, c8_blocks(S), first, n, H_kv, d_h, static_cast<unsigned>(chunks),
                    static_cast<__half*>(K_rows), static_cast<__half*>(V_rows), ld);
}

cudaError_t launch_cache8_evict(const void* K8, const void* V8, const float* K_scale,
                                const float* V_scale, const int32_t* pos_cache,
                                const float* weight_sum, int B, int S, int end, int H_kv, int d_h,
                                int keep, int recent, void* K8_dst, void* V8_dst,
                                float* K_scale_dst, float* V_scale_dst, int32_t* pos_dst,
                                float* weight_dst, int32_t* kept, int S_dst,
                                cudaStream_t stream) {
  SelectParams q;
  q.w = weight_sum;
  q.pos = pos_cache;
  q.S = S;
  q.end = end;
  q.first_recent = end - recent;
  q.keep = keep;
  q.S_dst = S_dst;
  q.kept = kept;
  q.pos_dst = pos_dst;
  q.w_dst = weight_dst;
  int cl = 1;
  while (cl < kSelMaxCluster && static_cast<long long>(cl) * kSelSlots < end) cl *= 2;
  const int run = ((end + cl - 1) / cl + kSelThreads - 1) / kSelThreads * kSelThreads;
  const bool kept_keys = run <= kSelKeys;
  const auto kern = kept_keys ? cache8_select_kernel<true> : cache8_select_kernel<false>;
  cudaError_t e = prepare_kernel(reinterpret_cast<const void*>(kern), (kSelHist + kSelKeys) * 4);
  if (e != cudaSuccess) return e;
  e = launch_pdl_cluster(kern, dim3(cl, B), dim3(kSelThreads),
                         static_cast<size_t>(kSelHist + (kept_keys ? run : 0)) * 4, cl, stream, q);
  if (e != cudaSuccess) return e;
  MoveParams p;
  p.K8 = static_cast<const uint8_t*>(K8);
  p.V8 = static_cast<const uint8_t*>(V8);
  p.K_scale = K_scale;
  p.V_scale = V_scale;
  p.S = S;
  p.H_kv = H_kv;
  p.nb = c8_blocks(S);
  p.keep = keep;
  p.nblk = c8_blocks(keep);
  p.S_dst = S_dst;
  p.nb_dst = c8_blocks(S_dst);
  p.kept = kept;
  p.K8_dst = static_cast<uint8_t*>(K8_dst);
  p.V8_dst = static_cast<uint8_t*>(V8_dst);
  p.K_scale_dst = K_scale_dst;
  p.V_scale_dst = V_scale_dst;
  const int u = d_h == 256 ? 2 : 4;
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(B) * p.nblk * ((2 * H_kv + u - 1) / u)));
  return launch_pdl(d_h == 256 ? cache8_move_kernel<256, 2> : cache8_move_kernel<128, 4>, grid,
                    dim3(kRowThreads), 0, stream, p);
}

}  // namespace g3
