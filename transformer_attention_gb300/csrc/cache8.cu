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
};

// One CTA per (block of 64 slots, kv head, K' or V, batch row): the block's
// new rows stay in registers between the search for their largest magnitude
// and the rounding, so each is read once.  Only a block that held tokens
// before and whose scale grows reads its older numbers (one block per row and
// call at most), and no other CTA touches them.
template <int DH>
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
  const int valid = p.T - (p.pad_lens != nullptr ? p.pad_lens[b] : 0);
  const int s0 = blk * kTile, c = (tid % TPR) * 8;
  const bool held = s0 < p.end;                // the block holds earlier tokens
  const float old = held ? *scale : 0.f;

  uint4 x[NP];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = s0 + i * RPP + tid / TPR - p.end;
    x[i] = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < valid && t < p.T)
      x[i] = __ldg(reinterpret_cast<const uint4*>(
          rows + (static_cast<size_t>(b) * p.T + t) * p.ld + static_cast<size_t>(j) * DH + c));
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) mx = fmaxf(mx, finite_max8(x[i]));
  mx = block_max(mx, red);                     // (also: every thread has read the old scale)
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
      const uint2 n = *d;
      *d = make_uint2(c8_rescale4(n.x, old * inv), c8_rescale4(n.y, old * inv));
    }
  }
  if (tid == 0) *scale = s;
  if (hk == 0 && tid < kTile) {
    const int t = s0 + tid - p.end;
    if (t >= 0 && t < p.T)
      p.posc[static_cast<size_t>(b) * p.S + s0 + tid] =
          t < valid ? p.segment_pos[static_cast<size_t>(b) * p.T + t] : -1;
  }
}

// ---------------------------------------------------------------- read
// Slots [first, first + n) of every row as fp16 rows: 16 numbers per thread.
__global__ void __launch_bounds__(256) cache8_read_kernel(
    const uint8_t* __restrict__ K8, const uint8_t* __restrict__ V8,
    const float* __restrict__ K_scale, const float* __restrict__ V_scale, long total, int S,
    int nb, int first, int n, int H_kv, int d_h, __half* K_rows, __half* V_rows, long ld) {
  pdl_enter();
  const int units = H_kv * d_h / 16;           // 16-byte units of one slot
  for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<long>(gridDim.x) * blockDim.x) {
    const int u = static_cast<int>(i % units);
    long q = i / units;
    const bool isv = q & 1;
    q >>= 1;                                   // output row b * n + t
    const int t = static_cast<int>(q % n);
    const long b = q / n;
    const int slot = first + t, c = u * 16, j = c / d_h;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(
        (isv ? V8 : K8) + (static_cast<size_t>(b) * S + slot) * H_kv * d_h + c));
    const float s = __ldg((isv ? V_scale : K_scale) +
                          (static_cast<size_t>(b) * nb + slot / kC8Block) * H_kv + j);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2 f = c8_float2(w[k >> 1] >> ((k & 1) * 16));
      f.x *= s;
      f.y *= s;
      // beyond fp16's largest (only 65504 itself rounds there): 65504; NaN passes
      f.x = f.x > 65504.f ? 65504.f : (f.x < -65504.f ? -65504.f : f.x);
      f.y = f.y > 65504.f ? 65504.f : (f.y < -65504.f ? -65504.f : f.y);
      o[k] = pack_half2(f.x, f.y);
    }
    uint4* d = reinterpret_cast<uint4*>((isv ? V_rows : K_rows) + q * ld + c);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------- evict
// Order of the candidates as unsigned keys: 0 for a slot without a token,
// ~0 for one of the last `recent` slots, in between the weight (NaN below
// every number, -0 as 0).
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int s, int first_recent) {
  if (pos < 0) return 0u;
  if (s >= first_recent) return 0xFFFFFFFFu;
  if (w != w) return 1u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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
constexpr int kSelSlots = 8192;      // slots per CTA worth one more CTA in the cluster
constexpr int kSelMaxCluster = 8;

// One cluster per batch row: the keep-th largest key by four rounds of 8-bit
// digit counts (each CTA counts its run of slots, the counts are summed over
// the cluster through distributed shared memory), then the slots above it,
// and the first of those equal to it, are written out in slot order.  The
// keys are read from L2 once per round: 8 bytes per slot.
__global__ void __launch_bounds__(kSelThreads) cache8_select_kernel(const SelectParams p) {
  pdl_enter();
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), C = cluster.num_blocks();
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int hist[2][256];
  __shared__ int sum[256];
  __shared__ int wsum[32];
  __shared__ int counts[2];
  __shared__ int found[2];           // digit, keys above it
  const float* w = p.w + static_cast<size_t>(b) * p.S;
  const int32_t* pos = p.pos + static_cast<size_t>(b) * p.S;
  int run = (p.end + C - 1) / C;
  run = (run + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int lo = min(static_cast<long long>(p.end), static_cast<long long>(rank) * run);
  const int hi = static_cast<int>(min(static_cast<long long>(p.end), static_cast<long long>(lo) + run));

  uint32_t prefix = 0;
  int want = p.keep;                 // rank still to find among keys that match the prefix
  bool all = false;                  // fewer tokens than places: keep every one
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    int* h = hist[round & 1];
    if (tid < 256) h[tid] = 0;
    __syncthreads();
    for (int base = lo; base < hi; base += kSelThreads) {
      const int s = base + tid;
      uint32_t key = 0;
      if (s < hi) key = evict_key(__ldg(w + s), __ldg(pos + s), s, p.first_recent);
      const bool in = key != 0 && (round == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)));
      const int digit = in ? static_cast<int>((key >> shift) & 255u) : 256;
      // keys share digits (weights of one magnitude): one add per digit and warp
      const unsigned same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&h[digit], __popc(same));
    }
    cluster.sync();
    if (tid < 256) {
      int n = 0;
      for (int r = 0; r < C; ++r) n += cluster.map_shared_rank(h, r)[tid];
      sum[tid] = n;
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8l .. 248 - 8l, largest first
      int mine = 0;
      for (int i = 0; i < 8; ++i) mine += sum[255 - 8 * lane - i];
      int before = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const int total = __shfl_sync(0xffffffffu, before, 31);
      before -= mine;
      if (lane == 0) found[0] = -1;
      __syncwarp();
      if (total >= want && before < want && before + mine >= want) {
        int above = before;
        for (int i = 0; i < 8; ++i) {
          const int d = 255 - 8 * lane - i;
          if (above + sum[d] >= want) {
            found[0] = d;
            found[1] = above;
            break;
          }
          above += sum[d];
        }
      }
    }
    __syncthreads();
    if (found[0] < 0) {              // (only in round 0)
      all = true;
      break;
    }
    prefix |= static_cast<uint32_t>(found[0]) << shift;
    want -= found[1];
  }
  // A slot stays if its key is above `prefix`, or equals it and is among the
  // first `want` that do.
  const uint32_t thr = all ? 0u : prefix;
  if (all) want = 0;
  int gt = 0, eq = 0;
  for (int base = lo; base < hi; base += kSelThreads) {
    const int s = base + tid;
    if (s < hi) {
      const uint32_t key = evict_key(__ldg(w + s), __ldg(pos + s), s, p.first_recent);
      gt += key > thr;
      eq += key == thr;
    }
  }
  if (tid < 2) counts[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    atomicAdd(&counts[0], gt);
    atomicAdd(&counts[1], eq);
  }
  cluster.sync();
  int gt0 = 0, eq0 = 0, n_kept = 0, n_eq = 0;
  for (int r = 0; r < C; ++r) {
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
  for (int base = lo; base < hi; base += kSelThreads) {
    const int s = base + tid;
    float ws = 0.f;
    int ps = -1;
    uint32_t key = 0;
    if (s < hi) {
      ws = __ldg(w + s);
      ps = __ldg(pos + s);
      key = evict_key(ws, ps, s, p.first_recent);
    }
    const bool g = s < hi && key > thr, e = s < hi && key == thr;
    const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    // counts of (above, equal) in 16 bits each: at most 1024 per step
    if (lane == 0) wsum[warp] = __popc(bg) | (__popc(be) << 16);
    __syncthreads();
    int v = wsum[lane];
    const int own = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += up;
    }
    const int total = __shfl_sync(0xffffffffu, v, 31);
    const int here = __shfl_sync(0xffffffffu, v - own, warp);
    const unsigned below = (1u << lane) - 1u;
    const int ng = gt0 + (here & 0xFFFF) + __popc(bg & below);
    const int ne = eq0 + (here >> 16) + __popc(be & below);
    if (g || (e && ne < want)) {
      const int d = ng + min(ne, want);
      kept[d] = s;
      pos_dst[d] = ps;
      w_dst[d] = ws;
    }
    gt0 += total & 0xFFFF;
    eq0 += total >> 16;
    __syncthreads();
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

// One CTA per (block of 64 kept slots, kv head, K' or V, batch row), heads
// fastest so that the CTAs at work at one time read whole slots.  The numbers
// of the block stay in registers between the search for the largest value and
// the move to the block's own scale.
template <int DH>
__global__ void __launch_bounds__(kRowThreads) cache8_move_kernel(const MoveParams p) {
  pdl_enter();
  constexpr int TPR = DH / 16;                 // threads per row, 16 channels each
  constexpr int RPP = kRowThreads / TPR;
  constexpr int NP = kTile / RPP;
  __shared__ float red[kRowThreads / 32];
  const int tid = threadIdx.x;
  unsigned idx = blockIdx.x;
  const int hk = idx % (2 * p.H_kv);
  idx /= 2 * p.H_kv;
  const int blk = idx % p.nblk, b = idx / p.nblk;
  const int j = hk >> 1;
  const bool isv = hk & 1;
  const int c = (tid % TPR) * 16;
  const size_t ldc = static_cast<size_t>(p.H_kv) * DH;
  const uint8_t* src = (isv ? p.V8 : p.K8) + static_cast<size_t>(b) * p.S * ldc +
                       static_cast<size_t>(j) * DH + c;
  const float* src_scale =
      (isv ? p.V_scale : p.K_scale) + static_cast<size_t>(b) * p.nb * p.H_kv + j;

  uint4 n[NP];
  float sc[NP], mx = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int d = blk * kTile + i * RPP + tid / TPR;
    const int s = d < p.keep ? __ldg(p.kept + static_cast<size_t>(b) * p.keep + d) : -1;
    n[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.f;
    if (s >= 0) {
      n[i] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<size_t>(s) * ldc));
      sc[i] = __ldg(src_scale + static_cast<size_t>(s / kC8Block) * p.H_kv);
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    // e4m3 magnitudes order like their codes; 0x7f is NaN
    const uint32_t w[4] = {n[i].x, n[i].y, n[i].z, n[i].w};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a = w[k] & 0x7F7F7F7Fu;
      a &= ~__vcmpeq4(a, 0x7F7F7F7Fu);
      m = __vmaxu4(m, a);
    }
    m = __vmaxu4(m, m >> 16);
    m = max(m & 0xFFu, (m >> 8) & 0xFFu);
    mx = fmaxf(mx, c8_float2(m).x * sc[i]);
  }
  mx = block_max(mx, red);
  const float s = c8_scale_for(mx);
  const float inv = 1.f / s;
  uint8_t* dst = (isv ? p.V8_dst : p.K8_dst) + static_cast<size_t>(b) * p.S_dst * ldc +
                 static_cast<size_t>(j) * DH + c;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int d = blk * kTile + i * RPP + tid / TPR;
    if (d < p.keep) {
      const float ratio = sc[i] * inv;
      uint4 v = n[i];
      if (ratio != 1.f)
        v = make_uint4(c8_rescale4(v.x, ratio), c8_rescale4(v.y, ratio), c8_rescale4(v.z, ratio),
                       c8_rescale4(v.w, ratio));
      *reinterpret_cast<uint4*>(dst + static_cast<size_t>(d) * ldc) = v;
    }
  }
  if (tid == 0)
    (isv ? p.V_scale_dst : p.K_scale_dst)[(static_cast<size_t>(b) * p.nb_dst + blk) * p.H_kv + j] = s;
}

}  // namespace

cudaError_t launch_cache8_write(const void* K_rows, const void* V_rows, long ld,
                                const int32_t* segment_pos, const int32_t* pad_lens, int B, int T,
                                int S, int end, int H_kv, int d_h, void* K8, void* V8,
                                float* K_scale, float* V_scale, int32_t* pos_cache,
                                cudaStream_t stream) {
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
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(B) * p.nblk * H_kv * 2));
  return launch_pdl(d_h == 256 ? cache8_write_kernel<256> : cache8_write_kernel<128>, grid,
                    dim3(kRowThreads), 0, stream, p);
}

cudaError_t launch_cache8_read(const void* K8, const void* V8, const float* K_scale,
                               const float* V_scale, int B, int S, int first, int n, int H_kv,
                               int d_h, void* K_rows, void* V_rows, long ld, cudaStream_t stream) {
  const long total = static_cast<long>(B) * n * 2 * (H_kv * d_h / 16);
  if (total <= 0) return cudaSuccess;
  const long ctas = std::min<long>((total + 255) / 256, 64L * num_sms());
  return launch_pdl(cache8_read_kernel, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, stream,
                    static_cast<const uint8_t*>(K8), static_cast<const uint8_t*>(V8), K_scale,
                    V_scale, total, S, c8_blocks(S), first, n, H_kv, d_h,
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
  cudaError_t e = launch_pdl_cluster(cache8_select_kernel, dim3(cl, B), dim3(kSelThreads), 0, cl,
                                     stream, q);
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
  const dim3 grid(static_cast<unsigned>(static_cast<long long>(B) * p.nblk * H_kv * 2));
  return launch_pdl(d_h == 256 ? cache8_move_kernel<256> : cache8_move_kernel<128>, grid,
                    dim3(kRowThreads), 0, stream, p);
}

}  // namespace g3
