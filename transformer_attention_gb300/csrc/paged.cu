// The paged KV cache's kernels beside its attention (paged_attn.cu): the
// positions of a batch's new tokens, the append, the commit (paged.cuh).
//
// append: x <- x / sqrt(mean(x^2) + 1e-6) * (1 + gamma), then RoPE at lens[b] +
//   depth (rope.cuh), Q also times the query scale; K' and V rows go straight
//   to their page slots.  Every number is read and written once: HBM bounds it
//   for prompts, latency for a step.  A CTA takes a few rows, finds their
//   sequences, positions and slots together, and its warps take up to 8 steps
//   of a row's head vectors (Q, K and V), d_h / 8 lanes per vector and 16 bytes
//   per lane, all loads first.
// commit: token accepted[b, i] moves to slot lens[b] + i.  accepted ascends, so
//   accepted[b, i] >= i, and a column of the rows is moved by one thread from
//   the first token to the last: a slot is written only after the token that
//   lay there was read.
#include <algorithm>

#include "paged.cuh"
#include "rope.cuh"

namespace g3 {

namespace {

constexpr float kEps = 1e-6f;
constexpr int kVecUnroll = 8;        // steps of head vectors per item
constexpr int kAppendRows = 32;      // rows of a CTA at a time
constexpr int kAppendWarps = 8;
constexpr int kStartsMax = 1024;     // row_start entries kept in shared memory

// Token row m's sequence and position (whole warp); seq -1 behind the last one.
struct PagedToken {
  int seq, i, len, depth;
};

__device__ __forceinline__ PagedToken paged_token(const PagedBatch& p, int m, int lane, int* status) {
  PagedToken t;
  t.seq = paged_find(p, m, lane);
  if (t.seq < 0) return t;
  const PagedSeq s = paged_seq(p, t.seq, status);
  t.i = m - s.row0;
  t.len = s.len;
  if (t.i < 0 || t.i >= s.n) {   // a sequence that does not fit
    t.seq = -1;
    return t;
  }
  t.depth = t.i;
  if (p.parents != nullptr) t.depth = __popcll(paged_ancestors(p, s, lane, status).of(t.i)) - 1;
  return t;
}

__global__ void __launch_bounds__(128)
    paged_positions_kernel(const PagedBatch p, int32_t* __restrict__ pos, int* status) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int m = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (m >= p.M) return;
  const PagedToken t = paged_token(p, m, lane, status);
  if (lane == 0) pos[m] = t.seq >= 0 ? t.len + t.depth : 0;
}

struct AppendParams {
  const __half* Q;
  __half* Qo;
  const __half* K;
  const __half* V;
  const __nv_bfloat16* gq;
  const __nv_bfloat16* gk;
  __half* Kp;
  __half* Vp;
  long ldq, ldqo, ldkv;
  int H, H_kv, chunk_u, rows, zero_behind, lost;   // rows: of a CTA at a time
  float query_scale;
  int* status;
};

// NORM: norm and rotation; else the rows go to the pages as they are.
template <int DH, bool NORM>
__global__ void __launch_bounds__(32 * kAppendWarps, 2)
    paged_append_kernel(const PagedBatch p, const AppendParams a, const __grid_constant__ RopeFreqs freqs) {
  pdl_enter();
  constexpr int LPV = DH / 8;      // lanes per head vector
  constexpr int VPW = 32 / LPV;    // head vectors per warp step
  constexpr int HALF = LPV / 2;    // lane distance of the RoPE partner
  __shared__ int starts[kStartsMax + 1];
  __shared__ int dst_sh[kAppendRows];      // pool row, -1: no page, -2: of no sequence
  __shared__ float pos_sh[kAppendRows];
  const bool lost = lost_work(a.status, a.lost);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / LPV, ll = lane % LPV;
  const bool second_half = ll >= HALF;
  const int c0 = (ll % HALF) * 8;
  uint4 gq_raw = make_uint4(0, 0, 0, 0), gk_raw = gq_raw;
  if constexpr (NORM) {
    gq_raw = *reinterpret_cast<const uint4*>(a.gq + ll * 8);
    gk_raw = *reinterpret_cast<const uint4*>(a.gk + ll * 8);
  }
  const bool in_smem = p.B <= kStartsMax;
  if (in_smem)
    for (int i = tid; i <= p.B; i += blockDim.x) starts[i] = __ldcg(p.row_start + i);
  const int h0 = NORM ? 0 : a.H;                   // Q is finished without gammas
  const int hk = a.H + a.H_kv, end = hk + a.H_kv;  // head vectors: Q, K, V
  const int vpc = VPW * a.chunk_u;
  const int nch = (end - h0 + vpc - 1) / vpc;      // items of a row
  const int KVD = a.H_kv * DH;

  // This lane's 16 bytes of the item's vectors.
  uint4 raw[kVecUnroll];
  auto load = [&](int m0, int item) {
    const int m = m0 + item / nch, first = h0 + item % nch * vpc + sub;
#pragma unroll
    for (int u = 0; u < kVecUnroll; ++u) {
      const int hv = first + u * VPW;
      const __half* src = hv < a.H ? a.Q + m * a.ldq + hv * DH
                                   : (hv < hk ? a.K + m * a.ldkv + (hv - a.H) * DH
                                              : a.V + m * a.ldkv + (hv - hk) * DH);
      raw[u] = (u < a.chunk_u && hv < end) ? __ldcg(reinterpret_cast<const uint4*>(src + ll * 8))
                                           : make_uint4(0, 0, 0, 0);
    }
  };

  for (int m0 = blockIdx.x * a.rows; m0 < p.M; m0 += gridDim.x * a.rows) {
    const int rows = min(a.rows, p.M - m0), items = rows * nch;
    int item = warp;
    if (item < items) load(m0, item);
    // ---------------- the rows' slots and positions
    __syncthreads();       // (starts are there; the rows before are done)
    if (tid < rows) {
      const int m = m0 + tid;
      auto start = [&](int i) { return in_smem ? starts[i] : __ldcg(p.row_start + i); };
      // the first sequence that ends behind m
      int b = 0, e = p.B;
      while (b < e) {
        const int mid = (b + e) / 2;
        if (start(mid + 1) <= m) b = mid + 1;
        else e = mid;
      }
      int dst = -2, pos = 0;
      if (b < p.B) {
        const PagedSeq s = paged_seq(p, b, a.status);
        const int i = m - s.row0;
        if (i >= 0 && i < s.n) {   // (a sequence that does not fit has none)
          dst = paged_row(p, b, s.len + i, a.status);
          pos = s.len + i;
        }
      }
      dst_sh[tid] = dst;
      pos_sh[tid] = static_cast<float>(pos);
    }
    if (p.parents != nullptr) {    // a tree: positions by depth, a warp per row
      __syncthreads();             // (behind the positions without one)
      for (int r = warp; r < rows; r += kAppendWarps) {
        const PagedToken t = paged_token(p, m0 + r, lane, a.status);
        if (lane == 0 && t.seq >= 0) pos_sh[r] = static_cast<float>(t.len + t.depth);
      }
    }
    if (__syncthreads_or(lost)) return;

    while (item < items) {
      const int r = item / nch, m = m0 + r;
      const int base = h0 + item % nch * vpc, first = base + sub;
      const int dst = dst_sh[r];
      if (dst == -2) {
        if (a.zero_behind && item % nch == 0)   // (the row's first item; the others write nothing)
          for (int v = lane; v < a.H * LPV; v += 32)
            *reinterpret_cast<uint4*>(a.Qo + m * a.ldqo + v * 8) = make_uint4(0, 0, 0, 0);
      } else {
        float cs[8], sn[8];
        if (NORM && base < hk) {
          const float pos = pos_sh[r];
#pragma unroll
          for (int e = 0; e < 8; ++e) rope_sincos(pos, freqs.f[c0 + e], sn[e], cs[e]);
        }
#pragma unroll
        for (int u = 0; u < kVecUnroll; ++u) {
          if (u >= a.chunk_u || base + u * VPW >= end) break;   // warp-uniform
          const int hv = first + u * VPW;
          const bool is_q = hv < a.H;
          uint4 w = raw[u];
          if (NORM && base + u * VPW < hk) {
            float x[8];
            const __half2* h2 = reinterpret_cast<const __half2*>(&raw[u]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = __half22float2(h2[e]);
              x[2 * e] = f.x;
              x[2 * e + 1] = f.y;
            }
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int off = HALF; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float rs = rsqrtf(ss * (1.f / DH) + kEps);
            const uint4 graw = is_q ? gq_raw : gk_raw;
            const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&graw);
            float y[8], o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 gf = __bfloat1622float2(g2[e]);
              y[2 * e] = x[2 * e] * rs * (1.f + gf.x);
              y[2 * e + 1] = x[2 * e + 1] * rs * (1.f + gf.y);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __shfl_xor_sync(0xffffffffu, y[e], HALF);
            const float sc = is_q ? a.query_scale : 1.f;
            uint32_t rot[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // first half: (x1 cos - x2 sin), second: (x2 cos + x1 sin)
              const float s0 = second_half ? sn[2 * e] : -sn[2 * e];
              const float s1 = second_half ? sn[2 * e + 1] : -sn[2 * e + 1];
              const float r0 = y[2 * e] * cs[2 * e] + o[2 * e] * s0;
              const float r1 = y[2 * e + 1] * cs[2 * e + 1] + o[2 * e + 1] * s1;
              rot[e] = pack_half2(r0 * sc, r1 * sc);
            }
            if (hv < hk) w = make_uint4(rot[0], rot[1], rot[2], rot[3]);
          }
          if (hv >= end) continue;
          __half* to = is_q ? a.Qo + m * a.ldqo + hv * DH
                            : (hv < hk ? a.Kp + static_cast<size_t>(dst) * KVD + (hv - a.H) * DH
                                       : a.Vp + static_cast<size_t>(dst) * KVD + (hv - hk) * DH);
          if (is_q || dst >= 0) *reinterpret_cast<uint4*>(to + ll * 8) = w;
        }
      }
      item += kAppendWarps;
      if (item < items) load(m0, item);
    }
  }
}

// ---------------------------------------------------------------- commit
constexpr int kCommitThreads = 256;
constexpr int kCommitAhead = 8;      // rows in flight per thread
constexpr int kCommitChunk = 256;    // accepted tokens per round of shared memory

// CTA (columns of 16 bytes, sequence, layer and K or V).
__global__ void __launch_bounds__(kCommitThreads)
    paged_commit_kernel(const PagedBatch p, const int32_t* __restrict__ accepted,
                        const int32_t* __restrict__ counts, int vecs, __half* Kp, __half* Vp,
                        int32_t* __restrict__ new_lens, int* status) {
  pdl_enter();
  const int b = blockIdx.y, tid = threadIdx.x;
  const PagedSeq s = paged_seq(p, b, status);
  const int count = counts != nullptr ? __ldcg(counts + b) : s.n;
  const int32_t* path = accepted != nullptr ? accepted + static_cast<size_t>(b) * p.T_max : nullptr;
  bool bad = count < 0 || count > s.n;
  if (!bad && path != nullptr)
    for (int i = tid; i < count; i += kCommitThreads) {
      const int at = __ldcg(path + i);
      bad |= at >= s.n || at < (i > 0 ? __ldcg(path + i - 1) + 1 : 0);
    }
  bad = __syncthreads_or(bad);
  const bool head = blockIdx.x == 0 && blockIdx.z == 0;
  if (bad) {
    if (head && tid == 0) {
      record_error(status, kDevErrBadPaged);
      new_lens[b] = s.len;
    }
    return;
  }
  if (head && tid == 0) new_lens[b] = s.len + count;
  if (path == nullptr) return;
  const size_t pool = (static_cast<size_t>(p.n_pages) << p.page_shift) * vecs;   // 16-byte vectors
  const int layer = blockIdx.z >> 1;
  uint4* base = reinterpret_cast<uint4*>(blockIdx.z & 1 ? Vp : Kp) + layer * pool;
  const int c = blockIdx.x * kCommitThreads + tid;
  __shared__ int src[kCommitChunk], dst[kCommitChunk];
  for (int i0 = 0; i0 < count; i0 += kCommitChunk) {
    const int n = min(kCommitChunk, count - i0);
    __syncthreads();
    for (int i = tid; i < n; i += kCommitThreads) {
      const int at = __ldcg(path + i0 + i);
      // a token that lies where it belongs is not moved
      src[i] = at == i0 + i ? -1 : paged_row(p, b, s.len + at, status);
      dst[i] = at == i0 + i ? -1 : paged_row(p, b, s.len + i0 + i, status);
    }
    __syncthreads();
    if (c >= vecs) continue;
    for (int i = 0; i < n; i += kCommitAhead) {
      uint4 v[kCommitAhead];
#pragma unroll
      for (int u = 0; u < kCommitAhead; ++u)
        if (i + u < n && src[i + u] >= 0) v[u] = __ldcg(base + static_cast<size_t>(src[i + u]) * vecs + c);
#pragma unroll
      for (int u = 0; u < kCommitAhead; ++u)
        if (i + u < n && src[i + u] >= 0 && dst[i + u] >= 0)
          base[static_cast<size_t>(dst[i + u]) * vecs + c] = v[u];
    }
  }
}

template <int DH>
cudaError_t launch_append_dh(const PagedBatch& batch, const AppendParams& p, bool norm,
                             const RopeFreqs& f, cudaStream_t stream) {
  AppendParams a = p;
  constexpr int vpw = 32 / (DH / 8);
  const int steps = ((norm ? a.H : 0) + 2 * a.H_kv + vpw - 1) / vpw;   // of a row
  // Few rows: one per CTA, its steps spread over the warps; many: as many as
  // share out the rows over two CTAs per SM.
  const int slots = 2 * num_sms();
  const int rounds = (batch.M + slots * kAppendRows - 1) / (slots * kAppendRows);
  a.rows = (batch.M + slots * rounds - 1) / (slots * rounds);
  a.chunk_u = std::min(kVecUnroll, std::max(1, steps * a.rows / kAppendWarps));
  const int blocks = (batch.M + a.rows - 1) / a.rows;
  const dim3 grid(std::min(blocks, slots)), block(32 * kAppendWarps);
  return norm ? launch_pdl(paged_append_kernel<DH, true>, grid, block, 0, stream, batch, a, f)
              : launch_pdl(paged_append_kernel<DH, false>, grid, block, 0, stream, batch, a, f);
}

// The frequencies of the thread's last call (128 powers in double take 6 us of
// host time, more than a step's kernel).
const RopeFreqs& rope_freqs(int d_h, double base, double scale) {
  thread_local RopeFreqs f;
  thread_local int at_d = 0;
  thread_local double at_base = 0, at_scale = 0;
  if (at_d != d_h || at_base != base || at_scale != scale) {
    f = make_rope_freqs(d_h, base, scale);
    at_d = d_h;
    at_base = base;
    at_scale = scale;
  }
  return f;
}

}  // namespace

cudaError_t launch_paged_positions(const PagedBatch& batch, int32_t* pos, cudaStream_t stream,
                                   int* status) {
  return launch_pdl(paged_positions_kernel, dim3((batch.M + 3) / 4), dim3(128), 0, stream, batch, pos,
                    status);
}

cudaError_t launch_paged_append(const PagedBatch& batch, const void* Q, long ldq, void* Q_out,
                                long ldqo, const void* K, const void* V, long ldkv,
                                const void* gamma_q, const void* gamma_k, int H, int H_kv, int d_h,
                                double rope_base, double rope_scale, float query_scale,
                                void* K_pages, void* V_pages, bool zero_behind,
                                cudaStream_t stream, int* status, int lost) {
  AppendParams a;
  a.Q = static_cast<const __half*>(Q);
  a.Qo = static_cast<__half*>(Q_out);
  a.K = static_cast<const __half*>(K);
  a.V = static_cast<const __half*>(V);
  a.gq = static_cast<const __nv_bfloat16*>(gamma_q);
  a.gk = static_cast<const __nv_bfloat16*>(gamma_k);
  a.Kp = static_cast<__half*>(K_pages);
  a.Vp = static_cast<__half*>(V_pages);
  a.ldq = ldq;
  a.ldqo = ldqo;
  a.ldkv = ldkv;
  a.H = H;
  a.H_kv = H_kv;
  a.zero_behind = zero_behind;
  a.lost = lost;
  a.query_scale = query_scale;
  a.status = status;
  const bool norm = gamma_k != nullptr;
  static const RopeFreqs none{};
  const RopeFreqs& f = norm ? rope_freqs(d_h, rope_base, rope_scale) : none;
  return d_h == 256 ? launch_append_dh<256>(batch, a, norm, f, stream)
                    : launch_append_dh<128>(batch, a, norm, f, stream);
}

cudaError_t launch_paged_commit(const PagedBatch& batch, const int32_t* accepted,
                                const int32_t* counts, int layers, int H_kv, int d_h,
                                void* K_pages, void* V_pages, int32_t* new_lens,
                                cudaStream_t stream, int* status) {
  const int vecs = H_kv * d_h / 8;
  const dim3 grid((vecs + kCommitThreads - 1) / kCommitThreads, batch.B, accepted != nullptr ? 2 * layers : 1);
  return launch_pdl(paged_commit_kernel, grid, dim3(kCommitThreads), 0, stream, batch, accepted, counts,
                    vecs, static_cast<__half*>(K_pages), static_cast<__half*>(V_pages), new_lens, status);
}

}  // namespace g3
