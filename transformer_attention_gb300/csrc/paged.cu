// The paged KV cache's kernels beside its attention (paged_attn.cu): the
// positions of a batch's new tokens, the append, the commit (paged.cuh).
//
// append: x <- x / sqrt(mean(x^2) + 1e-6) * (1 + gamma), then RoPE at lens[b] +
//   depth (rope.cuh), Q also times the query scale; K' and V rows go straight
//   to their page slots.  Every number is read and written once: HBM bounds it
//   for prompts, latency for a step.  A warp takes (row, up to 8 steps of head
//   vectors), d_h / 8 lanes per vector and 16 bytes per lane, all loads first.
// commit: token accepted[b, i] moves to slot lens[b] + i.  accepted ascends, so
//   accepted[b, i] >= i, and a column of the rows is moved by one thread from
//   the first token to the last: a slot is written only after the token that
//   lay there was read.
#include "paged.cuh"
#include "rope.cuh"

namespace g3 {

namespace {

constexpr float kEps = 1e-6f;
constexpr int kVecUnroll = 8;    // steps of head vectors per item

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
  int H, H_kv, chunk_u, zero_behind, lost;
  float query_scale;
  int* status;
};

// NORM: norm and rotation; else the rows go to the pages as they are.
template <int DH, bool NORM>
__global__ void __launch_bounds__(256, 2)
    paged_append_kernel(const PagedBatch p, const AppendParams a, const __grid_constant__ RopeFreqs freqs) {
  pdl_enter();
  if (lost_work(a.status, a.lost)) return;
  constexpr int LPV = DH / 8;      // lanes per head vector
  constexpr int VPW = 32 / LPV;    // head vectors per warp step
  constexpr int HALF = LPV / 2;    // lane distance of the RoPE partner
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPV, ll = lane % LPV;
  const bool second_half = ll >= HALF;
  const int c0 = (ll % HALF) * 8;
  uint4 gq_raw = make_uint4(0, 0, 0, 0), gk_raw = gq_raw;
  if constexpr (NORM) {
    gq_raw = *reinterpret_cast<const uint4*>(a.gq + ll * 8);
    gk_raw = *reinterpret_cast<const uint4*>(a.gk + ll * 8);
  }
  const int warps_total = gridDim.x * (blockDim.x >> 5);
  const int h0 = NORM ? 0 : a.H;                   // Q is finished without gammas
  const int nvec = a.H - h0 + a.H_kv;
  const int vpc = VPW * a.chunk_u;
  const int nch = (nvec + vpc - 1) / vpc;
  const long items = static_cast<long>(p.M) * nch;
  const int KVD = a.H_kv * DH;
  for (long item = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); item < items;
       item += warps_total) {
    const int m = static_cast<int>(item / nch);
    const int base = h0 + static_cast<int>(item % nch) * vpc;
    const int first = base + sub;
    uint4 raw[kVecUnroll];
#pragma unroll
    for (int u = 0; u < kVecUnroll; ++u) {
      const int hv = first + u * VPW;
      const __half* src = hv < a.H ? a.Q + m * a.ldq + hv * DH : a.K + m * a.ldkv + (hv - a.H) * DH;
      raw[u] = (u < a.chunk_u && hv < h0 + nvec) ? __ldcg(reinterpret_cast<const uint4*>(src + ll * 8))
                                                 : make_uint4(0, 0, 0, 0);
    }
    const PagedToken t = paged_token(p, m, lane, a.status);
    if (t.seq < 0) {
      if (a.zero_behind && item % nch == 0)   // (its first item; the others write nothing)
        for (int v = lane; v < a.H * LPV; v += 32)
          *reinterpret_cast<uint4*>(a.Qo + m * a.ldqo + v * 8) = make_uint4(0, 0, 0, 0);
      continue;
    }
    const int row = paged_row(p, t.seq, t.len + t.i, a.status);
    float cs[8], sn[8];
    if constexpr (NORM) {
      const float pos = static_cast<float>(t.len + t.depth);
#pragma unroll
      for (int e = 0; e < 8; ++e) rope_sincos(pos, freqs.f[c0 + e], sn[e], cs[e]);
    }
#pragma unroll
    for (int u = 0; u < kVecUnroll; ++u) {
      if (u >= a.chunk_u || base + u * VPW >= h0 + nvec) break;   // warp-uniform
      const int hv = first + u * VPW;
      const bool is_q = hv < a.H;
      uint4 w = raw[u];
      if constexpr (NORM) {
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
        uint32_t* wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // first half: (x1 cos - x2 sin), second: (x2 cos + x1 sin)
          const float s0 = second_half ? sn[2 * e] : -sn[2 * e];
          const float s1 = second_half ? sn[2 * e + 1] : -sn[2 * e + 1];
          const float r0 = y[2 * e] * cs[2 * e] + o[2 * e] * s0;
          const float r1 = y[2 * e + 1] * cs[2 * e + 1] + o[2 * e + 1] * s1;
          wp[e] = pack_half2(r0 * sc, r1 * sc);
        }
      }
      if (hv >= h0 + nvec) continue;
      if (is_q) {
        *reinterpret_cast<uint4*>(a.Qo + m * a.ldqo + hv * DH + ll * 8) = w;
      } else if (row >= 0) {
        const int off = (hv - a.H) * DH + ll * 8;
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(a.V + m * a.ldkv + off));
        *reinterpret_cast<uint4*>(a.Kp + static_cast<size_t>(row) * KVD + off) = w;
        *reinterpret_cast<uint4*>(a.Vp + static_cast<size_t>(row) * KVD + off) = v;
      }
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
  const int vpw = 32 / (DH / 8);
  const long nvec = (norm ? a.H : 0) + a.H_kv;
  // Few rows: a step of head vectors per warp, so that they spread over the
  // SMs; many: kVecUnroll, which share a row's angles.
  const long steps = batch.M * ((nvec + vpw - 1) / vpw);
  a.chunk_u = steps <= 16L * num_sms() ? 1 : kVecUnroll;
  const long items = batch.M * ((nvec + vpw * a.chunk_u - 1) / (vpw * a.chunk_u));
  const long blocks = (items + 7) / 8, most = 8L * num_sms();
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  return norm ? launch_pdl(paged_append_kernel<DH, true>, grid, dim3(256), 0, stream, batch, a, f)
              : launch_pdl(paged_append_kernel<DH, false>, grid, dim3(256), 0, stream, batch, a, f);
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
  RopeFreqs f{};
  if (norm) f = make_rope_freqs(d_h, rope_base, rope_scale);
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
