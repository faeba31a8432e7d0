// The paged KV cache's kernels beside its attention (paged_attn.cu): the
// positions of a batch's new tokens, the append, the commit (paged.cuh).
//
// append: x <- x / sqrt(mean(x^2) + 1e-6) * (1 + gamma), then RoPE at lens[b] +
//   depth (rope.cuh), Q also times the query scale; K' and V rows go straight
//   to their page slots.  Every number is read and written once: HBM bounds it
//   for prompts, latency for a step.  A CTA takes a few rows, finds their
//   sequences, positions and slots together, and its warps take up to 8 steps
//   of a row's head vectors (Q, K and V), all loads first; d_h / 8 lanes per
//   vector, each with four channels of both halves, whose pairs it rotates alone.
//   Measured: 17186 tokens of 64 heads of 128 channels 88.6 us (86% of the copy
//   rate); 16 trees of 5 to 12 tokens, 32 heads of 256, 6.4 us: the row's sequence,
//   its start and length, its page, then by a warp per row its sequence, start
//   and length again and its parents, one round trip each.  Finished rows, which go
//   to the pages as they are: 17186 of 16 + 16 heads of 128 48.4 us (86%), 4096 13.5
//   (73%), 130 of 8 + 8 heads of 256 3.3.
// commit: token accepted[b, i] moves to slot lens[b] + i.  accepted ascends, so
//   accepted[b, i] >= i, and a column of the rows is moved by one thread from
//   the first token to the last: a slot is written only after the token that
//   lay there was read.  Measured: 64 paths of 17 to 64 tokens in six layers, 90
//   MB, 20.8 us: 768 CTAs in two and a half rounds, each the path's rows, eight at
//   a time, behind 3 us of look-ups of its own.
#include <algorithm>

#include "paged.cuh"
#include "rope.cuh"

namespace g3 {

namespace {

constexpr float kEps = 1e-6f;
constexpr int kVecUnroll = 8;        // steps of head vectors per item at most
constexpr int kAppendRows = 64;      // rows of a CTA at a time
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

// Rows find their sequence by the first rows alone: the sequences that no row
// led to are checked here, by one CTA.
__device__ __forceinline__ void check_sequences(const PagedBatch& p, int* status) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) paged_seq(p, b, status);
}

// The first sequence that ends behind row m, B: none (one thread; start(i): row_start[i]).
template <class F>
__device__ __forceinline__ int sequence_of(const F& start, int B, int m) {
  int b = 0, e = B;
  while (b < e) {
    const int mid = (b + e) / 2;
    if (start(mid + 1) <= m) b = mid + 1;
    else e = mid;
  }
  return b;
}

// A thread per row, with trees a warp (4096 rows of a chain: 1.6 us, 4.3 by warps).
constexpr int kPositionThreads = 128;
__global__ void __launch_bounds__(kPositionThreads)
    paged_positions_kernel(const PagedBatch p, int32_t* __restrict__ pos, int* status) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  if (p.parents == nullptr) {
    const int m = blockIdx.x * kPositionThreads + threadIdx.x;
    if (m < p.M) {
      const int b = sequence_of([&](int i) { return __ldcg(p.row_start + i); }, p.B, m);
      int at = 0;
      if (b < p.B) {
        const PagedSeq s = paged_seq(p, b, status);
        const int i = m - s.row0;
        if (i >= 0 && i < s.n) at = s.len + i;   // (a sequence that does not fit has none)
      }
      pos[m] = at;
    }
  } else {
    const int m = blockIdx.x * (kPositionThreads / 32) + (threadIdx.x >> 5);
    if (m < p.M) {
      const PagedToken t = paged_token(p, m, lane, status);
      if (lane == 0) pos[m] = t.seq >= 0 ? t.len + t.depth : 0;
    }
  }
  check_sequences(p, status);
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

// NORM: norm and rotation; else the rows go to the pages as they are.  PACKED: a
// row's steps are one item, else an item has steps of Q, of K or of V alone.  Few
// heads leave most of such an item empty: 35000 rows of 4 + 1 + 1 heads of 256
// take 113 us apart and 67 packed, 17186 of 8 + 4 + 4 of 128 45 and 30.  Packed
// items of a part of a row take 6 to 20% more than those of one kind.
template <int DH, bool NORM, bool PACKED>
__global__ void __launch_bounds__(32 * kAppendWarps, 2)
    paged_append_kernel(const PagedBatch p, const AppendParams a, const __grid_constant__ RopeFreqs freqs) {
  pdl_enter();
  constexpr int LPV = DH / 8;      // lanes per head vector
  constexpr int VPW = 32 / LPV;    // head vectors per warp step
  __shared__ int starts[kStartsMax + 1];
  __shared__ int dst_sh[kAppendRows];      // pool row, -1: no page, -2: of no sequence
  __shared__ float pos_sh[kAppendRows];
  const bool lost = lost_work(a.status, a.lost);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int sub = lane / LPV;
  const int c0 = lane % LPV * 4;   // this lane's four pairs: channels c0 .. and c0 + d_h / 2 ..
  // (1 + gamma) of them, for Q times the query scale
  float2 gq[4], gk[4];
  if constexpr (NORM) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + (e & 1) * 2 + (e >> 1) * (DH / 2);
      const float2 q = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.gq + c));
      const float2 k = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.gk + c));
      gq[e] = make_float2((1.f + q.x) * a.query_scale, (1.f + q.y) * a.query_scale);
      gk[e] = make_float2(1.f + k.x, 1.f + k.y);
    }
  }
  const bool in_smem = p.B <= kStartsMax;
  if (in_smem)
    for (int i = tid; i <= p.B; i += blockDim.x) starts[i] = __ldcg(p.row_start + i);
  // A row's steps are VPW heads of Q (finished without gammas), of K or of V each,
  // an item up to chunk_u of them.
  const int sq = NORM ? (a.H + VPW - 1) / VPW : 0, skv = (a.H_kv + VPW - 1) / VPW;
  const int iq = (sq + a.chunk_u - 1) / a.chunk_u, ik = (skv + a.chunk_u - 1) / a.chunk_u;
  const int nch = PACKED ? 1 : iq + 2 * ik;
  const int KVD = a.H_kv * DH;
  struct Item {
    int r, kind, head, left;   // row, 0 Q, 1 K, 2 V; this lane's first head, heads from it on
  };
  auto item_at = [&](int i) -> Item {
    Item t;
    t.r = i / nch;
    const int c = i - t.r * nch;
    t.kind = PACKED || c < iq ? 0 : (c < iq + ik ? 1 : 2);
    t.head = (t.kind == 0 ? c : (t.kind == 1 ? c - iq : c - iq - ik)) * a.chunk_u * VPW + sub;
    t.left = min((t.kind == 0 ? a.H : a.H_kv) - t.head, a.chunk_u * VPW - sub);
    return t;
  };
  struct Step {
    int kind, head;
    bool live;
  };
  auto step_of = [&](const Item& t, int u) -> Step {
    if constexpr (!PACKED) {
      return {t.kind, t.head + u * VPW, u * VPW < t.left};
    } else {
      const int kind = u < sq ? 0 : (u < sq + skv ? 1 : 2);
      const int head = (u - (kind == 0 ? 0 : (kind == 1 ? sq : sq + skv))) * VPW + sub;
      return {kind, head, u < a.chunk_u && head < (kind == 0 ? a.H : a.H_kv)};
    }
  };

  // This lane's two times 8 bytes of the item's vectors.
  uint2 raw[kVecUnroll][2];
  auto load = [&](int m0, const Item& t) {
    const long m = m0 + t.r;
    const __half* const q = a.Q + m * a.ldq + c0;
    const __half* const k = a.K + m * a.ldkv + c0;
    const __half* const v = a.V + m * a.ldkv + c0;
    const __half* const one = (t.kind == 0 ? q : (t.kind == 1 ? k : v)) + t.head * DH;
#pragma unroll
    for (int u = 0; u < kVecUnroll; ++u) {
      const Step s = step_of(t, u);
      if (s.live) {
        const __half* src = PACKED ? (s.kind == 0 ? q : (s.kind == 1 ? k : v)) + s.head * DH : one + u * VPW * DH;
        raw[u][0] = __ldcg(reinterpret_cast<const uint2*>(src));
        raw[u][1] = __ldcg(reinterpret_cast<const uint2*>(src + DH / 2));
      } else {
        raw[u][0] = raw[u][1] = make_uint2(0, 0);
      }
    }
  };

  for (int m0 = blockIdx.x * a.rows; m0 < p.M; m0 += gridDim.x * a.rows) {
    const int rows = min(a.rows, p.M - m0), items = rows * nch;
    int item = warp;
    Item t = item_at(item);
    if (item < items) load(m0, t);
    // ---------------- the rows' slots and positions
    __syncthreads();       // (starts are there; the rows before are done)
    if (tid < rows) {
      const int m = m0 + tid;
      const int b = sequence_of([&](int i) { return in_smem ? starts[i] : __ldcg(p.row_start + i); }, p.B, m);
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
      const long m = m0 + t.r;
      const int dst = dst_sh[t.r];
      if (dst == -2) {
        if (a.zero_behind && item == t.r * nch)   // (the row's first item; the others write nothing)
          for (int v = lane; v < a.H * LPV; v += 32)
            *reinterpret_cast<uint4*>(a.Qo + m * a.ldqo + v * 8) = make_uint4(0, 0, 0, 0);
      } else {
        __half* const q = a.Qo + m * a.ldqo + c0;
        const size_t slot = static_cast<size_t>(max(dst, 0)) * KVD + c0;
        __half* const one = (t.kind == 0 ? q : (t.kind == 1 ? a.Kp : a.Vp) + slot) + t.head * DH;
        if (NORM && (PACKED || t.kind != 2)) {
          float2 cs[2], sn[2], neg[2], g[4];
          const float pos = pos_sh[t.r];
          rope_sincos2(pos, freqs.f[c0], freqs.f[c0 + 1], sn[0], cs[0]);
          rope_sincos2(pos, freqs.f[c0 + 2], freqs.f[c0 + 3], sn[1], cs[1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = t.kind == 0 ? gq[e] : gk[e];
#pragma unroll
          for (int e = 0; e < 2; ++e) neg[e] = make_float2(-sn[e].x, -sn[e].y);
#pragma unroll
          for (int u = 0; u < kVecUnroll; ++u) {
            if (u >= a.chunk_u) break;   // warp-uniform
            if (PACKED) {
              const int kind = step_of(t, u).kind;
              if (kind == 2) break;
#pragma unroll
              for (int e = 0; e < 4; ++e) g[e] = kind == 0 ? gq[e] : gk[e];
            }
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = __half22float2(reinterpret_cast<const __half2*>(&raw[u][e >> 1])[e & 1]);
            float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(x[e], x[e], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int off = LPV / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            const float rs = rsqrtf(ss * (1.f / DH) + kEps);
            const float2 rr = make_float2(rs, rs);
            float2 o0[2], o1[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y0 = __fmul2_rn(__fmul2_rn(x[e], rr), g[e]);
              const float2 y1 = __fmul2_rn(__fmul2_rn(x[2 + e], rr), g[2 + e]);
              o0[e] = __ffma2_rn(y1, neg[e], __fmul2_rn(y0, cs[e]));
              o1[e] = __ffma2_rn(y0, sn[e], __fmul2_rn(y1, cs[e]));
            }
            raw[u][0] = make_uint2(pack_half2(o0[0].x, o0[0].y), pack_half2(o0[1].x, o0[1].y));
            raw[u][1] = make_uint2(pack_half2(o1[0].x, o1[0].y), pack_half2(o1[1].x, o1[1].y));
          }
        }
#pragma unroll
        for (int u = 0; u < kVecUnroll; ++u) {
          const Step s = step_of(t, u);
          if (s.live && (s.kind == 0 || dst >= 0)) {   // (no page: nothing is written)
            __half* to = PACKED ? (s.kind == 0 ? q : (s.kind == 1 ? a.Kp : a.Vp) + slot) + s.head * DH : one + u * VPW * DH;
            *reinterpret_cast<uint2*>(to) = raw[u][0];
            *reinterpret_cast<uint2*>(to + DH / 2) = raw[u][1];
          }
        }
      }
      item += kAppendWarps;
      t = item_at(item);
      if (item < items) load(m0, t);
    }
  }
  check_sequences(p, a.status);
}

// ---------------------------------------------------------------- commit
constexpr int kCommitThreads = 256;
constexpr int kCommitAhead = 8;      // rows in flight per thread
constexpr int kCommitChunk = kCommitThreads;   // accepted tokens per round of shared memory

// CTA (columns of 16 bytes, sequence, some of the layers' K and V): the slots
// are looked up once for all its pools; the next rows' loads are under way
// while a batch is stored (their slots lie behind it).
__global__ void __launch_bounds__(kCommitThreads)
    paged_commit_kernel(const PagedBatch p, const int32_t* __restrict__ accepted,
                        const int32_t* __restrict__ counts, int pools, int vecs, __half* Kp, __half* Vp,
                        int32_t* __restrict__ new_lens, int* status) {
  pdl_enter();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int32_t* path = accepted != nullptr ? accepted + static_cast<size_t>(b) * p.T_max : nullptr;
  // (the first accepted tokens are loaded beside the sequence)
  const int at0 = path != nullptr && tid < p.T_max ? __ldcg(path + tid) : 0;
  const int before0 = path != nullptr && tid > 0 && tid < p.T_max ? __ldcg(path + tid - 1) : -1;
  const int given = counts != nullptr ? __ldcg(counts + b) : -1;
  const PagedSeq s = paged_seq(p, b, status);
  const int count = counts != nullptr ? given : s.n;
  bool bad = count < 0 || count > s.n;
  if (!bad && path != nullptr)
    for (int i = tid; i < count; i += kCommitThreads) {
      const int at = i == tid ? at0 : __ldcg(path + i), before = i == tid ? before0 : __ldcg(path + i - 1);
      bad |= at >= s.n || at <= before;
    }
  bad = __syncthreads_or(bad);
  const bool head = blockIdx.x == 0 && blockIdx.z == 0;
  if (bad) {
    if (head && tid == 0) {
      record_error(status, kDevErrBadPaged);
      new_lens[b] = __ldcg(p.lens + b);
    }
    return;
  }
  // (a sequence that does not fit, without accepted tokens: as it was)
  if (head && tid == 0) new_lens[b] = count > 0 ? s.len + count : __ldcg(p.lens + b);
  if (path == nullptr) return;
  const size_t pool = (static_cast<size_t>(p.n_pages) << p.page_shift) * vecs;   // 16-byte vectors
  const int c = blockIdx.x * kCommitThreads + tid;
  __shared__ int src[kCommitChunk], dst[kCommitChunk];
  for (int i0 = 0; i0 < count; i0 += kCommitChunk) {
    const int n = min(kCommitChunk, count - i0);
    __syncthreads();
    for (int i = tid; i < n; i += kCommitThreads) {
      const int at = i0 == 0 ? at0 : __ldcg(path + i0 + i);   // (kCommitChunk tokens, a thread each)
      // a token that lies where it belongs is not moved
      const int from = at == i0 + i ? -1 : paged_row(p, b, s.len + at, status);
      const int to = at == i0 + i ? -1 : paged_row(p, b, s.len + i0 + i, status);
      src[i] = to < 0 ? -1 : from;
      dst[i] = to;
    }
    __syncthreads();
    if (c >= vecs) continue;
    for (int z = blockIdx.z; z < pools; z += gridDim.z) {
      uint4* base = reinterpret_cast<uint4*>(z & 1 ? Vp : Kp) + (z >> 1) * pool + c;
      uint4 v[kCommitAhead];
      auto load = [&](int i) {
#pragma unroll
        for (int u = 0; u < kCommitAhead; ++u)
          if (i + u < n && src[i + u] >= 0) v[u] = __ldcg(base + static_cast<size_t>(src[i + u]) * vecs);
      };
      load(0);
      for (int i = 0; i < n; i += kCommitAhead) {
        uint4 w[kCommitAhead];
#pragma unroll
        for (int u = 0; u < kCommitAhead; ++u) w[u] = v[u];
        load(i + kCommitAhead);
#pragma unroll
        for (int u = 0; u < kCommitAhead; ++u)
          if (i + u < n && src[i + u] >= 0) base[static_cast<size_t>(dst[i + u]) * vecs] = w[u];
      }
    }
  }
}

template <int DH>
cudaError_t launch_append_dh(const PagedBatch& batch, const AppendParams& p, bool norm,
                             const RopeFreqs& f, cudaStream_t stream) {
  AppendParams a = p;
  constexpr int vpw = 32 / (DH / 8);
  const int sq = norm ? (a.H + vpw - 1) / vpw : 0, skv = (a.H_kv + vpw - 1) / vpw, steps = sq + 2 * skv;   // of a row
  // Few rows: one per CTA, its steps spread over the warps; many: as many as
  // share out the rows over two CTAs per SM.
  const int slots = 2 * num_sms();
  const int rounds = (batch.M + slots * kAppendRows - 1) / (slots * kAppendRows);
  a.rows = (batch.M + slots * rounds - 1) / (slots * rounds);
  a.chunk_u = std::min(kVecUnroll, std::max(1, steps * a.rows / kAppendWarps));
  const int blocks = (batch.M + a.rows - 1) / a.rows;
  const dim3 grid(std::min(blocks, slots)), block(32 * kAppendWarps);
  if (!norm) return launch_pdl(paged_append_kernel<DH, false, false>, grid, block, 0, stream, batch, a, f);
  return steps <= a.chunk_u ? launch_pdl(paged_append_kernel<DH, true, true>, grid, block, 0, stream, batch, a, f)
                            : launch_pdl(paged_append_kernel<DH, true, false>, grid, block, 0, stream, batch, a, f);
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
  const int rows = batch.parents == nullptr ? kPositionThreads : kPositionThreads / 32;   // of a CTA
  return launch_pdl(paged_positions_kernel, dim3((batch.M + rows - 1) / rows), dim3(kPositionThreads), 0, stream,
                    batch, pos, status);
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
  const int x = (vecs + kCommitThreads - 1) / kCommitThreads, pools = 2 * layers;
  // up to six CTAs per SM share the pools (two fit at a time: 92 registers)
  const long long most = std::max(1LL, 6LL * num_sms() / (static_cast<long long>(x) * batch.B));
  const dim3 grid(x, batch.B, accepted != nullptr ? static_cast<unsigned>(std::min<long long>(pools, most)) : 1);
  return launch_pdl(paged_commit_kernel, grid, dim3(kCommitThreads), 0, stream, batch, accepted, counts, pools,
                    vecs, static_cast<__half*>(K_pages), static_cast<__half*>(V_pages), new_lens, status);
}

}  // namespace g3
