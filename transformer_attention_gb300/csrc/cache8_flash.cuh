// Pieces shared by the tcgen05 kernels over the 8-bit cache: the launch
// arguments of the attention (cache8_flash.cu), and the conversion of cache
// bytes to swizzled fp16 tiles, used by it and by the weight pass
// (cache8_weights.cu).
#pragma once

#include <climits>
#include <cstdint>

#include "cache8.cuh"
#include "ptx.cuh"

namespace g3 {

struct Flash8Args {
  const void* Q;
  const void* K8;
  const void* V8;
  const float* K_scale;
  const float* V_scale;
  const int32_t* posc;
  const int32_t* qpos;
  const int32_t* pad_lens;
  int32_t* first;             // [B, items] scratch of local layers
  float2* stat;               // [B*T*H, nsplit] (max, sum) of each part, or null
  float* part;                // [B*T*H, nsplit, d_h] when nsplit > 1
  void* O;
  int o_f16, B, T, S, end, H, H_kv, d_h, window, nsplit;
  int* status;
};
// Tokens of one work item (one CTA per item, split, kv head and batch row).
int flash8_span(int d_h, int G);
cudaError_t launch_flash8(const Flash8Args& a, cudaStream_t stream);

// The probabilities that every slot received from the call's rows, added to
// weight_sum [B, S] (cache8_weights.cu).  rowstat [B*T*H] and wpart
// (weights8_part_floats() floats) are scratch.
constexpr int kWeights8MaxCtas = 1024;
constexpr size_t weights8_part_floats() { return static_cast<size_t>(kWeights8MaxCtas) * 128; }
cudaError_t launch_weights8(const Flash8Args& a, float2* rowstat, float* wpart, float* weight_sum,
                            cudaStream_t stream);

#ifdef __CUDACC__

// Stored positions [plo, phi] within the window of some query position in
// [qn, qx]: closer than `window`, and of a token (>= 0).
__device__ __forceinline__ void window_range(int qn, int qx, int window, int& plo, int& phi) {
  const long long a = static_cast<long long>(qn) - window + 1;
  const long long z = static_cast<long long>(qx) + window - 1;
  plo = static_cast<int>(a < 0 ? 0 : (a > INT_MAX ? INT_MAX : a));
  phi = static_cast<int>(z < -1 ? -1 : (z > INT_MAX ? INT_MAX : z));
}

// A part: 16 KB of cache bytes as 32 KB of fp16, by one warpgroup, 128 bytes
// per thread.  Wide parts (HALF false): 128 slots x 128 channels, 8 threads
// per slot; half parts: 64 slots x 256 channels, 16 threads per slot.  Global
// loads are whole 128-byte lines; the two 16-byte stores of a thread go out
// in an order that puts eight neighbouring threads on eight bank groups.
struct Part8 {
  const int32_t* pos;   // the batch row's positions
  int s_base, hi;       // first slot of tile 0; slots from hi on are hidden
  int plo, phi;         // positions outside are hidden
  int nb;               // blocks of the cache
};

struct Fetched8 {
  uint4 x[8];
  uint32_t ok;          // bit it: the slot of step it counts
  float s0, s1;         // scales of the first and second 64 slots
};

// Fetch part `half` (slots 64 * half .. of a half part) of tile i: num, scale
// point at the batch row's and head's first byte (plus a channel offset) and
// scale; ld, lds: elements between slots and between blocks.
template <bool HALF>
__device__ __forceinline__ void fetch8(Fetched8& f, const Part8& src, const uint8_t* num,
                                       const float* scale, int ld, int lds, int i, int half, int ct,
                                       bool any) {
  if (!any) return;
  constexpr int TPS = HALF ? 16 : 8;
  const int s0 = src.s_base + i * 128 + (HALF ? half * 64 : 0);
  const int row = ct / TPS;
  const uint8_t* a = num + (ct % TPS) * 16;
  uint32_t ok = 0;
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int s = s0 + row + it * (128 / TPS);
    int ps = -1;
    f.x[it] = make_uint4(0, 0, 0, 0);
    if (s < src.hi) {
      ps = __ldg(src.pos + s);
      f.x[it] = __ldg(reinterpret_cast<const uint4*>(a + static_cast<size_t>(s) * ld));
    }
    ok |= (ps >= src.plo && ps <= src.phi ? 1u : 0u) << it;
  }
  f.ok = ok;
  const int blk = s0 / kC8Block;
  f.s0 = __ldg(scale + static_cast<size_t>(min(blk, src.nb - 1)) * lds);
  f.s1 = HALF ? f.s0 : __ldg(scale + static_cast<size_t>(min(blk + 1, src.nb - 1)) * lds);
}

// Its values in fp16, hidden slots as zeros, to the 128-byte-swizzled chunks
// of 64 channels at dst.
template <bool HALF>
__device__ __forceinline__ void store8(const Fetched8& f, uint8_t* dst, int ct) {
  constexpr int TPS = HALF ? 16 : 8;
  constexpr uint32_t CH = HALF ? 64 * 128 : 128 * 128;
  const int col = ct % TPS;                    // 16-channel group
  const int u0 = (col & 3) * 2;
  const bool swap = (col & 4) != 0;
  const __half2 zero = __float2half2_rn(0.f);
  // (a scale above 128 can take a value past fp16's largest: 65504 there)
  const bool big = f.s0 > 128.f || f.s1 > 128.f;
  const __half2 h0 = __float2half2_rn(f.s0), h1 = __float2half2_rn(f.s1);
#pragma unroll
  for (int it = 0; it < 8; ++it) {
    const int row = ct / TPS + it * (128 / TPS);
    const bool ok = (f.ok >> it) & 1u;
    const __half2 s = ok ? (!HALF && it >= 4 ? h1 : h0) : zero;
    const uint32_t w[4] = {ok ? f.x[it].x : 0u, ok ? f.x[it].y : 0u, ok ? f.x[it].z : 0u,
                           ok ? f.x[it].w : 0u};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = c8_half2(w[k]), hi = c8_half2_hi(w[k]);
      __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), s);
      __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&hi), s);
      if (big) {
        const __half2 top = __float2half2_rn(65504.f);
        a = __hmax2_nan(__hmin2_nan(a, top), __hneg2(top));
        b = __hmax2_nan(__hmin2_nan(b, top), __hneg2(top));
      }
      o[2 * k] = *reinterpret_cast<uint32_t*>(&a);
      o[2 * k + 1] = *reinterpret_cast<uint32_t*>(&b);
    }
    uint8_t* base = dst + (col >> 2) * CH + row * 128;
    const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
    const int r7 = row & 7;
    *reinterpret_cast<uint4*>(base + (((u0 + (swap ? 1 : 0)) ^ r7) << 4)) = swap ? b : a;
    *reinterpret_cast<uint4*>(base + (((u0 + (swap ? 0 : 1)) ^ r7) << 4)) = swap ? a : b;
  }
}

// A warp's stores visible to the tensor core, then its arrival.
__device__ __forceinline__ void publish8(uint64_t& bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&bar));
}

#endif

}  // namespace g3
