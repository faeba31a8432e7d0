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
  float2* rowstat;            // [B, H_kv, T*G] (reference, 1 / sum) of every row, or null
  float2* pstat;              // [flash8_part_rows()] and
  float* part;                // [flash8_part_rows(), d_h]: scratch of cut units
  void* O;
  int o_f16, B, T, S, end, H, H_kv, d_h, window;
  int* status;
  int lost;                   // errors (ptx.cuh) after which no weight is added
};
// Tokens of one work item.
int flash8_span(int d_h, int G);
size_t flash8_part_rows(int B, int T, int S, int H, int H_kv, int d_h);
cudaError_t launch_flash8(const Flash8Args& a, cudaStream_t stream);

// The probabilities that every slot received from the call's rows, added to
// weight_sum [B, S] (cache8_weights.cu), from a.rowstat.  wpart: scratch of
// weights8_part_floats() floats.
constexpr int kWeights8MaxCtas = 1024;
constexpr size_t weights8_part_floats() { return static_cast<size_t>(kWeights8MaxCtas) * 128; }
cudaError_t launch_weights8(const Flash8Args& a, float* wpart, float* weight_sum,
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

// A block's scale in the fp16 tiles.  At scales above 128 a value can pass
// fp16's largest (a token's 65504 is stored as 65536, an infinity as 448 *
// 256): the tiles take half of it there, and the products with it are doubled.
__device__ __forceinline__ bool halved(float scale) { return scale > 128.f; }
__device__ __forceinline__ __half2 tile_scale(float scale) {
  return __float2half2_rn(halved(scale) ? 0.5f * scale : scale);
}

// 16 cache bytes (one slot's channels 16 col .. 16 col + 15) as fp16 values in
// a 128-byte-swizzled tile: base points at the slot's 128-byte row in the
// chunk of 64 channels that holds them.  scale: the block's as two fp16
// (tile_scale), or 0 with a = b = 0 for a hidden slot.  The two 16-byte stores go out
// in an order that puts eight neighbouring threads (col 0..7 of a slot) on
// eight bank groups: a and b are the 8 bytes of the first and the second
// store, the upper half first where swap8 is 1 (by the slot too, so that 8-byte
// loads of two slots' bytes meet no conflict either).
__device__ __forceinline__ int swap8(int col, int row) { return ((col >> 2) ^ row) & 1; }

__device__ __forceinline__ uint4 values8(uint2 w, __half2 scale) {
  const uint32_t in[2] = {w.x, w.y};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = c8_half2(in[k]), hi = c8_half2_hi(in[k]);
    const __half2 v0 = __hmul2(*reinterpret_cast<const __half2*>(&lo), scale);
    const __half2 v1 = __hmul2(*reinterpret_cast<const __half2*>(&hi), scale);
    o[2 * k] = *reinterpret_cast<const uint32_t*>(&v0);
    o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&v1);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void store16_values(uint2 a, uint2 b, __half2 scale, int col, int row,
                                               uint8_t* base) {
  const int u0 = (col & 3) * 2, swap = swap8(col, row), r7 = row & 7;
  *reinterpret_cast<uint4*>(base + (((u0 + swap) ^ r7) << 4)) = values8(a, scale);
  *reinterpret_cast<uint4*>(base + (((u0 + 1 - swap) ^ r7) << 4)) = values8(b, scale);
}

// A query row's entry of rowstat: (reference, 1 / sum of exp2 against it), or
// (inf, 0) for a row that saw nothing, whose weights come out as zeros.
__device__ __forceinline__ float2 row_stat(float m, float l, bool any) {
  return any ? make_float2(m, 1.f / l) : make_float2(INFINITY, 0.f);
}

// A warp's stores visible to the tensor core, then its arrival.
__device__ __forceinline__ void publish8(uint64_t& bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&bar));
}

#endif

}  // namespace g3
