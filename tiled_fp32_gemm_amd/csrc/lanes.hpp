// lanes.hpp -- sums over groups of lanes and over a workgroup.
//
// Every lane of a group gets the sum, with the same bits: a butterfly adds the
// same two halves on both sides.  Within 16 lanes it is four DPP steps; the four
// rows of a wave meet in scalar registers, the waves of a workgroup in LDS.
#pragma once

#include "common.hpp"

namespace sg {

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// Over the 16 lanes of a DPP row, all of them active.
__device__ __forceinline__ float sum16(float v) {
  v += dpp_of<0xB1>(v);    // quad_perm 1, 0, 3, 2
  v += dpp_of<0x4E>(v);    // quad_perm 2, 3, 0, 1
  v += dpp_of<0x141>(v);   // row_half_mirror
  v += dpp_of<0x140>(v);   // row_mirror
  return v;
}

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Over a whole wave.
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// K sums over the L lanes of a row: 16 or 64 lanes, or a workgroup of L threads,
// whose waves meet in `part` (K L / 64 floats that no wave still reads).
template <int L, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float* part) {
  static_assert(L == 16 || L == 64 || L == 256 || L == 1024, "lanes of a row");
  if constexpr (L == 16) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum16(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = sum64(v[k]);
  }
  if constexpr (L > 64) {
    constexpr int WAVES = L / 64;
    const int wave = (int)threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) part[wave * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s[WAVES];
#pragma unroll
      for (int w = 0; w < WAVES; ++w) s[w] = part[w * K + k];
#pragma unroll
      for (int half = WAVES / 2; half > 0; half /= 2)
#pragma unroll
        for (int w = 0; w < half; ++w) s[w] += s[w + half];
      v[k] = s[0];
    }
  }
}

}  // namespace sg
