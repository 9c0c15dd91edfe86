// Values exchanged between the lanes of a wave by register moves.
#pragma once

#include "common.hpp"

namespace gptq {

// The value of lane ^ M within the wave: register moves between lanes (a few
// cycles each; through LDS one is about 100, and a sort makes 21 in a row).
template <int M>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (M == 1) return __builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // quad 1 0 3 2
  else if constexpr (M == 2) return __builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // 2 3 0 1
  else if constexpr (M == 3) return __builtin_amdgcn_mov_dpp((int)v, 0x1B, 0xF, 0xF, true);  // 3 2 1 0
  else if constexpr (M == 7) return __builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);  // mirror of 8
  else if constexpr (M == 8) return __builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true);  // rotate 16 by 8
  else if constexpr (M == 15) return __builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);  // mirror of 16
  else if constexpr (M == 4) return lane_xor<3>(lane_xor<7>(v));
  else if constexpr (M == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? p[0] : p[1];
  } else if constexpr (M == 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? p[0] : p[1];
  } else if constexpr (M == 31) return lane_xor<16>(lane_xor<15>(v));
  else {
    static_assert(M == 63, "masks that the sort uses");
    return lane_xor<32>(lane_xor<31>(v));
  }
}
template <int M>
__device__ __forceinline__ uint64_t lane_xor64(uint64_t v) {
  return (uint64_t)lane_xor<M>((uint32_t)(v >> 32)) << 32 | lane_xor<M>((uint32_t)v);
}
template <int M>
__device__ __forceinline__ float lane_xorf(float v) {
  return __uint_as_float(lane_xor<M>(__float_as_uint(v)));
}

// The largest v of each aligned run of LPG lanes (a power of two), in all of them.
// After the steps before, a lane and its mirror image hold the same value, so the
// mirrors of 8 and 16 stand for the exchanges with lane ^ 4 and lane ^ 8.
template <int LPG>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPG >= 2) v = fmaxf(v, lane_xorf<1>(v));
  if constexpr (LPG >= 4) v = fmaxf(v, lane_xorf<2>(v));
  if constexpr (LPG >= 8) v = fmaxf(v, lane_xorf<7>(v));
  if constexpr (LPG >= 16) v = fmaxf(v, lane_xorf<15>(v));
  if constexpr (LPG >= 32) v = fmaxf(v, lane_xorf<16>(v));
  if constexpr (LPG >= 64) v = fmaxf(v, lane_xorf<32>(v));
  return v;
}

}  // namespace gptq
