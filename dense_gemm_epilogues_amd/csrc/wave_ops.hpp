// Reductions over the lanes of a wave by DPP, whose moves ride on vector instructions (a shuffle through LDS takes its latency).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// lane ^ D of an already reduced group of D lanes: within 16 lanes the mirrored half or row holds the same value
template <int D>
__device__ __forceinline__ uint32_t lane_xor32(uint32_t v) {
  constexpr int ctrl = D == 1 ? 0xb1 : D == 2 ? 0x4e : D == 4 ? 0x141 : 0x140;  // quad_perm [1,0,3,2], [2,3,0,1], row_half_mirror, row_mirror
  if constexpr (D < 16) return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, ctrl, 0xf, 0xf, true);
  else return (uint32_t)__shfl_xor((int)v, D);
}
template <int D, class T>
__device__ __forceinline__ T lane_xor(T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, lane_xor32<D>(__builtin_bit_cast(uint32_t, v)));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(T, (uint64_t)lane_xor32<D>((uint32_t)(b >> 32)) << 32 | lane_xor32<D>((uint32_t)b));
  }
}

// f over L neighbouring lanes, in every one of them; f is associative and commutative (the sums' order is fixed: the same in all lanes)
template <int L, class T, class F>
__device__ __forceinline__ T lanes_reduce(T v, F f) {
  if constexpr (L > 1) v = f(v, lane_xor<1>(v));
  if constexpr (L > 2) v = f(v, lane_xor<2>(v));
  if constexpr (L > 4) v = f(v, lane_xor<4>(v));
  if constexpr (L > 8) v = f(v, lane_xor<8>(v));
  if constexpr (L > 16) v = f(v, lane_xor<16>(v));
  if constexpr (L > 32) v = f(v, lane_xor<32>(v));
  return v;
}

template <class T>
__device__ __forceinline__ T read_lane(T v, int lane) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(T, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32 |
                                     (uint32_t)__builtin_amdgcn_readlane((int)b, lane));
  }
}

// the same over a whole wave, from the first lanes of its four rows, as a uniform value
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, F f) {
  v = lanes_reduce<16>(v, f);
  return f(f(read_lane(v, 0), read_lane(v, 16)), f(read_lane(v, 32), read_lane(v, 48)));
}

}  // namespace ep
