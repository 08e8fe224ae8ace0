// Reductions over the lanes of a wave.
#pragma once
#include "device_common.h"

namespace gmlp {

// Rotation by N within each 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float ror16(float v) { return __uint_as_float(ror16<N>(__float_as_uint(v))); }
template <int N>
__device__ __forceinline__ uint64_t ror16(uint64_t v) {
  return ((uint64_t)ror16<N>((uint32_t)(v >> 32)) << 32) | ror16<N>((uint32_t)v);
}
template <int N>
__device__ __forceinline__ double ror16(double v) {
  return __longlong_as_double((long long)ror16<N>((uint64_t)__double_as_longlong(v)));
}
// All-reduce over LPR = 16 or 64 lanes (all of the wave active): the same value, bit for bit, in every one of them
// (each step joins the same two values in either order; f commutes).
template <int LPR, class T, class F>
__device__ __forceinline__ T lanes_reduce(T v, F f) {
  v = f(v, ror16<8>(v));
  v = f(v, ror16<4>(v));
  v = f(v, ror16<2>(v));
  v = f(v, ror16<1>(v));
  if constexpr (LPR == 64) {
    v = f(v, __shfl_xor(v, 16, 64));
    v = f(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int LPR, class T>
__device__ __forceinline__ T lanes_sum(T v) { return lanes_reduce<LPR>(v, [](T a, T b) { return a + b; }); }
template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_reduce<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}
// What the wave's lanes wrote to LDS before is what they read from it behind.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

}  // namespace gmlp
