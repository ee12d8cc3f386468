// qpn_kv_lanes.h -- values of other lanes of a wavefront, and reductions over it, without LDS.
#pragma once

#include "qpn_common.h"

namespace qpn {

namespace {

// x (32 bits, or a double) of another lane by a data-parallel move: within four lanes (quad_perm
// 1 0 3 2: 0xB1, 2 3 0 1: 0x4E), mirrored within eight (0x141), within sixteen (0x140).
template <int CTRL, typename T>
__device__ __forceinline__ T moved(T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ double moved(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// x of a given lane: uniform.
template <typename T>
__device__ __forceinline__ T of_lane(T x, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ double of_lane(double x, int lane) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Over the wavefront, all of whose lanes are here: within 16 lanes by moves, then the four
// rows' first lanes.  Uniform.
template <typename T, typename Op>
__device__ __forceinline__ T wave_reduced(T x, Op op) {
  x = op(x, moved<0xB1>(x));
  x = op(x, moved<0x4E>(x));
  x = op(x, moved<0x141>(x));
  x = op(x, moved<0x140>(x));
  return op(op(of_lane(x, 0), of_lane(x, 16)), op(of_lane(x, 32), of_lane(x, 48)));
}

}  // namespace

}  // namespace qpn
