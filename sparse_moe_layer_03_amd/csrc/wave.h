// Reductions over a wave without LDS: rows of 16 lanes by shifts within the
// row, then rows to rows, the result taken from lane 63.  Fixed order; some 8
// instructions where a butterfly of LDS permutes waits for LDS six times.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
// (lanes that a shift leaves without a source take `neutral`)
template <typename OP>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t neutral, OP op) {
  v = op(v, dpp<0x111, 0xf>(neutral, v));  // row_shr 1
  v = op(v, dpp<0x112, 0xf>(neutral, v));
  v = op(v, dpp<0x114, 0xf>(neutral, v));
  v = op(v, dpp<0x118, 0xf>(neutral, v));
  v = op(v, dpp<0x142, 0xa>(neutral, v));  // lane 15 of rows 0, 2 to rows 1, 3
  v = op(v, dpp<0x143, 0xc>(neutral, v));  // lane 31 to rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_min_u(uint32_t v) {
  return wave_reduce(v, ~0u, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_max_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0xff800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(lane_value(__float_as_uint(v), lane));
}

// The value of lane ^ O, once lanes that differ in lower bits only hold the same
// one (as in a butterfly from 1 upwards): a mirror serves for 4 and 8.
template <int O>
__device__ __forceinline__ float partner(float v) {
  const uint32_t u = __float_as_uint(v);
  if constexpr (O == 1) return __uint_as_float(dpp<0xb1, 0xf>(u, u));        // quads 1 0 3 2
  else if constexpr (O == 2) return __uint_as_float(dpp<0x4e, 0xf>(u, u));   // quads 2 3 0 1
  else if constexpr (O == 4) return __uint_as_float(dpp<0x141, 0xf>(u, u));  // 8 lanes mirrored
  else if constexpr (O == 8) return __uint_as_float(dpp<0x140, 0xf>(u, u));  // 16 lanes mirrored
  else return __shfl_xor(v, O, 64);
}

}  // namespace moe
