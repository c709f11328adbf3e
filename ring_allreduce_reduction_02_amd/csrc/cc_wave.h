// Reductions over a wave or over groups of its lanes by data-parallel moves (no
// trip through LDS), in a fixed order, and 16-byte vectors of results.
#pragma once

#include "cc_device.h"

namespace cc {
namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_of(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, false);
}

// f over each L = 2^k consecutive lanes (from a multiple of L), on all of them; f
// gives the same in either order of its arguments.  All lanes of a group are
// active.
template <int L, class F>
__device__ __forceinline__ uint32_t over_group(uint32_t x, F f) {
  if constexpr (L >= 2) x = f(x, dpp_of<0xB1>(x));     // quad_perm [1,0,3,2]
  if constexpr (L >= 4) x = f(x, dpp_of<0x4E>(x));     // quad_perm [2,3,0,1]
  if constexpr (L >= 8) x = f(x, dpp_of<0x141>(x));    // row_half_mirror
  if constexpr (L >= 16) x = f(x, dpp_of<0x140>(x));   // row_mirror
  if constexpr (L >= 32) x = f(x, (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401F));   // lanes i ^ 16
  if constexpr (L >= 64) x = f(x, (uint32_t)__shfl_xor((int)x, 32));
  return x;
}
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  return __uint_as_float(over_group<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ float group_max(float x) {
  return __uint_as_float(over_group<L>(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t group_usum(uint32_t x) {
  return over_group<L>(x, [](uint32_t a, uint32_t b) { return a + b; });
}
template <int L>
__device__ __forceinline__ uint32_t group_umax(uint32_t x) {
  return over_group<L>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// Reductions over a wave by data-parallel moves (within 16 lanes, then across
// rows), the result on every lane (a scalar): a tenth of the latency of shuffles
// through LDS.  The order is fixed.  All 64 lanes are active.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, 0xf, 0xf, false);
}
template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, uint32_t none, F f) {
  x = f(x, moved<0x111>(x, none));   // row_shr 1, 2, 4, 8
  x = f(x, moved<0x112>(x, none));
  x = f(x, moved<0x114>(x, none));
  x = f(x, moved<0x118>(x, none));
  x = f(x, moved<0x142>(x, none));   // row_bcast 15, 31
  x = f(x, moved<0x143>(x, none));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
  return wave_reduce(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ uint32_t wave_umin(uint32_t x) {
  return wave_reduce(x, 0xffffffffu, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float wave_max(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), 0xff800000u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// V floats in one 16-byte vector; bf16 by the hardware's conversion (nearest,
// ties to even), one instruction for two elements
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ u32x4 pack_row(const float* v) {
  if constexpr (DT == DT_BF16) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{v[2 * i], v[2 * i + 1]}), bf16x2));
    return w;
  } else {
    return pack<DT>(v);
  }
}

}  // namespace
}  // namespace cc
