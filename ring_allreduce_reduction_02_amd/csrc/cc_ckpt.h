// Device code of the 8-bit activation checkpoints: 32 consecutive elements of a
// row share a power of two 2^e, the least for which the largest of them rounds
// to at most 127, and are kept as the integers nearest v / 2^e (ties to even).
// Dividing by a power of two and multiplying by it are exact, so a kept value is
// off by at most 2^e / 2, and has 7 significant bits: bf16 holds it as it is.
// The exponent's byte is e + 127, from 1 (blocks below 2^-120, and of zeros) to
// 248 (the largest floats, cut at 127 2^121); 255 marks a block that holds a NaN
// or an infinity and stands for NaN.
#pragma once

#include "cc_device.h"
#include "cc_llm.h"
#include "cc_wave.h"

namespace cc {
namespace {

// the exponent's byte for the largest magnitude's bits
__device__ __forceinline__ uint32_t kept_exponent(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  // top = 1.f 2^E: 2^(E - 6) gives [64, 128), of which 127.5 and above round to 128
  const int b = (int)(top >> 23) - 6 + ((top & 0x7fffffu) >= 0x7f0000u ? 1 : 0);
  return (uint32_t)(b < 1 ? 1 : b > 248 ? 248 : b);
}

template <int V>
struct Kept {
  uint32_t w[V / 4];
  uint32_t ex;
};

// V (4 or 8) kept integers on a multiple of V bytes, and their block's exponent
template <int V>
__device__ __forceinline__ Kept<V> kept_load(const char* p, const char* pe) {
  Kept<V> k;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) k.w[i] = ((const uint32_t*)p)[i];
  k.ex = *(const uint8_t*)pe;
  return k;
}
template <int V>
__device__ __forceinline__ void kept_unpack(const Kept<V>& k, float* v) {
  const float s = __uint_as_float(k.ex << 23);   // of 255: infinity, and 0 times it NaN
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = (float)((int)(k.w[i / 4] << (24 - 8 * (i & 3))) >> 24) * s;
}

// A block of 32 that LANES consecutive lanes hold, V each, `left` of this lane's
// inside the row: integers to p (zeros for those outside), the exponent to pe.
template <int V, int LANES>
__device__ __forceinline__ void kept_store(const float* v, int left, int lane, char* p, char* pe) {
  static_assert(V * LANES == kCkptBlock && (LANES == 4 || LANES == 8), "a block");
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = i < left && b > top ? b : top;
  }
  top = group_umax<LANES>(top);
  const uint32_t ex = kept_exponent(top);
  const float inv = __uint_as_float((254u - ex) << 23);   // 2^-e (unused where ex is 255)
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = __builtin_amdgcn_fmed3f(v[4 * i + j] * inv, -127.0f, 127.0f);
      // 1.5 2^23 more: the sum is rounded to an integer, whose low byte is the last of the bits
      b[j] = 4 * i + j < left ? __float_as_uint(t + 12582912.0f) : 0u;
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    w[i] = ex == 255u ? 0u : lo | hi;
  }
  if (left <= 0) return;
#pragma unroll
  for (int i = 0; i < V / 4; ++i) ((uint32_t*)p)[i] = w[i];
  if (lane % LANES == 0) *(uint8_t*)pe = (uint8_t)ex;
}

}  // namespace
}  // namespace cc
