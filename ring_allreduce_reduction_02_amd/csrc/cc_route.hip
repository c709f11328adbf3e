// Routing of tokens to experts and its gradient.
//
// A token's probabilities are the softmax of its E logits; its experts are
// the topk largest logits, ties to the lowest index.  A logit of -inf (a
// masked expert) or NaN is never chosen: the slot's expert is -1, its weight
// 0.  Weights are the chosen probabilities, or with `normalize` those divided
// by their sum.  Maximum and sums are float32.
//
// The gradient, with w the weights and u the weights' gradient put back on
// the experts: dl = p (u - sum p u), p the softmax over all experts, or over
// the chosen ones with `normalize`.

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

constexpr int kRouteBlock = 256;
constexpr int kRouteWaves = kRouteBlock / 64;

struct RouteArgs {
  const char* logits;
  uint64_t ls;
  char* experts;
  uint64_t es;
  char* weights;
  uint64_t wgs;
  char* dlogits;
  uint64_t ds;
  uint64_t tokens;
  int E, K, normalize;
};

// order-preserving bits of a logit; 0 for NaN and -inf (never chosen), and
// -0 as +0
__device__ __forceinline__ uint32_t rank_bits(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  if ((u & 0x7fffffffu) > 0x7f800000u || u == 0xff800000u) return 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Reductions over a wave by data-parallel moves (within 16 lanes, then across
// rows), the result on every lane: a tenth of the latency of shuffles through
// LDS.  The order is fixed.
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

// A token's logits over a wave, V a lane: lane l holds experts q * 64 + l.
// ex becomes exp(logit - maximum); returns its sum (NaN if a logit is NaN, or
// the maximum +inf; 0 if every logit is -inf).
template <int DT, int V>
__device__ __forceinline__ float load_exp(const char* row, int E, int lane, float* x, float* ex) {
  float top = -INFINITY;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int e = q * 64 + lane;
    x[q] = e < E ? ld1<DT>(row + (uint64_t)e * Ty<DT>::SZ) : -INFINITY;
    top = fmaxf(top, x[q]);
  }
  top = wave_max(top);
  const float m = top == -INFINITY ? 0.0f : top;
  float s = 0.0f;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    ex[q] = expf(x[q] - m);
    s += ex[q];
  }
  return wave_sum(s);
}

// Both kernels are bound by their vector instructions, 265 and 176 a token of top-8
// of 64, which take about 90 and 80% of the cycles: 8 x 4096 tokens 16 us and 12 us
// (4.2 to 17 MB of memory traffic, 1-4 us of it).
//
// One wave a token.  The chosen experts one after the other: the largest bits
// of the wave, the lowest index that has them, then taken out.
template <int DT, int V>
__global__ __launch_bounds__(kRouteBlock) void k_route(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t t = (uint64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6), r = blockIdx.y;
  if (t >= a.tokens) return;
  float x[V], ex[V];
  const float all = load_exp<DT, V>(a.logits + r * a.ls + t * a.E * Ty<DT>::SZ, a.E, lane, x, ex);
  uint32_t key[V];
#pragma unroll
  for (int q = 0; q < V; ++q) key[q] = rank_bits(x[q]);
  int my_e = -1;       // slot `lane`
  float my_p = 0.0f, chosen = 0.0f;
  for (int s = 0; s < a.K; ++s) {
    uint32_t mine = key[0], first = 0;
#pragma unroll
    for (int q = 1; q < V; ++q)
      if (key[q] > mine) {
        mine = key[q];
        first = q;
      }
    const uint32_t best = wave_umax(mine);
    if (best == 0) break;
    // the lowest index that has it
    int e;
    if constexpr (V == 1) e = __builtin_ctzll(__ballot(mine == best));
    else e = (int)wave_umin(mine == best ? first * 64 + lane : 0xffffffffu);
    float p = 0.0f;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (q * 64 + lane == e) {
        key[q] = 0;
        p = ex[q];
      }
    }
    p = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(p), e & 63));
    chosen += p;
    if (lane == s) {
      my_e = e;
      my_p = p;
    }
  }
  if (lane < a.K) {
    const uint64_t at = t * a.K + lane;
    ((int*)(a.experts + r * a.es))[at] = my_e;
    float w = 0.0f;
    if (my_e >= 0) w = all != all ? all : my_p / (a.normalize ? chosen : all);
    ((float*)(a.weights + r * a.wgs))[at] = w;
  }
}

template <int DT, int V>
__global__ __launch_bounds__(kRouteBlock) void k_route_grad(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t t = (uint64_t)blockIdx.x * kRouteWaves + (threadIdx.x >> 6), r = blockIdx.y;
  if (t >= a.tokens) return;
  float x[V], p[V], u[V];
  float all = load_exp<DT, V>(a.logits + r * a.ls + t * a.E * Ty<DT>::SZ, a.E, lane, x, p);
  const bool nan = all != all;
  const int my_e = lane < a.K ? ((const int*)(a.experts + r * a.es))[t * a.K + lane] : -1;
  const float my_d = lane < a.K ? ((const float*)(a.weights + r * a.wgs))[t * a.K + lane] : 0.0f;
  uint32_t picked = 0;
#pragma unroll
  for (int q = 0; q < V; ++q) u[q] = 0.0f;
  for (int s = 0; s < a.K; ++s) {
    const int e = __builtin_amdgcn_readlane(my_e, s);
    const float d = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(my_d), s));
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (q * 64 + lane == e) {
        u[q] += d;
        picked |= 1u << q;
      }
    }
  }
  if (a.normalize) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (!((picked >> q) & 1u)) p[q] = 0.0f;
      s += p[q];
    }
    all = wave_sum(s);
  }
  const float inv = all > 0.0f ? 1.0f / all : 0.0f;
  float dot = 0.0f;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    p[q] *= inv;
    dot += p[q] != 0.0f ? p[q] * u[q] : 0.0f;
  }
  dot = wave_sum(dot);
  char* o = a.dlogits + r * a.ds + t * a.E * Ty<DT>::SZ;
#pragma unroll
  for (int q = 0; q < V; ++q) {
    const int e = q * 64 + lane;
    const float d = nan ? __uint_as_float(0x7fc00000u) : p[q] != 0.0f ? p[q] * (u[q] - dot) : 0.0f;
    if (e < a.E) st1<DT>(o + (uint64_t)e * Ty<DT>::SZ, d);
  }
}

template <bool GRAD, int DT, int V>
hipError_t run_route(const RouteArgs& a, const RouteLaunch& L) {
  const dim3 grid((unsigned)((L.tokens + kRouteWaves - 1) / kRouteWaves), (unsigned)L.N), blk(kRouteBlock);
  if constexpr (GRAD) CC_LAUNCH((k_route_grad<DT, V>), grid, blk, 0, L.st, a);
  else CC_LAUNCH((k_route<DT, V>), grid, blk, 0, L.st, a);
  return hipGetLastError();
}

template <bool GRAD, int DT>
hipError_t pick_route(const RouteArgs& a, const RouteLaunch& L) {
  if (a.E <= 64) return run_route<GRAD, DT, 1>(a, L);
  if (a.E <= 128) return run_route<GRAD, DT, 2>(a, L);
  if (a.E <= 256) return run_route<GRAD, DT, 4>(a, L);
  if (a.E <= 512) return run_route<GRAD, DT, 8>(a, L);
  return run_route<GRAD, DT, kMaxRouteExperts / 64>(a, L);
}

RouteArgs route_args(const RouteLaunch& L) {
  return RouteArgs{L.logits, L.logits_stride, L.experts, L.experts_stride, L.weights, L.weights_stride,
                   L.dlogits, L.dlogits_stride, L.tokens, L.nexperts, L.topk, L.normalize};
}

}  // namespace

hipError_t launch_route(const RouteLaunch& L) {
  return L.dt == DT_F32 ? pick_route<false, DT_F32>(route_args(L), L) : pick_route<false, DT_BF16>(route_args(L), L);
}

hipError_t launch_route_grad(const RouteLaunch& L) {
  return L.dt == DT_F32 ? pick_route<true, DT_F32>(route_args(L), L) : pick_route<true, DT_BF16>(route_args(L), L);
}

}  // namespace cc
