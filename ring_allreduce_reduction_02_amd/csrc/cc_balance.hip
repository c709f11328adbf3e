// The loss that keeps the experts evenly used, and its gradient.  Over the T
// tokens of a batch that have a logit above -inf, with C_e the rows that the
// router gave expert e, S their sum and p_t the softmax of token t's E logits,
//
//   f_e = C_e / S      P_e = (1 / T) sum_t p_te      loss = E sum_e f_e P_e
//
// which is 1 where either is even.  C counts, so f has no gradient:
//
//   d loss / d l_te = (E / T) p_te (f_e - sum_j f_j p_tj).
//
// Both passes read the logits once, p in registers; sums are float32, each in a
// fixed order.

#include <algorithm>

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

constexpr int kV = 16;   // experts of a lane, so that 2^k lanes hold a token

struct BalArgs {
  const char* logits;
  uint64_t ls;
  const char* counts;
  uint64_t cs;
  char* total;
  uint64_t ts;
  char* prob;
  uint64_t ps;
  char* loss;
  uint64_t os;
  const char* base;
  uint64_t bs;
  char* dlogits;
  uint64_t ds;
  float* part;       // [N][blocks][E]
  uint32_t* live;    // [N][blocks]
  uint64_t tokens;
  uint32_t blocks;   // workgroups a rank
  int E, N, summed;
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Sums and maxima over the L = 2^k consecutive lanes of a token, on all of them,
// in a fixed order.
template <int L, class T, class F>
__device__ __forceinline__ T over_lanes(T x, F f) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) x = f(x, __shfl_xor(x, d));
  return x;
}

// Lane l of a token holds the 16-byte chunks q L + l of its row.
template <int DT, int L>
struct Row {
  static constexpr int CH = Ty<DT>::V, Q = kV / CH, SZ = Ty<DT>::SZ;
  __device__ __forceinline__ static int expert(int l, int q) { return (q * L + l) * CH; }
  __device__ __forceinline__ static void load(const char* row, int E, int l, float none, float* x) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = expert(l, q);
      if (e + CH <= E) {
        unpack<DT>(*(const u32x4_any*)(row + (uint64_t)e * SZ), x + q * CH);
      } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) x[q * CH + i] = e + i < E ? ld1<DT>(row + (uint64_t)(e + i) * SZ) : none;
      }
    }
  }
  __device__ __forceinline__ static void store(char* row, int E, int l, const float* x) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = expert(l, q);
      if (e + CH <= E) {
        *(u32x4_any*)(row + (uint64_t)e * SZ) = pack<DT>(x + q * CH);
      } else {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (e + i < E) st1<DT>(row + (uint64_t)(e + i) * SZ, x[q * CH + i]);
      }
    }
  }
};

// exp(l - max l) in place of the logits, and their sum: NaN if a logit is NaN or
// the maximum +inf, 0 if every logit is -inf.
template <int L>
__device__ __forceinline__ float exps(float* x) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kV; ++i) top = fmaxf(top, x[i]);
  top = over_lanes<L>(top, [](float a, float b) { return fmaxf(a, b); });
  const float m = top == -INFINITY ? 0.0f : top;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    x[i] = expf(x[i] - m);
    s += x[i];
  }
  return over_lanes<L>(s, [](float a, float b) { return a + b; });
}

// Workgroup b of a rank sums the probabilities of every blocks-th group of
// tokens and counts those that have any.
template <int DT, int L>
__global__ __launch_bounds__(kBalanceBlock) void k_balance(BalArgs a) {
  constexpr int PER = kBalanceBlock / L;    // tokens at a time
  typedef Row<DT, L> R;
  __shared__ float red[kBalanceBlock / 64][L * kV];
  __shared__ uint32_t red_live[kBalanceBlock / 64];
  const int tid = threadIdx.x, l = tid % L, lane = tid & 63, wave = tid >> 6;
  const uint64_t r = blockIdx.y;
  float sum[kV] = {};
  uint32_t live = 0;
  for (uint64_t t = (uint64_t)blockIdx.x * PER + tid / L; t < a.tokens; t += (uint64_t)a.blocks * PER) {
    float x[kV];
    R::load(a.logits + r * a.ls + t * a.E * R::SZ, a.E, l, -INFINITY, x);
    const float s = exps<L>(x);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[i] += x[i] * inv;
    live += l == 0 && s != 0.0f ? 1 : 0;
  }
#pragma unroll
  for (int d = L; d < 64; d <<= 1) {
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[i] += __shfl_xor(sum[i], d);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) live += __shfl_xor(live, d);
  if (lane < L) {
#pragma unroll
    for (int i = 0; i < kV; ++i) red[wave][R::expert(l, i / R::CH) + i % R::CH] = sum[i];
  }
  if (lane == 0) red_live[wave] = live;
  __syncthreads();
  const uint64_t at = r * a.blocks + blockIdx.x;
  for (int e = tid; e < a.E; e += kBalanceBlock)
    a.part[at * a.E + e] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
  if (tid == 0) a.live[at] = red_live[0] + red_live[1] + red_live[2] + red_live[3];
}

// The sums of a rank's workgroups (or of all ranks'), a workgroup: its threads
// are C = 64 .. 1024 columns times 1024 / C parts of the rows.
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void k_balance_join(BalArgs a) {
  __shared__ float sum[kJoin];
  __shared__ long long num[kJoin];
  const int tid = threadIdx.x, E = a.E;
  int C = 64;
  while (C < E) C *= 2;
  const int parts = kJoin / C, e = tid % C, part = tid / C;
  const uint32_t first = a.summed ? 0 : blockIdx.x, ranks = a.summed ? a.N : 1;
  const uint64_t row0 = (uint64_t)first * a.blocks, rows = (uint64_t)ranks * a.blocks;
  float s = 0.0f;
  if (e < E)
    for (uint64_t k = part; k < rows; k += parts) s += a.part[(row0 + k) * E + e];
  long long n = 0;
  for (uint64_t k = tid; k < rows; k += kJoin) n += a.live[row0 + k];
  sum[tid] = s;
  num[tid] = n;
  __syncthreads();
  for (int d = kJoin / 2; d; d >>= 1) {
    if (tid < d) {
      num[tid] += num[tid + d];
      if (d >= C) sum[tid] += sum[tid + d];
    }
    __syncthreads();
  }
  const long long T = num[0];
  const float p = e < E && part == 0 && T ? sum[tid] / (float)T : 0.0f;
  long long c = 0;
  if (e < E && part == 0)
    for (uint32_t r = 0; r < ranks; ++r) c += ((const int*)(a.counts + (uint64_t)(first + r) * a.cs))[e];
  __syncthreads();
  num[tid] = c;
  __syncthreads();
  for (int d = kJoin / 2; d; d >>= 1) {
    if (tid < d) num[tid] += num[tid + d];
    __syncthreads();
  }
  const long long S = num[0];
  sum[tid] = S ? ((float)c / (float)S) * p : 0.0f;
  __syncthreads();
  for (int d = kJoin / 2; d; d >>= 1) {
    if (tid < d) sum[tid] += sum[tid + d];
    __syncthreads();
  }
  for (uint32_t r = first; r < first + ranks; ++r) {
    if (e < E && part == 0) {
      ((int*)(a.total + (uint64_t)r * a.ts))[e] = (int)c;
      ((float*)(a.prob + (uint64_t)r * a.ps))[e] = p;
    }
    if (tid == 0) {
      ((int*)(a.total + (uint64_t)r * a.ts))[E] = (int)T;
      *(float*)(a.loss + (uint64_t)r * a.os) = (float)E * sum[0];
    }
  }
}

template <int DT, int L>
__global__ __launch_bounds__(kBalanceBlock) void k_balance_grad(BalArgs a) {
  constexpr int PER = kBalanceBlock / L;
  typedef Row<DT, L> R;
  const int tid = threadIdx.x, l = tid % L, E = a.E;
  const uint64_t r = blockIdx.y;
  const int* total = (const int*)(a.total + r * a.ts);
  float f[kV];
  long long S = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = R::expert(l, i / R::CH) + i % R::CH, c = e < E ? total[e] : 0;
    S += c;
    f[i] = (float)c;
  }
  S = over_lanes<L>(S, [](long long x, long long y) { return x + y; });
#pragma unroll
  for (int i = 0; i < kV; ++i) f[i] = S ? f[i] / (float)S : 0.0f;
  const int T = total[E];
  const float scale = T > 0 ? *(const float*)(a.loss + r * a.os) * ((float)E / (float)T) : 0.0f;
  for (uint64_t t = (uint64_t)blockIdx.x * PER + tid / L; t < a.tokens; t += (uint64_t)a.blocks * PER) {
    float x[kV], b[kV];
    R::load(a.logits + r * a.ls + t * E * R::SZ, E, l, -INFINITY, x);
    if (a.base) R::load(a.base + r * a.bs + t * E * R::SZ, E, l, 0.0f, b);
    const float s = exps<L>(x);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      x[i] *= inv;
      dot += x[i] * f[i];
    }
    dot = over_lanes<L>(dot, [](float u, float v) { return u + v; });
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      x[i] = scale * x[i] * (f[i] - dot);
      if (a.base) x[i] += b[i];
    }
    R::store(a.dlogits + r * a.ds + t * E * R::SZ, E, l, x);
  }
}

// lanes of a token
int lanes_of(int E) {
  int L = 1;
  while (L * kV < E) L *= 2;
  return L;
}

// Workgroups a rank: each takes `rounds` groups of tokens where there are enough
// of them to leave `most` workgroups.
uint32_t blocks_of(int N, uint64_t tokens, int E, uint32_t rounds, uint32_t most) {
  const uint64_t per = kBalanceBlock / lanes_of(E), groups = (tokens + per - 1) / per;
  const uint64_t each = std::max<uint64_t>(1, most / N);
  return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(each, (groups + rounds - 1) / rounds));
}
constexpr uint32_t kSumRounds = 4, kSumMost = 512, kGradRounds = 2, kGradMost = 2048;

BalArgs balance_args(const BalanceLaunch& L) {
  BalArgs a = {};
  a.logits = L.logits; a.ls = L.logits_stride;
  a.counts = L.counts; a.cs = L.counts_stride;
  a.total = L.total; a.ts = L.total_stride;
  a.prob = L.prob; a.ps = L.prob_stride;
  a.loss = L.loss; a.os = L.loss_stride;
  a.base = L.base; a.bs = L.base_stride;
  a.dlogits = L.dlogits; a.ds = L.dlogits_stride;
  a.tokens = L.tokens;
  a.E = L.nexperts; a.N = L.N; a.summed = L.summed;
  return a;
}

template <bool GRAD, int DT, int LN>
hipError_t run_balance(const BalArgs& a, hipStream_t st) {
  const dim3 grid(a.blocks, (unsigned)a.N), blk(kBalanceBlock);
  if constexpr (GRAD) CC_LAUNCH((k_balance_grad<DT, LN>), grid, blk, 0, st, a);
  else CC_LAUNCH((k_balance<DT, LN>), grid, blk, 0, st, a);
  return hipGetLastError();
}
template <bool GRAD, int DT>
hipError_t pick_balance(const BalArgs& a, hipStream_t st) {
  switch (lanes_of(a.E)) {
    case 1: return run_balance<GRAD, DT, 1>(a, st);
    case 2: return run_balance<GRAD, DT, 2>(a, st);
    case 4: return run_balance<GRAD, DT, 4>(a, st);
    case 8: return run_balance<GRAD, DT, 8>(a, st);
    case 16: return run_balance<GRAD, DT, 16>(a, st);
    case 32: return run_balance<GRAD, DT, 32>(a, st);
    default: return run_balance<GRAD, DT, 64>(a, st);
  }
}
static_assert(kMaxRouteExperts <= 64 * kV, "a wave holds a token");

}  // namespace

uint64_t balance_ws(int N, uint64_t tokens, int nexperts) {
  return (uint64_t)N * blocks_of(N, tokens, nexperts, kSumRounds, kSumMost) * ((uint64_t)nexperts + 1) * 4;
}

hipError_t launch_balance(const BalanceLaunch& L) {
  BalArgs a = balance_args(L);
  a.blocks = blocks_of(L.N, L.tokens, L.nexperts, kSumRounds, kSumMost);
  a.part = (float*)L.ws;
  a.live = (uint32_t*)(a.part + (uint64_t)L.N * a.blocks * L.nexperts);
  const hipError_t e = L.dt == DT_F32 ? pick_balance<false, DT_F32>(a, L.st) : pick_balance<false, DT_BF16>(a, L.st);
  if (e != hipSuccess) return e;
  CC_LAUNCH(k_balance_join, dim3(L.summed ? 1u : (unsigned)L.N), dim3(kJoin), 0, L.st, a);
  return hipGetLastError();
}

hipError_t launch_balance_grad(const BalanceLaunch& L) {
  BalArgs a = balance_args(L);
  a.blocks = blocks_of(L.N, L.tokens, L.nexperts, kGradRounds, kGradMost);
  return L.dt == DT_F32 ? pick_balance<true, DT_F32>(a, L.st) : pick_balance<true, DT_BF16>(a, L.st);
}

}  // namespace cc
