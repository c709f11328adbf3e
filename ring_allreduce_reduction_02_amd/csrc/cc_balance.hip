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
#include "cc_wave.h"

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

// Lane l of the L that hold a token has the 16-byte chunks q L + l of its row.
template <int DT, int L>
struct Row {
  static constexpr int CH = Ty<DT>::V, Q = kV / CH, SZ = Ty<DT>::SZ;
  u32x4 w[Q];
  __device__ __forceinline__ static int expert(int l, int q) { return (q * L + l) * CH; }
  // elements past E: -inf (PAD_LOW) or 0
  template <bool PAD_LOW>
  __device__ __forceinline__ void load(const char* row, int E, int l) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = expert(l, q);
      if (e + CH <= E) {
        w[q] = __builtin_nontemporal_load((const u32x4_any*)(row + (uint64_t)e * SZ));
      } else {
        float x[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i)
          x[i] = e + i < E ? ld1<DT>(row + (uint64_t)(e + i) * SZ) : PAD_LOW ? -INFINITY : 0.0f;
        w[q] = pack_row<DT>(x);   // widened and packed again: the same bits
      }
    }
  }
  __device__ __forceinline__ void values(float* x) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) unpack<DT>(w[q], x + q * CH);
  }
  __device__ __forceinline__ static void store(char* row, int E, int l, const float* x) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = expert(l, q);
      if (e + CH <= E) {
        __builtin_nontemporal_store((u32x4_any)pack_row<DT>(x + q * CH), (u32x4_any*)(row + (uint64_t)e * SZ));
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
// bf16: the hardware's exp2 (1 ulp) of the difference d times log2(e), whose
// rounding and the constant's make (1.25 |d| + 2) 2^-24 of the value, the size of
// what d's own rounding makes of float32 logits; expf on them.
template <int DT, int L>
__device__ __forceinline__ float exps(float* x) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < kV; ++i) top = fmaxf(top, x[i]);
  top = group_max<L>(top);
  const float m = top > -INFINITY ? top : 0.0f;   // (NaN, where every logit is one: they stay NaN)
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if constexpr (DT == DT_BF16) x[i] = __builtin_amdgcn_exp2f((x[i] - m) * 1.44269504088896341f);
    else x[i] = expf(x[i] - m);
    s += x[i];
  }
  return group_sum<L>(s);
}

// Workgroup b of a rank sums the probabilities of every blocks-th group of
// tokens and counts those that have any; the next group's logits are under way
// meanwhile.  16 experts a lane: of 64, 4 lanes hold a token and each sum over
// them takes 2 moves where a wave a token takes 6 (with 8-byte chunks and moves
// through LDS 8.0 us where this takes 4.2).  Bound by the latency of a group's
// loads and exponentials: 8 x 4096 tokens of 64 bf16 4.2 us (at best 3.9), 1.0 TB/s;
// 3 x 1023 of 61 float32 5.3 (4.7); long batches by memory: 8 x 32768 of 256 bf16,
// 134 MB, 28 us (26), 4.8 TB/s, float32 48, 5.6 TB/s.
template <int DT, int L>
__global__ __launch_bounds__(kBalanceBlock) void k_balance(BalArgs a) {
  constexpr int G = kBalanceBlock / L, C = L * kV;      // tokens at a time, columns
  constexpr int P = C < kBalanceBlock ? kBalanceBlock / C : 1;   // parts of a column's sum
  typedef Row<DT, L> R;
  __shared__ __attribute__((aligned(16))) float red[G][C];
  __shared__ float part[P][C];
  __shared__ uint32_t red_live[kBalanceBlock / 64];
  const int tid = threadIdx.x, l = tid % L;
  const uint64_t r = blockIdx.y, step = (uint64_t)a.blocks * G, pitch = (uint64_t)a.E * R::SZ;
  const char* logits = a.logits + r * a.ls;
  float sum[kV] = {};
  uint32_t live = 0;
  R now, next;
  uint64_t t = (uint64_t)blockIdx.x * G + tid / L;
  if (t < a.tokens) next.template load<true>(logits + t * pitch, a.E, l);
  for (; t < a.tokens; t += step) {
    now = next;
    if (t + step < a.tokens) next.template load<true>(logits + (t + step) * pitch, a.E, l);
    float x[kV];
    now.values(x);
    const float s = exps<DT, L>(x);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[i] = __builtin_fmaf(x[i], inv, sum[i]);
    live += l == 0 && s != 0.0f ? 1 : 0;
  }
  live = group_usum<64>(live);
  if ((tid & 63) == 0) red_live[tid >> 6] = live;
#pragma unroll
  for (int i = 0; i < kV; ++i) red[tid / L][R::expert(l, i / R::CH) + i % R::CH] = sum[i];
  __syncthreads();
  const uint64_t at = r * a.blocks + blockIdx.x;
  for (int e = tid % C; e < C; e += kBalanceBlock) {
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < G / P; ++g) s += red[tid / C * (G / P) + g][e];
    if constexpr (P > 1) part[tid / C][e] = s;
    else if (e < a.E) a.part[at * a.E + e] = s;
  }
  if constexpr (P > 1) {
    __syncthreads();
    if (tid < a.E) {
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) s += part[p][tid];
      a.part[at * a.E + tid] = s;
    }
  }
  if (tid == 0) a.live[at] = red_live[0] + red_live[1] + red_live[2] + red_live[3];
}

// The sums of a rank's workgroups (or of all ranks'), a workgroup: its threads
// are C = 64 .. 1024 columns times 1024 / C parts of the rows.  One column's sums,
// counts and loss then lie in the threads below C, whose waves are joined.  Bound by
// the latency of a launch and of its rounds of loads: 5.0 us (at best 4.6) after 8 x 4096
// tokens of 64, 3.6 (3.3) after 3 x 1023 of 61, 10.4 (10.0) after 8 x 32768 of 256,
// whose 512 rows of sums are 16 rounds.
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void k_balance_join(BalArgs a) {
  __shared__ float sum[kJoin];
  __shared__ uint32_t num[2][kJoin / 64];
  __shared__ float lsum[kJoin / 64];
  const int tid = threadIdx.x, wave = tid >> 6, E = a.E;
  int C = 64;
  while (C < E) C *= 2;
  const int parts = kJoin / C, e = tid % C, part = tid / C;
  const uint32_t first = a.summed ? 0 : blockIdx.x, ranks = a.summed ? a.N : 1;
  const uint64_t row0 = (uint64_t)first * a.blocks;
  const uint32_t rows = ranks * a.blocks;
  float s = 0.0f;
  if (e < E) {
    const float* p = a.part + row0 * E + e;
    uint32_t k = part;
    for (; k + 7 * parts < rows; k += 8 * parts) {   // eight loads under way
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[(uint64_t)(k + i * parts) * E];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; k < rows; k += parts) s += p[(uint64_t)k * E];
  }
  uint32_t n = 0;
  for (uint32_t k = tid; k < rows; k += kJoin) n += a.live[row0 + k];
  long long c = 0;
  if (tid < E)
    for (uint32_t r = 0; r < ranks; ++r) c += ((const int*)(a.counts + (uint64_t)(first + r) * a.cs))[tid];
  sum[tid] = s;
  n = group_usum<64>(n);
  // 64-bit sums in two halves (ranks times int32: the upper ones below 2^21)
  const uint32_t lo = group_usum<64>((uint32_t)(c & 0xffff)), hi = group_usum<64>((uint32_t)(c >> 16));
  __shared__ uint32_t live[kJoin / 64];
  if ((tid & 63) == 0) {
    live[wave] = n;
    num[0][wave] = lo;
    num[1][wave] = hi;
  }
  __syncthreads();
  uint32_t T = 0;
  long long S = 0;
#pragma unroll
  for (int w = 0; w < kJoin / 64; ++w) {
    T += live[w];
    S += (long long)num[0][w] + ((long long)(int)num[1][w] << 16);
  }
  float p = 0.0f, v = 0.0f;
  if (tid < E) {
    for (int k = 0; k < parts; ++k) p += sum[k * C + tid];
    p = T ? p / (float)T : 0.0f;
    v = S ? ((float)c / (float)S) * p : 0.0f;
  }
  v = group_sum<64>(v);
  if ((tid & 63) == 0) lsum[wave] = v;
  __syncthreads();
  float loss = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoin / 64; ++w) loss += lsum[w];
  for (uint32_t r = first; r < first + ranks; ++r) {
    int* total = (int*)(a.total + (uint64_t)r * a.ts);
    if (tid < E) {
      total[tid] = (int)c;
      ((float*)(a.prob + (uint64_t)r * a.ps))[tid] = p;
    }
    if (tid == 0) {
      total[E] = (int)T;
      *(float*)(a.loss + (uint64_t)r * a.os) = (float)E * loss;
    }
  }
}

// A group of tokens at a time as in the sums; f from the counts, once a workgroup.
// Bound by memory from some megabytes on: 8 x 32768 tokens of 256 bf16, 268 MB in and
// out, 54 us, 5.0 TB/s, its vector instructions 51% of the cycles, float32 91, 5.9 TB/s;
// below that by latency: 8 x 4096 of 64 float32 added to another gradient 7.5 us (at
// best 6.8), 3.4 TB/s.
template <int DT, int L, bool BASE>
__global__ __launch_bounds__(kBalanceBlock) void k_balance_grad(BalArgs a) {
  constexpr int G = kBalanceBlock / L;
  typedef Row<DT, L> R;
  const int tid = threadIdx.x, l = tid % L, E = a.E;
  const uint64_t r = blockIdx.y, step = (uint64_t)a.blocks * G, pitch = (uint64_t)E * R::SZ;
  const char* logits = a.logits + r * a.ls;
  const char* base = a.base + r * a.bs;
  char* out = a.dlogits + r * a.ds;
  uint64_t t = (uint64_t)blockIdx.x * G + tid / L;
  R now, next, add, next_add;
  if (t < a.tokens) {
    next.template load<true>(logits + t * pitch, E, l);
    if constexpr (BASE) next_add.template load<false>(base + t * pitch, E, l);
  }
  const int* total = (const int*)(a.total + r * a.ts);
  float f[kV];
  uint32_t lo = 0, hi = 0;   // the counts' sum, of at most 1024 below 2^31, in two halves
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = R::expert(l, i / R::CH) + i % R::CH, c = e < E ? total[e] : 0;
    lo += (uint32_t)(c & 0xffff);
    hi += (uint32_t)(c >> 16);
    f[i] = (float)c;
  }
  const long long S = (long long)group_usum<L>(lo) + ((long long)(int)group_usum<L>(hi) << 16);
  const float one = S ? 1.0f / (float)S : 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) f[i] *= one;
  const int T = total[E];
  const float scale = T > 0 ? *(const float*)(a.loss + r * a.os) * ((float)E / (float)T) : 0.0f;
  for (; t < a.tokens; t += step) {
    now = next;
    add = next_add;
    if (t + step < a.tokens) {
      next.template load<true>(logits + (t + step) * pitch, E, l);
      if constexpr (BASE) next_add.template load<false>(base + (t + step) * pitch, E, l);
    }
    float x[kV], b[kV];
    now.values(x);
    if constexpr (BASE) add.values(b);
    const float s = exps<DT, L>(x);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    float dot = 0.0f;   // of f and the exponentials
#pragma unroll
    for (int i = 0; i < kV; ++i) dot = __builtin_fmaf(x[i], f[i], dot);
    dot = group_sum<L>(dot) * inv;
    const float k = s == 0.0f ? 0.0f : scale * inv;   // a padding token's row is 0 for any dloss
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      x[i] *= k;
      x[i] = BASE ? __builtin_fmaf(x[i], f[i] - dot, b[i]) : x[i] * (f[i] - dot);
    }
    R::store(out + t * pitch, E, l, x);
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
// Measured, a pass in a graph.  Sums and join of 8 x 4096 tokens of 64 bf16 and
// 3 x 1023 of 61 float32: with 1 round 8.9 and 6.6 us, 2 8.4 and 7.5, 4 9.9 and 9.4; of
// 8 x 32768 of 256 and 32768 of 1024 bf16: with 256 workgroups in all 50 and 40, 512 38
// and 44, 1024 43 and 65 (the join's one workgroup reads their sums).  Gradient of
// 8 x 512, 4096 and 16384 tokens of 64 float32, added: with 1 round 4.3, 7.7 and 24.1, 2
// 5.2, 7.7 and 22.9, 4 8.2, 11.1 and 23.6; of 8 x 32768 of 256 float32: 512 107, 1024 96,
// 2048 91, 4096 89.
uint32_t blocks_of(int N, uint64_t tokens, int E, uint32_t rounds, uint32_t most) {
  const uint64_t per = kBalanceBlock / lanes_of(E), groups = (tokens + per - 1) / per;
  const uint64_t each = std::max<uint64_t>(1, most / N);
  return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(each, (groups + rounds - 1) / rounds));
}
constexpr uint32_t kSumRounds = 2, kSumMost = 512, kGradRounds = 2, kGradMost = 2048;

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
  if constexpr (!GRAD) CC_LAUNCH((k_balance<DT, LN>), grid, blk, 0, st, a);
  else if (a.base) CC_LAUNCH((k_balance_grad<DT, LN, true>), grid, blk, 0, st, a);
  else CC_LAUNCH((k_balance_grad<DT, LN, false>), grid, blk, 0, st, a);
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
