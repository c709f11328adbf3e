// The gated feed-forward block of MoE experts on the expert side of the
// capacity-padded dispatch, and its gradients.  For a row x of an expert with
// weights w_in = [gate; up] (2F x W) and w_out (W x F):
//
//   [g | u] = x w_in^T      h = act(g) u      y = h w_out^T
//   dh = dy w_out           dg = dh u act'(g)      du = dh act(g)
//   dx = [dg | du] w_in     dw_in = [dg | du]^T x  dw_out = dy^T h
//
// Five grouped matrix products over the experts' kept rows, each one launch:
// the first ends in the activation and the product, the third in the
// activation's derivative.  Products run on the matrix cores and sum in
// float32; h, dg and du are rounded once to the buffers' type between two
// products, because the matrix cores read that type.

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

enum Kind { K_GATEUP = 0, K_DOWN = 1, K_DHID = 2, K_DX = 3, K_DW = 4 };

constexpr int kKBytes = 128;   // bytes of the summed axis per stage and line
constexpr int kUnits = 4;      // matrix instruction steps per stage: 32 bytes of the summed axis each

// ------------------------------------------------------------------ plan

constexpr int kPlanCounts = 896;   // counts that fit a launch's arguments
struct PutArgs {
  uint32_t v[kPlanCounts];
  uint32_t* to;
  int n;
};
__global__ __launch_bounds__(256) void k_ffn_put(PutArgs a) {
  for (int i = threadIdx.x; i < a.n; i += 256) a.to[i] = a.v[i];
}

struct PlanArgs {
  uint32_t v[kPlanCounts];
  const uint32_t* kept;   // in memory, or NULL: v
  int N, E, tile;
  uint64_t cap;
  int* start;
  int2* mtab;
  int* rowmap;
};

// Workgroup e writes expert e's first compact row, its row tiles and its rows'
// places in the rank's buffer.
__global__ __launch_bounds__(256) void k_ffn_plan(PlanArgs a) {
  __shared__ uint32_t red[2][256];
  const int e = blockIdx.x, tid = threadIdx.x, N = a.N;
  const uint32_t* kept = a.kept ? a.kept : a.v;
  uint32_t rows = 0, tiles = 0;
  for (int x = tid; x < e; x += 256) {
    uint32_t n = 0;
    for (int i = 0; i < N; ++i) n += kept[x * N + i];
    rows += n;
    tiles += (n + a.tile - 1) / a.tile;
  }
  red[0][tid] = rows;
  red[1][tid] = tiles;
  __syncthreads();
  for (int d = 128; d; d >>= 1) {
    if (tid < d) {
      red[0][tid] += red[0][tid + d];
      red[1][tid] += red[1][tid + d];
    }
    __syncthreads();
  }
  const uint32_t r0 = red[0][0], t0 = red[1][0];
  const int per = a.E / N, l = e % per;
  uint32_t at = r0;
  for (int i = 0; i < N; ++i) {
    const uint32_t n = kept[e * N + i];
    const uint32_t src = (uint32_t)(((uint64_t)i * per + l) * a.cap);
    for (uint32_t s = tid; s < n; s += 256) a.rowmap[at + s] = (int)(src + s);
    at += n;
  }
  const uint32_t nt = (at - r0 + a.tile - 1) / a.tile;
  for (uint32_t t = tid; t < nt; t += 256) a.mtab[t0 + t] = make_int2(e, (int)(r0 + t * a.tile));
  if (tid == 0) {
    a.start[e] = (int)r0;
    if (e == a.E - 1) a.start[a.E] = (int)at;
  }
}

// ------------------------------------------------------------------ operands

// Rows of the experts: compact (map NULL), or in the ranks' buffers.
struct RowSide {
  char* base;
  uint64_t rank_stride;
  uint64_t pitch;
  const int* map;
};
// One matrix an expert.
struct WtSide {
  char* base;
  uint64_t rank_stride;
  uint64_t expert_stride;
  uint64_t pitch;
};

__device__ __forceinline__ char* row_ptr(const RowSide& s, int rank, int p) {
  return s.map ? s.base + (uint64_t)rank * s.rank_stride + (uint64_t)s.map[p] * s.pitch
               : s.base + (uint64_t)p * s.pitch;
}
__device__ __forceinline__ char* wt_ptr(const WtSide& s, int rank, int local) {
  return s.base + (uint64_t)rank * s.rank_stride + (uint64_t)local * s.expert_stride;
}

struct GemmArgs {
  const int* start;
  const int2* mtab;
  int mtiles, ntiles;
  int E, per;            // experts, experts per rank
  int M, N, K;           // columns of the result; summed length (row products); K_DW: M x N results
  int F;                 // hidden size
  int act;
  RowSide a;             // rows: the m lines, or (K_DW) the summed lines
  WtSide b;              // weights (row products)
  RowSide b_rows;        // K_DW: the other factor
  RowSide out;           // rows out
  RowSide pre;           // gate and up pre-activations (base NULL: not kept)
  RowSide h;             // compact h (K_DHID)
  WtSide wout;           // K_DW
};

// ------------------------------------------------------------------ LDS tiles

// Lines along the summed axis ("row" tiles: R lines of 128 bytes): 16-byte
// chunks permuted by the line's low bits, so that a fragment's lanes, one
// line each, spread over the banks.
__device__ __forceinline__ int row_at(int r, int chunk) { return r * kKBytes + ((chunk ^ (r & 7)) << 4); }

template <int DT>
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (DT == DT_BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
  }
}

// The 16 bytes of a lane for unit u of 32 lines from i0: line i0 + lane % 32,
// elements of half lane / 32 of the unit.
template <int DT, bool COL, int R>
__device__ __forceinline__ u32x4 frag(const char* t, int u, int i0, int lane) {
  const int i = i0 + (lane & 31), half = lane >> 5;
  if constexpr (!COL) {
    return *(const u32x4*)(t + row_at(i, 2 * u + half));
  } else if constexpr (DT == DT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 16 * u + 8 * half + 2 * j;
      w[j] = (uint32_t)*(const uint16_t*)(t + (k * R + i) * 2) |
             (uint32_t)*(const uint16_t*)(t + ((k + 1) * R + i) * 2) << 16;
    }
    return u32x4{w[0], w[1], w[2], w[3]};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = *(const uint32_t*)(t + ((8 * u + 4 * half + j) * R + i) * 4);
    return u32x4{w[0], w[1], w[2], w[3]};
  }
}

// Element-wise staging of a tile: any alignment.  Row tiles: lp[r] is line
// r's first byte (NULL: zeros), elements [k0, K).  Column tiles: lp[k] is
// summed line k0 + k (NULL: zeros), columns [c0, C).
template <int DT, bool COL, int R, int NT>
__device__ __forceinline__ void stage_elems(char* t, const char* const* lp, int64_t k0, int64_t K, int64_t c0,
                                            int64_t C) {
  constexpr int SZ = Ty<DT>::SZ, BK = kKBytes / SZ;
  for (int e = threadIdx.x; e < R * BK; e += NT) {
    uint32_t v = 0;
    int at;
    if constexpr (!COL) {
      const int r = e / BK, k = e % BK;
      const char* p = lp[r];
      if (p && k0 + k < K) v = SZ == 2 ? *(const uint16_t*)(p + (k0 + k) * SZ) : *(const uint32_t*)(p + (k0 + k) * SZ);
      at = row_at(r, k * SZ / 16) + (k * SZ) % 16;
    } else {
      const int k = e / R, c = e % R;
      const char* p = lp[k];
      if (p && c0 + c < C) v = SZ == 2 ? *(const uint16_t*)(p + (c0 + c) * SZ) : *(const uint32_t*)(p + (c0 + c) * SZ);
      at = (k * R + c) * SZ;
    }
    if constexpr (SZ == 2) *(uint16_t*)(t + at) = (uint16_t)v;
    else *(uint32_t*)(t + at) = v;
  }
}

// ------------------------------------------------------------------ activations

enum Act { ACT_SILU = 0, ACT_GELU = 1 };

__device__ __forceinline__ float act_of(float g, int act) {
  if (act == ACT_SILU) return g / (1.0f + expf(-g));
  return 0.5f * g * erfcf(-g * 0.70710678118654752f);
}
// the activation and its derivative
__device__ __forceinline__ void act_both(float g, int act, float* a, float* d) {
  if (act == ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-g));
    *a = g * s;
    *d = s * (1.0f + g * (1.0f - s));
  } else {
    const float c = 0.5f * erfcf(-g * 0.70710678118654752f);
    *a = g * c;
    *d = c + g * expf(-0.5f * g * g) * 0.39894228040143268f;
  }
}

// four consecutive elements of a row, n of them inside it
template <int DT, bool VEC>
__device__ __forceinline__ void store4(char* p, const float* v, int n) {
  if constexpr (VEC) {
    if (n <= 0) return;
    if constexpr (DT == DT_BF16)
      *(u32x2*)p = u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
    else
      *(u32x4*)p = pack<DT_F32>(v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) st1<DT>(p + i * Ty<DT>::SZ, v[i]);
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ void load4(const char* p, float* v, int n) {
  if constexpr (VEC) {
    if (n <= 0) return;
    if constexpr (DT == DT_BF16) {
      const u32x2 w = *(const u32x2*)p;
      v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      unpack<DT_F32>(*(const u32x4*)p, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? ld1<DT>(p + i * Ty<DT>::SZ) : 0.0f;
  }
}

// ------------------------------------------------------------------ the products

// A workgroup computes a BM x BN tile with (BM / WM) x (BN / WN) waves, each
// WM x WN of it in tiles of 32 x 32.  The weights' lines are the matrix
// instruction's first operand, so a lane ends with groups of four consecutive
// columns of one row.  K_GATEUP takes BN / 2 hidden columns: the tile's lines
// alternate 32 gate rows and the 32 up rows of the same columns, so that one
// lane holds both.
template <int DT, int KIND, bool VEC, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_ffn_gemm(GemmArgs g) {
  constexpr int NT = 64 * (BM / WM) * (BN / WN);
  constexpr int SZ = Ty<DT>::SZ, BK = kKBytes / SZ;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr bool ACOL = KIND == K_DW, BCOL = KIND == K_DHID || KIND == K_DX || KIND == K_DW;
  static_assert(KIND != K_GATEUP || TN == 2, "a wave holds 32 gate and the same 32 up columns");
  __shared__ __attribute__((aligned(16))) char ta[BM * kKBytes];
  __shared__ __attribute__((aligned(16))) char tb[BN * kKBytes];
  __shared__ const char* la[ACOL ? BK : BM];
  __shared__ const char* lb[BCOL ? BK : BN];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % (BM / WM), wn = wave / (BM / WM);
  int e, p0, p1, m0, n0;   // expert, its rows from here, their end, tile origin
  if constexpr (KIND == K_DW) {
    const int per_e = g.mtiles * g.ntiles;
    e = blockIdx.x / per_e;
    const int t = blockIdx.x - e * per_e;
    m0 = (t % g.mtiles) * BM;
    n0 = (t / g.mtiles) * BN;
    p0 = g.start[e];
    p1 = g.start[e + 1];
  } else {
    const int2 mt = g.mtab[blockIdx.x % g.mtiles];
    e = mt.x;
    p0 = mt.y;
    p1 = g.start[e + 1];
    m0 = 0;
    n0 = (blockIdx.x / g.mtiles) * (KIND == K_GATEUP ? BN / 2 : BN);
  }
  const int rank = e / g.per, local = e % g.per;
  const int64_t K = KIND == K_DW ? p1 - p0 : g.K;

  // lines that stay for the whole product
  if constexpr (!ACOL)
    for (int r = tid; r < BM; r += NT) la[r] = p0 + r < p1 ? row_ptr(g.a, rank, p0 + r) : nullptr;
  if constexpr (!BCOL) {
    const char* w = wt_ptr(g.b, rank, local);
    for (int r = tid; r < BN; r += NT) {
      int64_t row;
      bool in;
      if constexpr (KIND == K_GATEUP) {
        const int f = n0 + (r / 64) * 32 + (r & 31);
        in = f < g.F;
        row = (int64_t)((r >> 5) & 1) * g.F + f;
      } else {
        in = n0 + r < g.N;
        row = n0 + r;
      }
      lb[r] = in ? w + row * (int64_t)g.b.pitch : nullptr;
    }
  }

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  for (int64_t k0 = 0; k0 < K; k0 += BK) {
    __syncthreads();
    if constexpr (ACOL || BCOL) {
      if (tid < BK) {
        const int64_t k = k0 + tid;
        if constexpr (ACOL) la[tid] = k < K ? row_ptr(g.a, rank, (int)(p0 + k)) : nullptr;
        if constexpr (KIND == K_DW) lb[tid] = k < K ? row_ptr(g.b_rows, rank, (int)(p0 + k)) : nullptr;
        else lb[tid] = k < K ? wt_ptr(g.b, rank, local) + k * (int64_t)g.b.pitch : nullptr;
      }
      __syncthreads();
    }
    stage_elems<DT, ACOL, BM, NT>(ta, la, k0, K, m0, g.M);
    stage_elems<DT, BCOL, BN, NT>(tb, lb, k0, K, n0, g.N);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      u32x4 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = frag<DT, ACOL, BM>(ta, u, wm * WM + 32 * i, lane);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = frag<DT, BCOL, BN>(tb, u, wn * WN + 32 * j, lane);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[j], fa[i], acc[i][j]);
    }
  }

  // a lane's results: row m (of the tile) = lane % 32 of a 32-tile, columns
  // 8 q + 4 (lane / 32) + 0..3 of it for q = 0..3
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = wm * WM + 32 * i + (lane & 31);
    const bool in = KIND == K_DW ? m0 + m < g.M : p0 + m < p1;
    if (!in) continue;
    if constexpr (KIND == K_DW) {
      char* o = wt_ptr(g.wout, rank, local) + (uint64_t)(m0 + m) * g.wout.pitch;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * WN + 32 * j + 8 * q + 4 * (lane >> 5);
          const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          store4<DT, VEC>(o + (int64_t)n * SZ, v, g.N - n);
        }
    } else if constexpr (KIND == K_DOWN || KIND == K_DX) {
      char* o = row_ptr(g.out, rank, p0 + m);
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * WN + 32 * j + 8 * q + 4 * (lane >> 5);
          const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          store4<DT, VEC>(o + (int64_t)n * SZ, v, g.N - n);
        }
    } else if constexpr (KIND == K_GATEUP) {
      char* o = row_ptr(g.out, rank, p0 + m);
      char* pre = g.pre.base ? row_ptr(g.pre, rank, p0 + m) : nullptr;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int f = n0 + wn * 32 + 8 * q + 4 * (lane >> 5);
        float gt[4], up[4], h[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          gt[x] = acc[i][0][4 * q + x];
          up[x] = acc[i][1][4 * q + x];
          h[x] = act_of(gt[x], g.act) * up[x];
        }
        store4<DT, VEC>(o + (int64_t)f * SZ, h, g.F - f);
        if (pre) {
          store4<DT, VEC>(pre + (int64_t)f * SZ, gt, g.F - f);
          store4<DT, VEC>(pre + ((int64_t)g.F + f) * SZ, up, g.F - f);
        }
      }
    } else {   // K_DHID
      char* o = row_ptr(g.out, rank, p0 + m);
      char* oh = row_ptr(g.h, rank, p0 + m);
      const char* pre = row_ptr(g.pre, rank, p0 + m);
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = n0 + wn * WN + 32 * j + 8 * q + 4 * (lane >> 5);
          float gt[4], up[4], dg[4], du[4], h[4];
          load4<DT, VEC>(pre + (int64_t)f * SZ, gt, g.F - f);
          load4<DT, VEC>(pre + ((int64_t)g.F + f) * SZ, up, g.F - f);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float dh = acc[i][j][4 * q + x];
            float a, d;
            act_both(gt[x], g.act, &a, &d);
            dg[x] = dh * up[x] * d;
            du[x] = dh * a;
            h[x] = a * up[x];
          }
          store4<DT, VEC>(o + (int64_t)f * SZ, dg, g.F - f);
          store4<DT, VEC>(o + ((int64_t)g.F + f) * SZ, du, g.F - f);
          store4<DT, VEC>(oh + (int64_t)f * SZ, h, g.F - f);
        }
    }
  }
}

template <int DT, int KIND, bool VEC>
hipError_t run_gemm(GemmArgs g, hipStream_t st) {
  constexpr int BM = kFfnRowTile, BN = 128;
  const int cols = KIND == K_GATEUP ? g.F : g.N;
  g.ntiles = (cols + (KIND == K_GATEUP ? BN / 2 : BN) - 1) / (KIND == K_GATEUP ? BN / 2 : BN);
  uint64_t blocks;
  if constexpr (KIND == K_DW) {
    g.mtiles = (g.M + BM - 1) / BM;
    blocks = (uint64_t)g.E * g.mtiles * g.ntiles;
  } else {
    blocks = (uint64_t)g.mtiles * g.ntiles;
  }
  if (blocks == 0) return hipSuccess;
  CC_LAUNCH((k_ffn_gemm<DT, KIND, VEC, BM, BN, 64, 64>), dim3((unsigned)blocks), dim3(256), 0, st, g);
  return hipGetLastError();
}

template <int KIND>
hipError_t pick_gemm(const GemmArgs& g, const FfnLaunch& L) {
  if (L.s.dt == DT_F32)
    return L.vec_ok ? run_gemm<DT_F32, KIND, true>(g, L.st) : run_gemm<DT_F32, KIND, false>(g, L.st);
  return L.vec_ok ? run_gemm<DT_BF16, KIND, true>(g, L.st) : run_gemm<DT_BF16, KIND, false>(g, L.st);
}

uint64_t up256(uint64_t v) { return (v + 255) / 256 * 256; }

// the tables, from the counts in the launch's arguments or (many) in memory
hipError_t plan(const FfnLaunch& L, int tile) {
  PlanArgs a;
  const int n = L.s.N * L.s.E;
  a.kept = nullptr;
  if (n <= kPlanCounts) {
    for (int i = 0; i < n; ++i) a.v[i] = L.kept[i];
  } else {
    uint32_t* to = (uint32_t*)(L.ws + L.o.kept);
    for (int i = 0; i < n; i += kPlanCounts) {
      PutArgs p;
      p.n = n - i < kPlanCounts ? n - i : kPlanCounts;
      for (int k = 0; k < p.n; ++k) p.v[k] = L.kept[i + k];
      p.to = to + i;
      CC_LAUNCH(k_ffn_put, dim3(1), dim3(256), 0, L.st, p);
    }
    a.kept = to;
  }
  a.N = L.s.N; a.E = L.s.E; a.tile = tile; a.cap = L.s.cap;
  a.start = (int*)(L.ws + L.o.start);
  a.mtab = (int2*)(L.ws + L.o.mtab);
  a.rowmap = (int*)(L.ws + L.o.rowmap);
  CC_LAUNCH(k_ffn_plan, dim3((unsigned)L.s.E), dim3(256), 0, L.st, a);
  return hipGetLastError();
}

GemmArgs gemm_args(const FfnLaunch& L) {
  GemmArgs g = {};
  g.start = (const int*)(L.ws + L.o.start);
  g.mtab = (const int2*)(L.ws + L.o.mtab);
  g.mtiles = (int)L.s.mtiles;
  g.E = L.s.E;
  g.per = L.s.E / L.s.N;
  g.F = (int)L.s.F;
  g.act = L.s.act;
  return g;
}

RowSide rows_of(const FfnLaunch& L, const Side& s, uint64_t cols) {
  return RowSide{s.base, s.stride, cols * elem_size(L.s.dt), (const int*)(L.ws + L.o.rowmap)};
}
RowSide compact(const FfnLaunch& L, uint64_t off, uint64_t cols) {
  return RowSide{L.ws + off, 0, cols * elem_size(L.s.dt), nullptr};
}
WtSide wts(const FfnLaunch& L, const Side& s, uint64_t r, uint64_t c) {
  const uint64_t es = elem_size(L.s.dt);
  return WtSide{s.base, s.stride, r * c * es, c * es};
}

}  // namespace

FfnWs ffn_ws(const FfnShape& s, int grad) {
  FfnWs o;
  const uint64_t es = elem_size(s.dt);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += up256(bytes);
    return p;
  };
  o.kept = take((uint64_t)s.N * s.E * 4);
  o.start = take(((uint64_t)s.E + 1) * 4);
  o.mtab = take(s.mtiles * 8);
  o.rowmap = take(s.rows * 4);
  o.h = take(s.rows * s.F * es);
  o.dgu = grad ? take(s.rows * 2 * s.F * es) : 0;
  o.bytes = at;
  return o;
}

hipError_t launch_ffn(const FfnLaunch& L) {
  const uint64_t W = L.s.W, F = L.s.F;
  hipError_t e = plan(L, kFfnRowTile);
  if (e != hipSuccess) return e;
  GemmArgs g = gemm_args(L);
  g.K = (int)W;
  g.N = (int)(2 * F);
  g.a = rows_of(L, L.x, W);
  g.b = wts(L, L.w_in, 2 * F, W);
  g.out = compact(L, L.o.h, F);
  g.pre = rows_of(L, L.pre, 2 * F);
  if ((e = pick_gemm<K_GATEUP>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.K = (int)F;
  g.N = (int)W;
  g.a = compact(L, L.o.h, F);
  g.b = wts(L, L.w_out, W, F);
  g.out = rows_of(L, L.y, W);
  return pick_gemm<K_DOWN>(g, L);
}

hipError_t launch_ffn_grad(const FfnLaunch& L) {
  const uint64_t W = L.s.W, F = L.s.F;
  hipError_t e = plan(L, kFfnRowTile);
  if (e != hipSuccess) return e;
  GemmArgs g = gemm_args(L);
  g.K = (int)W;
  g.N = (int)F;
  g.a = rows_of(L, L.dy, W);
  g.b = wts(L, L.w_out, W, F);
  g.out = compact(L, L.o.dgu, 2 * F);
  g.h = compact(L, L.o.h, F);
  g.pre = rows_of(L, L.pre, 2 * F);
  if ((e = pick_gemm<K_DHID>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.K = (int)(2 * F);
  g.N = (int)W;
  g.a = compact(L, L.o.dgu, 2 * F);
  g.b = wts(L, L.w_in, 2 * F, W);
  g.out = rows_of(L, L.dx, W);
  if ((e = pick_gemm<K_DX>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.M = (int)W;
  g.N = (int)F;
  g.a = rows_of(L, L.dy, W);
  g.b_rows = compact(L, L.o.h, F);
  g.wout = wts(L, L.dw_out, W, F);
  if ((e = pick_gemm<K_DW>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.M = (int)(2 * F);
  g.N = (int)W;
  g.a = compact(L, L.o.dgu, 2 * F);
  g.b_rows = rows_of(L, L.x, W);
  g.wout = wts(L, L.dw_in, 2 * F, W);
  return pick_gemm<K_DW>(g, L);
}

}  // namespace cc
