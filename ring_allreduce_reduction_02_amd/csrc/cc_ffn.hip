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
// products, because the matrix cores read that type.  bf16 results are so off
// by 0.0024 of their norm against 64 bits, where float32 between the products
// would leave 0.0017, the rounding of the results themselves.

#include <algorithm>

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kKBytes = 128;   // bytes of the summed axis per stage and line: a cache line
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
  int N, E;
  uint64_t cap;
  int* start;
  int2* mtab[kFfnTiles];
  int* rowmap;
};

// Workgroup e writes expert e's first compact row, its row tiles and its rows'
// places in the rank's buffer.
__global__ __launch_bounds__(256) void k_ffn_plan(PlanArgs a) {
  __shared__ uint32_t red[1 + kFfnTiles][256];
  const int e = blockIdx.x, tid = threadIdx.x, N = a.N;
  const uint32_t* kept = a.kept ? a.kept : a.v;
  uint32_t sum[1 + kFfnTiles] = {};
  for (int x = tid; x < e; x += 256) {
    uint32_t n = 0;
    for (int i = 0; i < N; ++i) n += kept[x * N + i];
    sum[0] += n;
#pragma unroll
    for (int k = 0; k < kFfnTiles; ++k) sum[1 + k] += (n + kFfnTile[k] - 1) / kFfnTile[k];
  }
#pragma unroll
  for (int k = 0; k <= kFfnTiles; ++k) red[k][tid] = sum[k];
  __syncthreads();
  for (int d = 128; d; d >>= 1) {
    if (tid < d)
#pragma unroll
      for (int k = 0; k <= kFfnTiles; ++k) red[k][tid] += red[k][tid + d];
    __syncthreads();
  }
  const uint32_t r0 = red[0][0];
  const int per = a.E / N, l = e % per;
  uint32_t at = r0;
  for (int i = 0; i < N; ++i) {
    const uint32_t n = kept[e * N + i];
    const uint32_t src = (uint32_t)(((uint64_t)i * per + l) * a.cap);
    for (uint32_t s = tid; s < n; s += 256) a.rowmap[at + s] = (int)(src + s);
    at += n;
  }
#pragma unroll
  for (int k = 0; k < kFfnTiles; ++k) {
    const uint32_t nt = (at - r0 + kFfnTile[k] - 1) / kFfnTile[k], t0 = red[1 + k][0];
    for (uint32_t t = tid; t < nt; t += 256) a.mtab[k][t0 + t] = make_int2(e, (int)(r0 + t * kFfnTile[k]));
  }
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
  uint64_t span;   // bytes that 32-bit offsets may reach: a rank's buffer, or the rows of one expert
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
  const int* map;        // compact rows' places in their rank's buffer
  WtSide wout;           // K_DW
};

// ------------------------------------------------------------------ LDS tiles

// Lines along the summed axis ("row" tiles: R lines of 128 bytes): 16-byte
// chunks permuted by the line's number, so that a fragment's lanes, one line
// each, spread over all 64 banks (256 bytes: two lines) for any 16 lines in a
// row.  (Permuted by r & 7, 8 places, 4 of the 8 cycles of every fragment read
// were conflicts.)
constexpr int kChunks = kKBytes / 16;
__device__ __forceinline__ int row_place(int r, int chunk) { return chunk ^ ((r / (16 / kChunks)) & (kChunks - 1)); }
__device__ __forceinline__ int row_at(int r, int chunk) { return r * kKBytes + (row_place(r, chunk) << 4); }

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

// Column tiles: a line per summed index, R columns long.  bf16 columns are read
// with the transposing LDS load (16 lanes give the addresses of 4 summed
// lines x 16 columns and get 4 summed elements of one column each); 32-byte
// pieces are permuted by the line's number, so that the 4 lines and 2 pieces
// (or 2 line groups) that 32 lanes read lie in different banks.  float32
// columns are read one element a lane, from two lines 4 apart at a time.
template <int DT, int R>
__device__ __forceinline__ int col_place(int k, int chunk) {   // of a 16-byte chunk in its line
  if constexpr (DT == DT_F32) return chunk ^ ((k & 4) << 1);
  else if constexpr (R * 2 >= 256) return chunk ^ ((k & 3) << 2) ^ ((k & 8) >> 2);
  else return chunk ^ ((k & 2) << 1) ^ ((k & 8) >> 2);         // 128-byte lines: two of them span the banks
}
template <int DT, int R>
__device__ __forceinline__ int col_at(int k, int col) {
  constexpr int SZ = Ty<DT>::SZ;
  static_assert(R >= 64, "a line holds every permuted place");
  return k * R * SZ + (col_place<DT, R>(k, col * SZ / 16) << 4) + col * SZ % 16;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ u32x2 lds_transposed(const char* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// The 16 bytes of a lane for unit u of 32 lines from i0: line i0 + lane % 32,
// elements of half lane / 32 of the unit.
template <int DT, bool COL, int R>
__device__ __forceinline__ u32x4 frag(const char* t, int u, int i0, int lane) {
  const int half = lane >> 5;
  if constexpr (!COL) {
    return *(const u32x4*)(t + row_at(i0 + (lane & 31), 2 * u + half));
  } else if constexpr (DT == DT_BF16) {
    const int k = 16 * u + 8 * half + ((lane & 15) >> 2), c = i0 + (lane & 16) + 4 * (lane & 3);
    const u32x2 lo = lds_transposed(t + col_at<DT, R>(k, c)), hi = lds_transposed(t + col_at<DT, R>(k + 4, c));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  } else {
    const int k = 8 * u + 4 * half, c = i0 + (lane & 31);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = *(const uint32_t*)(t + col_at<DT, R>(k + j, c));
    return u32x4{w[0], w[1], w[2], w[3]};
  }
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

// Staging of a tile of lines that start anywhere, through registers: 16-byte
// chunks (global memory takes whole vectors at any element), a line's last
// one by elements.  Row tiles: lp[r] is line r's first byte (the last line
// repeated past the end), elements [k0, K).  Column tiles: lp[k] is summed line
// k0 + k (NULL past the end: zeros), columns [c0, C).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <int DT, bool COL, int R, int NT>
struct Chunks {
  static constexpr int SZ = Ty<DT>::SZ, V = Ty<DT>::V, Q = R * kKBytes / 16 / NT;
  static constexpr int PER = COL ? R * SZ / 16 : kKBytes / 16;   // chunks per line
  u32x4 v[Q];
  __device__ __forceinline__ void load(const char* const* lp, int64_t k0, int64_t K, int64_t c0, int64_t C) {
    if (k0 + kKBytes / SZ <= K && (!COL || c0 + R <= C)) {   // whole chunks only
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int e = threadIdx.x + q * NT;
        v[q] = *(const u32x4_any*)(lp[e / PER] + ((COL ? c0 : k0) + (int64_t)(e % PER) * V) * SZ);
      }
      return;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = threadIdx.x + q * NT;
      const int64_t at = (COL ? c0 : k0) + (int64_t)(e % PER) * V, left = (COL ? C : K) - at;
      const char* p = lp[e / PER];
      v[q] = u32x4{0u, 0u, 0u, 0u};
      if (p && left >= V) {
        v[q] = *(const u32x4_any*)(p + at * SZ);
      } else if (p && left > 0) {
        float x[V] = {};
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < left) x[i] = ld1<DT>(p + (at + i) * SZ);
        v[q] = pack_row<DT>(x);   // widened and packed again: the same bits
      }
    }
  }
  __device__ __forceinline__ void store(char* t) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = threadIdx.x + q * NT;
      *(u32x4*)(t + (COL ? col_at<DT, R>(e / PER, e % PER * V) : row_at(e / PER, e % PER))) = v[q];
    }
  }
};

// ------------------------------------------------------------------ activations

enum Act { ACT_SILU = 0, ACT_GELU = 1 };

// The sigmoid s = 1 / (1 + exp(-g)) and its complement c = 1 - s.
// float32: from e = exp(-|g|), 1 / (1 + e) and e / (1 + e), off by at most 6 half
// steps (2^-24) of their value, also where they are small (with exp2 and the
// reciprocal as for bf16 the case of 8 x 2048 tokens, top-2 of 16 experts, 768 x
// 768 takes 847 us against 850 forward, 2092 against 2109 for the gradients, and
// silu is off by up to 64 half steps for |g| up to 87).
// bf16: from the hardware's exp2 and reciprocal (1 ulp each).  log2(e) is off
// by 0.23 half steps and its product with g by one, so s is off by at most
// (1.25 |g| + 6) 2^-24 of its value, 2^-17 at |g| = 87, below the 2^-8 that the
// result is rounded by; below 2^-126 it may be 0.
template <int DT>
__device__ __forceinline__ void sigmoid(float g, float& s, float& c) {
  if constexpr (DT == DT_BF16) {
    s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * g));
    c = 1.0f - s;
  } else {
    const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e), t = e * r;
    s = g >= 0.0f ? r : t;
    c = g >= 0.0f ? t : r;
  }
}
// The normal distribution function.  The argument is off by 2 half steps, which
// a small value takes g^2 times (erfc(x) falls by 2 x^2 of its value a step).
__device__ __forceinline__ float normal_cdf(float g) { return 0.5f * erfcf(-g * 0.70710678118654752f); }

// h = act(g) u
template <int DT, int V>
__device__ __forceinline__ void gate(const float* g, const float* u, int act, float* h) {
  if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s, c;
      sigmoid<DT>(g[i], s, c);
      h[i] = g[i] * s * u[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) h[i] = g[i] * normal_cdf(g[i]) * u[i];
  }
}
// dh -> dg, du and h
template <int DT, int V>
__device__ __forceinline__ void gate_grad(const float* g, const float* u, int act, const float* dh, float* dg,
                                          float* du, float* h) {
  if (act == ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float s, c;
      sigmoid<DT>(g[i], s, c);
      const float a = g[i] * s, d = s * (1.0f + g[i] * c);
      dg[i] = dh[i] * u[i] * d;
      du[i] = dh[i] * a;
      h[i] = a * u[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float c = normal_cdf(g[i]), a = g[i] * c, d = c + g[i] * expf(-0.5f * g[i] * g[i]) * 0.39894228040143268f;
      dg[i] = dh[i] * u[i] * d;
      du[i] = dh[i] * a;
      h[i] = a * u[i];
    }
  }
}

// V (4 or 8) consecutive elements of a row, n of them inside it
template <int DT, bool VEC, int V>
__device__ __forceinline__ void store_n(char* p, const float* v, int n) {
  if constexpr (VEC) {
    if (n <= 0) return;
    static_assert(V * Ty<DT>::SZ == 16, "one vector");
    stg(p, pack_row<DT>(v));   // past the caches, which the operands' tiles need
  } else if (n >= V) {
    *(u32x4_any*)p = pack_row<DT>(v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) st1<DT>(p + i * Ty<DT>::SZ, v[i]);
  }
}
// their 16 bytes, zeros past the n
template <int DT, bool VEC>
__device__ __forceinline__ u32x4 load_n(const char* p, int n) {
  constexpr int V = Ty<DT>::V;
  if constexpr (VEC) {
    return n > 0 ? *(const u32x4*)p : u32x4{0u, 0u, 0u, 0u};
  } else {
    if (n >= V) return *(const u32x4_any*)p;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < n ? ld1<DT>(p + i * Ty<DT>::SZ) : 0.0f;
    return pack_row<DT>(x);   // widened and packed again: the same bits
  }
}

// ------------------------------------------------------------------ the products

// A workgroup computes a BM x BN tile with (BM / WM) x (BN / WN) waves, each
// WM x WN of it in tiles of 32 x 32.  The weights' lines are the matrix
// instruction's first operand, so a lane ends with groups of four consecutive
// columns of one row.  K_GATEUP takes BN / 2 hidden columns: the tile's lines
// alternate 32 gate rows and the 32 up rows of the same columns, so that one
// lane holds both.
template <int KIND, int BN>
constexpr int tile_cols() {
  return KIND == K_GATEUP ? BN / 2 : BN;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

// LDS written by a wave's lanes is read by others of the same wave: its LDS
// accesses complete in program order, which the compiler has to keep.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int V>
__device__ __forceinline__ void read_row(const char* p, float* v) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const f32x4 w = *(const f32x4*)(p + 4 * i);
    v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
  }
}

struct Part {
  int e, rank, local;
  int p0, p1;   // compact rows: the tile's first, the expert's end
  int m0, n0;   // origin in the result (row products: m0 = 0, rows from p0)
  int64_t K;
};

// Workgroups go round the 8 XCDs in turn; each XCD gets one run of tiles, in
// which 4 row tiles share the columns' weights and a few columns the rows.
template <int KIND, int BM, int BN>
__device__ __forceinline__ Part tile_of(const GemmArgs& g) {
  const uint32_t n = gridDim.x, x = blockIdx.x & 7, q = n >> 3, r = n & 7;
  const uint32_t b = x * q + (x < r ? x : r) + (blockIdx.x >> 3);
  Part t;
  const uint32_t mt = (uint32_t)g.mtiles, nt = (uint32_t)g.ntiles;
  uint32_t tb = b;
  if constexpr (KIND == K_DW) {
    t.e = (int)(b / (mt * nt));
    tb = b - (uint32_t)t.e * mt * nt;
  }
  const uint32_t grp = tb / (4 * nt), in = tb - grp * 4 * nt, left = mt - grp * 4, rows = left < 4 ? left : 4;
  const uint32_t m = grp * 4 + in % rows;
  t.n0 = (int)(in / rows) * tile_cols<KIND, BN>();
  if constexpr (KIND == K_DW) {
    t.m0 = (int)m * BM;
    t.p0 = g.start[t.e];
    t.p1 = g.start[t.e + 1];
    t.K = t.p1 - t.p0;
  } else {
    const int2 at = g.mtab[m];
    t.e = at.x;
    t.p0 = at.y;
    t.p1 = g.start[t.e + 1];
    t.m0 = 0;
    t.K = g.K;
  }
  t.rank = t.e / g.per;
  t.local = t.e % g.per;
  return t;
}

// The weight row of line r of a row tile of weights, or -1.
template <int KIND>
__device__ __forceinline__ int64_t weight_line(const GemmArgs& g, const Part& t, int r) {
  if constexpr (KIND == K_GATEUP) {
    const int f = t.n0 + (r >> 6) * 32 + (r & 31);
    return f < g.F ? (int64_t)((r >> 5) & 1) * g.F + f : -1;
  } else {
    return t.n0 + r < g.N ? t.n0 + r : -1;
  }
}

// The wave's results, rows from mw and columns from nw of the tile.  A lane
// holds row lane % 32 of a 32 x 32 tile, columns 8 q + 4 (lane / 32) + 0..3 of
// it for q = 0..3.  They go through the wave's own piece of LDS (32 rows of
// WN floats, 16 bytes of padding a row so that the rows lie in different
// banks), so that a group of lanes holds a row's consecutive columns and
// stores (and, K_DHID, loads) whole runs of them.
template <int WN>
constexpr int finish_bytes() {
  return 32 * (WN * 4 + 16);
}

template <int DT, int KIND, bool VEC, int TM, int TN>
__device__ __forceinline__ void finish(const GemmArgs& g, const Part& t, const f32x16 (&acc)[TM][TN], int mw, int nw,
                                       int lane, char* lds) {
  constexpr int SZ = Ty<DT>::SZ, V = Ty<DT>::V, WN = 32 * TN, PITCH = WN * 4 + 16;
  constexpr int COLS = KIND == K_GATEUP ? WN / 2 : WN;   // result columns of the wave
  constexpr int LPR = COLS / V, RPP = 64 / LPR;          // lanes per row, rows per pass
  constexpr int PASSES = 32 / RPP;
  const int cl = (lane % LPR) * V;
  // K_GATEUP: columns alternate 32 gate and 32 up
  const int at = KIND == K_GATEUP ? (cl / 32) * 64 + cl % 32 : cl;
  const int n = t.n0 + (KIND == K_GATEUP ? nw / 2 : nw) + cl;
  const int left = (KIND == K_GATEUP ? g.F : g.N) - n;
  const int rows = KIND == K_DW ? g.M - t.m0 : t.p1 - t.p0;
  // the rows' places in the rank's buffer, 64 rows of the wave a register
  constexpr bool MAPPED = KIND != K_DW;
  int place[(TM + 1) / 2];
  if constexpr (MAPPED) {
#pragma unroll
    for (int k = 0; k < (TM + 1) / 2; ++k) {
      const int m = mw + 64 * k + lane;
      place[k] = KIND == K_GATEUP && !g.pre.base ? 0 : m < rows ? g.map[t.p0 + m] : 0;
    }
  }
  auto place_of = [&](int i, int row) { return __shfl(place[i / 2], (i & 1) * 32 + row); };
  auto mapped = [&](const RowSide& s, int place) {
    return s.base + (uint64_t)t.rank * s.rank_stride + (uint64_t)(uint32_t)place * s.pitch + (int64_t)n * SZ;
  };
  auto packed = [&](const RowSide& s, int m) { return s.base + (uint64_t)(t.p0 + m) * s.pitch + (int64_t)n * SZ; };
  // K_DHID: the pre-activations, loaded 32 rows ahead (bf16; of float32 they
  // would fill the registers)
  constexpr bool AHEAD = KIND == K_DHID && PASSES <= 4;
  u32x4 fg[2][PASSES], fu[2][PASSES];
  auto ahead = [&](int i) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int r = 0; r < PASSES; ++r) {
        const int row = r * RPP + lane / LPR;
        const char* pre = mapped(g.pre, place_of(i, row));
        const int n = mw + 32 * i + row < rows ? left : 0;
        fg[i & 1][r] = load_n<DT, VEC>(pre, n);
        fu[i & 1][r] = load_n<DT, VEC>(pre + (int64_t)g.F * SZ, n);
      }
    }
  };
  ahead(0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (i + 1 < TM) ahead(i + 1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4*)(lds + (lane & 31) * PITCH + (32 * j + 8 * q + 4 * (lane >> 5)) * 4) =
            f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < PASSES; ++r) {
      const int row = r * RPP + lane / LPR, m = mw + 32 * i + row;
      int at_row = 0;
      if constexpr (MAPPED) at_row = place_of(i, row);
      if (m >= rows) continue;
      float v[V];
      read_row<V>(lds + row * PITCH + at * 4, v);
      if constexpr (KIND == K_DW) {
        store_n<DT, VEC, V>(wt_ptr(g.wout, t.rank, t.local) + (uint64_t)(t.m0 + m) * g.wout.pitch + (int64_t)n * SZ, v,
                            left);
      } else if constexpr (KIND == K_DOWN || KIND == K_DX) {
        store_n<DT, VEC, V>(mapped(g.out, at_row), v, left);
      } else if constexpr (KIND == K_GATEUP) {
        float up[V], h[V];
        read_row<V>(lds + row * PITCH + (at + 32) * 4, up);
        gate<DT, V>(v, up, g.act, h);
        store_n<DT, VEC, V>(packed(g.out, m), h, left);
        if (g.pre.base) {
          char* pre = mapped(g.pre, at_row);
          store_n<DT, VEC, V>(pre, v, left);
          store_n<DT, VEC, V>(pre + (int64_t)g.F * SZ, up, left);
        }
      } else {   // K_DHID
        float gt[V], up[V], dg[V], du[V], h[V];
        if constexpr (AHEAD) {
          unpack<DT>(fg[i & 1][r], gt);
          unpack<DT>(fu[i & 1][r], up);
        } else {
          const char* pre = mapped(g.pre, at_row);
          unpack<DT>(load_n<DT, VEC>(pre, left), gt);
          unpack<DT>(load_n<DT, VEC>(pre + (int64_t)g.F * SZ, left), up);
        }
        gate_grad<DT, V>(gt, up, g.act, v, dg, du, h);
        char* o = packed(g.out, m);
        store_n<DT, VEC, V>(o, dg, left);
        store_n<DT, VEC, V>(o + (int64_t)g.F * SZ, du, left);
        store_n<DT, VEC, V>(packed(g.h, m), h, left);
      }
    }
    wave_lds_sync();
  }
}

// One stage's products of a wave: the next unit's fragments are read while the
// matrix instructions of the last ones run.
template <int DT, bool ACOL, bool BCOL, int BM, int BN, int TM, int TN>
__device__ __forceinline__ void multiply(const char* ta, const char* tb, f32x16 (&acc)[TM][TN], int mw, int nw,
                                         int lane) {
  u32x4 fa[2][TM], fb[2][TN];
  auto read = [&](int u) {
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[u & 1][j] = frag<DT, BCOL, BN>(tb, u, nw + 32 * j, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[u & 1][i] = frag<DT, ACOL, BM>(ta, u, mw + 32 * i, lane);
  };
  read(0);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (u + 1 < kUnits) read(u + 1);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[u & 1][j], fa[u & 1][i], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);   // keeps at most two units' fragments in registers
  }
}

template <int TM, int TN>
__device__ __forceinline__ void clear(f32x16 (&acc)[TM][TN]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
}

// Any alignment: tiles staged through registers, the next stage's on their way
// while this one's products run.  2 x 333 tokens, top-2 of 6 experts, 515 x 331
// float32: 32 and 20 us.  Its 506 and 414 waves leave half of the 1024 SIMDs idle,
// and a wave spends half of its time, 14 of 28 us, in matrix instructions, the
// rest on the latency of 17 and 11 stages; element by element they took 54 and 35.
template <int DT, int KIND, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_ffn_any(GemmArgs g) {
  constexpr int NT = 64 * (BM / WM) * (BN / WN);
  constexpr int BK = kKBytes / Ty<DT>::SZ;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr bool ACOL = KIND == K_DW, BCOL = KIND == K_DHID || KIND == K_DX || KIND == K_DW;
  __shared__ __attribute__((aligned(16))) char ta[BM * kKBytes];
  __shared__ __attribute__((aligned(16))) char tb[BN * kKBytes];
  __shared__ __attribute__((aligned(16))) char fin[(NT / 64) * finish_bytes<WN>()];
  // lines of the tile, or (column tiles) of a stage's summed lines
  __shared__ const char* la[ACOL ? BK : BM];
  __shared__ const char* lb[BCOL ? BK : BN];
  static_assert(BK <= NT, "a thread sets a summed line");

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int mw = (wave % (BM / WM)) * WM, nw = (wave / (BM / WM)) * WN;
  const Part t = tile_of<KIND, BM, BN>(g);
  if constexpr (!ACOL)
    for (int r = tid; r < BM; r += NT) la[r] = row_ptr(g.a, t.rank, t.p0 + r < t.p1 ? t.p0 + r : t.p1 - 1);
  if constexpr (!BCOL) {
    const char* w = wt_ptr(g.b, t.rank, t.local);
    for (int r = tid; r < BN; r += NT) {
      const int64_t row = weight_line<KIND>(g, t, r);
      lb[r] = w + (row >= 0 ? row : 0) * (int64_t)g.b.pitch;
    }
  }
  auto summed_lines = [&](int64_t k0) {
    if (tid < BK) {
      const int64_t k = k0 + tid;
      if constexpr (ACOL) la[tid] = k < t.K ? row_ptr(g.a, t.rank, (int)(t.p0 + k)) : nullptr;
      if constexpr (KIND == K_DW) lb[tid] = k < t.K ? row_ptr(g.b_rows, t.rank, (int)(t.p0 + k)) : nullptr;
      else if constexpr (BCOL) lb[tid] = k < t.K ? wt_ptr(g.b, t.rank, t.local) + k * (int64_t)g.b.pitch : nullptr;
    }
  };
  Chunks<DT, ACOL, BM, NT> ea;
  Chunks<DT, BCOL, BN, NT> eb;
  f32x16 acc[TM][TN];
  clear(acc);
  summed_lines(0);
  __syncthreads();
  if (t.K > 0) {
    ea.load(la, 0, t.K, t.m0, g.M);
    eb.load(lb, 0, t.K, t.n0, g.N);
  }
  for (int64_t k0 = 0; k0 < t.K; k0 += BK) {
    __syncthreads();   // the last stage's tiles and lines are read
    ea.store(ta);
    eb.store(tb);
    summed_lines(k0 + BK);
    __syncthreads();
    if (k0 + BK < t.K) {
      ea.load(la, k0 + BK, t.K, t.m0, g.M);
      eb.load(lb, k0 + BK, t.K, t.n0, g.N);
    }
    multiply<DT, ACOL, BCOL, BM, BN>(ta, tb, acc, mw, nw, lane);
  }
  finish<DT, KIND, false>(g, t, acc, mw, nw, lane, fin + wave * finish_bytes<WN>());
}

// ---- aligned rows: tiles come by direct loads to LDS, 16 bytes a lane.  Buffer
// loads, because the compiler counts them apart from the LDS reads around
// them (behind a global load to LDS it waits for all LDS reads before it uses
// any).  An offset outside the buffer (kOutside) reads as zeros.

constexpr uint32_t kOutside = 0xfffffff0u;
static_assert(kMaxSpan <= kOutside, "an offset inside a buffer is not kOutside");

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const char* base, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)bytes, 0x00020000);
}

__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t uniform_off, char* to) {
  typedef __attribute__((address_space(3))) void lv;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lv*)to, 16, (int)off, (int)uniform_off, 0, 0);
}

// until at most N of the wave's loads are under way, and none of its LDS reads
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}

// One operand's tile of R lines, loaded by NW waves: a wave's load fills 1 KiB
// of LDS in lane order, so the lane fetches the chunk that the permuted layout
// has at its place.  Lines and columns outside the matrix repeat the last
// one (their results are not stored); summed elements outside read zeros.
template <int DT, bool COL, int R, int NW>
struct Loader {
  static constexpr int SZ = Ty<DT>::SZ, BK = kKBytes / SZ;
  static constexpr int Q = R * kKBytes / 1024 / NW;           // loads per wave and stage
  static constexpr int LANES = COL ? R * SZ / 16 : kChunks;   // lanes per line
  __amdgpu_buffer_rsrc_t buf;
  uint32_t off[Q];      // this lane's bytes at stage 0 (summed lines by a row map: the column chunk's)
  int last[Q];          // stages in which they lie inside the summed elements
  uint32_t step;        // bytes per stage

  __device__ __forceinline__ static int line_of(int wave, int q, int lane) {
    return (wave * Q + q) * (64 / LANES) + lane / LANES;
  }
  // chunk of a row tile's line that lies at this lane's place
  __device__ __forceinline__ static int chunk_of(int wave, int q, int lane) {
    return row_place(line_of(wave, q, lane), lane % kChunks);
  }
  // row tiles: off[] are the lines' first bytes
  __device__ __forceinline__ void lines(int wave, int lane, int K) {
    step = kKBytes;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int c = 16 * chunk_of(wave, q, lane);
      off[q] += c;
      last[q] = (int)(((int64_t)K * SZ - c + kKBytes - 1) / kKBytes);
    }
  }
  // column tiles: off[] become the column chunks' bytes, columns c0.. of C (the
  // padding of a copied row's last chunk among them: no result of it is stored)
  __device__ __forceinline__ void columns(int wave, int lane, int c0, int C, int K) {
    const int end = ((C - c0) * SZ + 15) / 16 * 16 - 16;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int k = line_of(wave, q, lane), c = 16 * col_place<DT, R>(k, lane % LANES);   // its own inverse
      off[q] = (uint32_t)(c0 * SZ + (c < end ? c : end));
      last[q] = (K - k + BK - 1) / BK;
    }
  }
  // load q of stage s (zeros past the end, s_end the last stage inside)
  __device__ __forceinline__ void issue(char* t, int wave, int q, int s, int s_end) const {
    const uint32_t at = (uint32_t)(s < s_end ? s : s_end) * step;   // never past the buffer by itself
    load_lds(buf, s < last[q] ? off[q] : kOutside, at, t + (wave * Q + q) * 1024);
  }
  // the same with the summed line's row
  __device__ __forceinline__ void issue_row(char* t, int wave, int q, int s, uint32_t pitch, int row) const {
    load_lds(buf, s < last[q] ? (uint32_t)row * pitch + off[q] : kOutside, 0, t + (wave * Q + q) * 1024);
  }
  // the rows of stage s: from the map, or counted from the expert's first
  __device__ __forceinline__ void rows(int (&idx)[Q], const int* map, int p0, int K, int wave, int lane,
                                       int s) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      int k = s * BK + line_of(wave, q, lane);
      k = k < K ? k : K - 1;
      idx[q] = map ? map[p0 + k] : k;
    }
  }
};

// The buffer that a row operand's offsets count in: the rank's, or for compact
// rows the part from row p0 on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const RowSide& s, int rank, int p0) {
  return buffer_of(s.map ? s.base + (uint64_t)rank * s.rank_stride : s.base + (uint64_t)p0 * s.pitch, s.span);
}

// Two stages of whole 128-byte lines are in LDS (128 KiB of a 256 x 256 tile),
// one barrier a stage.  Measured on 8 x 4096 tokens, top-2 of 16 experts,
// 2048 x 2048 bf16 (60.7k rows): gate and up 1.04 ms (980 TFLOP/s), down 0.48-0.51
// (1000-1060), hidden gradient 0.65 (780; it reads and writes 1.5 GB more), row
// gradient 0.87 (1170), weight gradients 0.54 and 1.10 (930).  The matrix units
// are busy 57, 60, 40, 64 and 49-51% of the cycles, at 1.6, 1.6, 1.9, 1.8 and 1.9
// GHz: the card lowers its clock under this load.  With the loads left out a stage took 1.36 us, with loads that
// hit the L2 1.58, as it is 1.95.
// What else was tried there: four stages of 64-byte lines (twice the cache
// requests: 10% slower), 128 x 128 tiles two to a unit (10-25% slower), four
// waves of 128 x 128 (faster per stage, slower results), loads of later
// stages' lines into the L2 ahead (within 2%), row groups of 8 and 16 (0-5%
// slower).
template <int DT, int KIND, bool VEC, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN)) void k_ffn_tile(GemmArgs g) {
  constexpr int NW = (BM / WM) * (BN / WN);
  constexpr int SZ = Ty<DT>::SZ, BK = kKBytes / SZ;
  constexpr int TM = WM / 32, TN = WN / 32;
  constexpr bool ACOL = KIND == K_DW, BCOL = KIND == K_DHID || KIND == K_DX || KIND == K_DW;
  // separate arrays: the compiler then knows which of them a load to LDS fills,
  // and waits for no other
  __shared__ __attribute__((aligned(16))) char t0[(BM + BN) * kKBytes], t1[(BM + BN) * kKBytes];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mw = (wave % (BM / WM)) * WM, nw = (wave / (BM / WM)) * WN;
  const Part t = tile_of<KIND, BM, BN>(g);
  typedef Loader<DT, ACOL, BM, NW> LA;
  typedef Loader<DT, BCOL, BN, NW> LB;
  LA la;
  LB lb;
  const int K = (int)t.K;
  int ia[LA::Q], ib[LB::Q];
  la.buf = rows_buffer(g.a, t.rank, t.p0);
  if constexpr (!ACOL) {
#pragma unroll
    for (int q = 0; q < LA::Q; ++q) {
      int r = LA::line_of(wave, q, lane);
      r = t.p0 + r < t.p1 ? r : t.p1 - 1 - t.p0;
      la.off[q] = (uint32_t)(g.a.map ? g.a.map[t.p0 + r] : r) * (uint32_t)g.a.pitch;
    }
    la.lines(wave, lane, K);
  } else {
    la.columns(wave, lane, t.m0, g.M, K);
  }
  if constexpr (KIND == K_DW) {
    lb.buf = rows_buffer(g.b_rows, t.rank, t.p0);
    lb.columns(wave, lane, t.n0, g.N, K);
  } else {
    lb.buf = buffer_of(wt_ptr(g.b, t.rank, t.local), g.b.expert_stride);
    if constexpr (BCOL) {
      lb.columns(wave, lane, t.n0, g.N, K);
      lb.step = (uint32_t)BK * (uint32_t)g.b.pitch;
#pragma unroll
      for (int q = 0; q < LB::Q; ++q) lb.off[q] += (uint32_t)LB::line_of(wave, q, lane) * (uint32_t)g.b.pitch;
    } else {
#pragma unroll
      for (int q = 0; q < LB::Q; ++q) {
        const int64_t row = weight_line<KIND>(g, t, LB::line_of(wave, q, lane));
        lb.off[q] = (uint32_t)(row >= 0 ? row : 0) * (uint32_t)g.b.pitch;
      }
      lb.lines(wave, lane, K);
    }
  }

  f32x16 acc[TM][TN];
  clear(acc);
  const int S = (K + 2 * BK - 1) / (2 * BK) * 2;                // an odd last stage is zeros
  const int s_end = (K + BK - 1) / BK - 1;                      // the last stage with elements
  auto issue_a = [&](char* to, int s, int q) {
    if constexpr (KIND == K_DW) la.issue_row(to, wave, q, s, (uint32_t)g.a.pitch, ia[q]);
    else la.issue(to, wave, q, s, s_end);
  };
  auto issue_b = [&](char* to, int s, int q) {
    if constexpr (KIND == K_DW) lb.issue_row(to + BM * kKBytes, wave, q, s, (uint32_t)g.b_rows.pitch, ib[q]);
    else lb.issue(to + BM * kKBytes, wave, q, s, s_end);
  };
  auto rows = [&](int s) {
    if constexpr (KIND == K_DW) {
      la.rows(ia, g.a.map, t.p0, K, wave, lane, s);
      lb.rows(ib, g.b_rows.map, t.p0, K, wave, lane, s);
    }
  };
  u32x4 fa[2][TM], fb[2][TN];
  auto read = [&](const char* from, int u) {
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[u & 1][j] = frag<DT, BCOL, BN>(from + BM * kKBytes, u, nw + 32 * j, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[u & 1][i] = frag<DT, ACOL, BM>(from, u, mw + 32 * i, lane);
  };
  // unit u's matrix instructions; before each TN of them fragments of unit ru
  // of the stage rd are read, and after them one of TM calls between
  auto multiply_unit = [&](int u, const char* rd, int ru, auto between) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = i; j < TN; j += TM)
        fb[(u + 1) & 1][j] = frag<DT, BCOL, BN>(rd + BM * kKBytes, ru, nw + 32 * j, lane);
      fa[(u + 1) & 1][i] = frag<DT, ACOL, BM>(rd, ru, mw + 32 * i, lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mma<DT>(fb[u & 1][j], fa[u & 1][i], acc[i][j]);
      between(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto nothing = [](int) {};
  // Stage s.  The next unit's fragments are read between the matrix instructions
  // of the last ones.  Before the last unit's, every wave has read all of
  // this stage and its loads of the next one have come (three units or more
  // after they were sent): the barrier then frees this stage's LDS for the
  // stage after the next, whose loads go out between the matrix instructions
  // of this unit and the next one, and the next stage's first fragments are
  // read.
  auto stage = [&](char* now, char* next, int s) {
#pragma unroll
    for (int u = 0; u + 1 < kUnits; ++u) {
      if (u == 0) {
        multiply_unit(u, now, u + 1, [&](int i) {
#pragma unroll
          for (int q = i; q < LB::Q; q += TM) issue_b(next, s + 1, q);
        });
        rows(s + 2);
      } else {
        multiply_unit(u, now, u + 1, nothing);
      }
    }
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    multiply_unit(kUnits - 1, next, 0, [&](int i) {
#pragma unroll
      for (int q = i; q < LA::Q; q += TM) issue_a(now, s + 2, q);
    });
  };
  if (S) {
    // stage 0, and of stage 1 what a stage sends before its first unit
    rows(0);
#pragma unroll
    for (int q = 0; q < LA::Q; ++q) issue_a(t0, 0, q);
#pragma unroll
    for (int q = 0; q < LB::Q; ++q) issue_b(t0, 0, q);
    rows(1);
    wait_loads<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < LA::Q; ++q) issue_a(t1, 1, q);
    read(t0, 0);
  }
  for (int s = 0; s < S; s += 2) {
    stage(t0, t1, s);
    stage(t1, t0, s + 1);
  }
  wait_loads<0>();   // the zeros of stages past the end also land in LDS
  __syncthreads();   // other waves may still read the last tiles
  constexpr int PER = (BM + BN) * kKBytes / finish_bytes<WN>();   // waves that one stage's LDS serves
  static_assert(NW <= 2 * PER, "every wave has its piece");
  char* fin = wave < PER ? t0 : t1;
  finish<DT, KIND, VEC>(g, t, acc, mw, nw, lane, fin + (wave % PER) * finish_bytes<WN>());
}

// ------------------------------------------------------------------ aligned copies

uint64_t up256(uint64_t v) { return (v + 255) / 256 * 256; }

struct CopyArgs {
  const int* start;
  const int2* mtab;      // row tiles of 64
  const int* map;
  int per;
  struct {
    const char* from;
    uint64_t rank_stride;
    uint64_t lines, each;          // weights: lines in all, and of an expert; rows: tiles, 0
    char* to;
    uint64_t cols, pitch;
  } job[4];
  char* h;               // padding of the rows between the products
  char* dgu;
  uint64_t F, h_pitch, dgu_pitch;
};

constexpr int kCopyLines = kFfnTile[kFfnTiles - 1];

// Workgroup x of job y copies 64 lines.  Bound by memory: the weights of 16
// experts of 2047 x 2047 bf16 and 60.7k rows, 1.3 GB in and out, 300 us, 4.3 TB/s
// (350 us with one load of a lane under way).
template <int DT>
__global__ __launch_bounds__(256) void k_ffn_copy(CopyArgs a) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const auto& j = a.job[blockIdx.y];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool rows = j.each == 0;
  uint64_t first, end;
  const char* from = j.from;
  if (rows) {
    if (blockIdx.x >= j.lines) return;
    const int2 at = a.mtab[blockIdx.x];
    first = (uint64_t)at.y;
    const uint64_t stop = (uint64_t)a.start[at.x + 1];
    end = first + kCopyLines < stop ? first + kCopyLines : stop;
    from += (uint64_t)(at.x / a.per) * j.rank_stride;
  } else {
    first = (uint64_t)blockIdx.x * kCopyLines;
    if (first >= j.lines) return;
    end = first + kCopyLines < j.lines ? first + kCopyLines : j.lines;
  }
  for (uint64_t l = first + wave; l < end; l += 4) {
    const char* p;
    if (rows) {
      p = from + (uint64_t)a.map[l] * j.cols * SZ;
    } else {
      const uint64_t e = l / j.each, r = e / a.per;
      if (a.start[e] == a.start[e + 1]) continue;   // no rows: never read
      p = from + r * j.rank_stride + (l - r * a.per * j.each) * j.cols * SZ;
    }
    char* o = j.to + l * j.pitch;
    for (uint64_t c = (uint64_t)lane * V; c * SZ < j.pitch; c += 4 * 64 * V) {   // four loads under way
      u32x4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t left = (int64_t)j.cols - (int64_t)(c + q * 64 * V);
        w[q] = load_n<DT, false>(p + (c + q * 64 * V) * SZ, left < V ? (int)(left > 0 ? left : 0) : V);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if ((c + q * 64 * V) * SZ < j.pitch) *(u32x4*)(o + (c + q * 64 * V) * SZ) = w[q];
    }
    if (rows && blockIdx.y == 0) {
      for (uint64_t c = a.F * SZ + lane * SZ; c < a.h_pitch; c += 64 * SZ) st1<DT>(a.h + l * a.h_pitch + c, 0.0f);
      if (a.dgu)
        for (uint64_t c = 2 * a.F * SZ + lane * SZ; c < a.dgu_pitch; c += 64 * SZ)
          st1<DT>(a.dgu + l * a.dgu_pitch + c, 0.0f);
    }
  }
}

template <int DT, int KIND, bool VEC>
hipError_t launch_tile(const GemmArgs& g, int k, dim3 grid, hipStream_t st) {
  if (k == 0) CC_LAUNCH((k_ffn_tile<DT, KIND, VEC, 256, 256, 128, 64>), grid, dim3(512), 0, st, g);
  else if (k == 1) CC_LAUNCH((k_ffn_tile<DT, KIND, VEC, 128, 128, 64, 64>), grid, dim3(256), 0, st, g);
  else CC_LAUNCH((k_ffn_tile<DT, KIND, VEC, 64, 64, 32, 64>), grid, dim3(128), 0, st, g);
  return hipGetLastError();
}

template <int DT, int KIND>
hipError_t run_gemm(GemmArgs g, const FfnLaunch& L) {
  const bool fast = ffn_tiled(L.s, L.o.copied, L.vec_ok);
  const int cus = dev_info().cus > 0 ? dev_info().cus : 256, cols = KIND == K_GATEUP ? g.F : g.N;
  const int k = ffn_pick_tile(L.s, KIND, g.M, cols, fast, cus);
  const FfnGrid tiles = ffn_grid(L.s, KIND, g.M, cols, k);
  const uint64_t blocks = tiles.blocks;
  if (blocks == 0) return hipSuccess;
  g.mtiles = (int)tiles.mt;
  g.ntiles = (int)tiles.nt;
  g.mtab = (const int2*)(L.ws + L.o.mtab[k]);
  const dim3 grid((unsigned)blocks);
  if (fast && L.o.copied) return launch_tile<DT, KIND, false>(g, k, grid, L.st);   // results start anywhere
  if (fast) return launch_tile<DT, KIND, true>(g, k, grid, L.st);
  if (k == 1) CC_LAUNCH((k_ffn_any<DT, KIND, 128, 128, 64, 64>), grid, dim3(256), 0, L.st, g);
  else CC_LAUNCH((k_ffn_any<DT, KIND, 64, 64, 32, 64>), grid, dim3(128), 0, L.st, g);
  return hipGetLastError();
}

template <int KIND>
hipError_t pick_gemm(const GemmArgs& g, const FfnLaunch& L) {
  return L.s.dt == DT_F32 ? run_gemm<DT_F32, KIND>(g, L) : run_gemm<DT_BF16, KIND>(g, L);
}

// the tables, from the counts in the launch's arguments or (many) in memory
hipError_t plan(const FfnLaunch& L) {
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
  a.N = L.s.N; a.E = L.s.E; a.cap = L.s.cap;
  a.start = (int*)(L.ws + L.o.start);
  for (int k = 0; k < kFfnTiles; ++k) a.mtab[k] = (int2*)(L.ws + L.o.mtab[k]);
  a.rowmap = (int*)(L.ws + L.o.rowmap);
  CC_LAUNCH(k_ffn_plan, dim3((unsigned)L.s.E), dim3(256), 0, L.st, a);
  return hipGetLastError();
}

GemmArgs gemm_args(const FfnLaunch& L) {
  GemmArgs g = {};
  g.start = (const int*)(L.ws + L.o.start);
  g.map = (const int*)(L.ws + L.o.rowmap);
  g.E = L.s.E;
  g.per = L.s.E / L.s.N;
  g.F = (int)L.s.F;
  g.act = L.s.act;
  return g;
}

RowSide rows_of(const FfnLaunch& L, const Side& s, uint64_t cols) {
  const uint64_t pitch = cols * elem_size(L.s.dt);
  return RowSide{s.base, s.stride, pitch, (const int*)(L.ws + L.o.rowmap), (uint64_t)L.s.E * L.s.cap * pitch};
}
RowSide compact(const FfnLaunch& L, uint64_t off, uint64_t cols) {
  const uint64_t pitch = L.o.copied ? line_pitch(L.s, cols) : cols * elem_size(L.s.dt);
  return RowSide{L.ws + off, 0, pitch, nullptr, L.s.most * pitch};
}
WtSide wts(const FfnLaunch& L, const Side& s, uint64_t r, uint64_t c) {
  const uint64_t es = elem_size(L.s.dt);
  return WtSide{s.base, s.stride, r * c * es, c * es};
}

// the operands as the products read them: the caller's, or their copies
RowSide rows_in(const FfnLaunch& L, const Side& s, uint64_t copy) {
  return L.o.copied ? compact(L, copy, L.s.W) : rows_of(L, s, L.s.W);
}
WtSide wts_in(const FfnLaunch& L, const Side& s, uint64_t copy, uint64_t r, uint64_t c) {
  if (!L.o.copied) return wts(L, s, r, c);
  const uint64_t p = line_pitch(L.s, c);
  return WtSide{L.ws + copy, (uint64_t)(L.s.E / L.s.N) * r * p, r * p, p};
}

hipError_t copy_operands(const FfnLaunch& L, int grad) {
  const uint64_t W = L.s.W, F = L.s.F, n = L.s.E, tiles = L.s.mtiles[kFfnTiles - 1];
  CopyArgs a = {};
  a.start = (const int*)(L.ws + L.o.start);
  a.mtab = (const int2*)(L.ws + L.o.mtab[kFfnTiles - 1]);
  a.map = (const int*)(L.ws + L.o.rowmap);
  a.per = L.s.E / L.s.N;
  a.job[0] = {L.x.base, L.x.stride, tiles, 0, L.ws + L.o.x, W, line_pitch(L.s, W)};
  a.job[1] = {L.w_in.base, L.w_in.stride, n * 2 * F, 2 * F, L.ws + L.o.w_in, W, line_pitch(L.s, W)};
  a.job[2] = {L.w_out.base, L.w_out.stride, n * W, W, L.ws + L.o.w_out, F, line_pitch(L.s, F)};
  if (grad) a.job[3] = {L.dy.base, L.dy.stride, tiles, 0, L.ws + L.o.dy, W, line_pitch(L.s, W)};
  a.h = L.ws + L.o.h;
  a.dgu = grad ? L.ws + L.o.dgu : nullptr;
  a.F = F;
  a.h_pitch = line_pitch(L.s, F);
  a.dgu_pitch = line_pitch(L.s, 2 * F);
  const uint64_t blocks = std::max(tiles, (n * std::max(2 * F, W) + kCopyLines - 1) / kCopyLines);
  const dim3 grid((unsigned)blocks, grad ? 4 : 3), blk(256);
  if (L.s.dt == DT_F32) CC_LAUNCH(k_ffn_copy<DT_F32>, grid, blk, 0, L.st, a);
  else CC_LAUNCH(k_ffn_copy<DT_BF16>, grid, blk, 0, L.st, a);
  return hipGetLastError();
}

hipError_t prepare(const FfnLaunch& L, int grad) {
  const hipError_t e = plan(L);
  return e == hipSuccess && L.o.copied ? copy_operands(L, grad) : e;
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
  for (int k = 0; k < kFfnTiles; ++k) o.mtab[k] = take(s.mtiles[k] * 8);
  o.rowmap = take(s.rows * 4);
  o.copied = ffn_copied(s, grad);
  o.x = o.dy = o.w_in = o.w_out = 0;
  if (o.copied) {
    o.h = take(s.rows * line_pitch(s, s.F));
    o.dgu = grad ? take(s.rows * line_pitch(s, 2 * s.F)) : 0;
    o.x = take(s.rows * line_pitch(s, s.W));
    if (grad) o.dy = take(s.rows * line_pitch(s, s.W));
    o.w_in = take((uint64_t)s.E * 2 * s.F * line_pitch(s, s.W));
    o.w_out = take((uint64_t)s.E * s.W * line_pitch(s, s.F));
  } else {
    o.h = take(s.rows * s.F * es);
    o.dgu = grad ? take(s.rows * 2 * s.F * es) : 0;
  }
  o.bytes = at;
  return o;
}

hipError_t launch_ffn(const FfnLaunch& L) {
  const uint64_t W = L.s.W, F = L.s.F;
  hipError_t e = prepare(L, 0);
  if (e != hipSuccess) return e;
  GemmArgs g = gemm_args(L);
  g.K = (int)W;
  g.N = (int)(2 * F);
  g.a = rows_in(L, L.x, L.o.x);
  g.b = wts_in(L, L.w_in, L.o.w_in, 2 * F, W);
  g.out = compact(L, L.o.h, F);
  g.pre = rows_of(L, L.pre, 2 * F);
  if ((e = pick_gemm<K_GATEUP>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.K = (int)F;
  g.N = (int)W;
  g.a = compact(L, L.o.h, F);
  g.b = wts_in(L, L.w_out, L.o.w_out, W, F);
  g.out = rows_of(L, L.y, W);
  return pick_gemm<K_DOWN>(g, L);
}

hipError_t launch_ffn_grad(const FfnLaunch& L) {
  const uint64_t W = L.s.W, F = L.s.F;
  hipError_t e = prepare(L, 1);
  if (e != hipSuccess) return e;
  GemmArgs g = gemm_args(L);
  g.K = (int)W;
  g.N = (int)F;
  g.a = rows_in(L, L.dy, L.o.dy);
  g.b = wts_in(L, L.w_out, L.o.w_out, W, F);
  g.out = compact(L, L.o.dgu, 2 * F);
  g.h = compact(L, L.o.h, F);
  g.pre = rows_of(L, L.pre, 2 * F);
  if ((e = pick_gemm<K_DHID>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.K = (int)(2 * F);
  g.N = (int)W;
  g.a = compact(L, L.o.dgu, 2 * F);
  g.b = wts_in(L, L.w_in, L.o.w_in, 2 * F, W);
  g.out = rows_of(L, L.dx, W);
  if ((e = pick_gemm<K_DX>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.M = (int)W;
  g.N = (int)F;
  g.a = rows_in(L, L.dy, L.o.dy);
  g.b_rows = compact(L, L.o.h, F);
  g.wout = wts(L, L.dw_out, W, F);
  if ((e = pick_gemm<K_DW>(g, L)) != hipSuccess) return e;
  g = gemm_args(L);
  g.M = (int)(2 * F);
  g.N = (int)W;
  g.a = compact(L, L.o.dgu, 2 * F);
  g.b_rows = rows_in(L, L.x, L.o.x);
  g.wout = wts(L, L.dw_in, 2 * F, W);
  return pick_gemm<K_DW>(g, L);
}

}  // namespace cc
