// Products of 8-bit integers with a scale for each row (token) and each column
// (channel), grouped by experts.
//
// A row v becomes the integers q nearest v / s (ties to even) with s = max|v| / 127
// rounded to float32, cut to [-127, 127]; q = 0 where s = 0, and s = NaN, q = 0
// where the row holds a NaN or an infinity.  A product's sums of q's are exact
// in int32; float32 takes a sum, its row's scale and its column's.

#include <algorithm>

#include "cc_ffn_tile.h"

namespace cc {
namespace {

// ------------------------------------------------------------------ rows

struct RowsArgs {
  const char* x;
  uint64_t x_stride;
  char* q;
  uint64_t q_stride, q_pitch;
  char* s;
  uint64_t s_stride;
  uint64_t rows, width;
  const int* start;
  const int2* mtab;
  const int* map;
  int per;
};

// The integer nearest u / s, ties to even.  u times the hardware reciprocal of s
// is within 2.5e-5 of the quotient (127 at most, off by the reciprocal's 2^-23 and
// the product's 2^-24 of it); where that lies closer to a half-integer, and for
// scales whose reciprocal is not normal, the quotient in float64 decides.  That
// is exact: u and (k + 1/2) s are multiples of s 2^-26 unless equal, and float64 is
// off by 2^-46.
__device__ __forceinline__ float nearest(float u, float s, float inv) {
  const float est = u * inv;
  float r = __builtin_rintf(est);
  if (__builtin_expect(!(fabsf(fabsf(est - r) - 0.5f) > 4e-5f), 0)) r = (float)__builtin_rint((double)u / (double)s);
  return __builtin_amdgcn_fmed3f(r, -127.0f, 127.0f);
}

typedef uint32_t u32_byte __attribute__((aligned(1)));

template <int V>
__device__ __forceinline__ void put_bytes(char* p, const float* q, int n, int room) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[i] |= 4 * i + j < n ? ((uint32_t)(int)q[4 * i + j] & 0xffu) << (8 * j) : 0u;
  }
  if (room >= V) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) ((u32_byte*)p)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < room) p[i] = (char)(w[i / 4] >> (8 * (i & 3)));
  }
}

// A row by WPR waves (1 or 4), R vectors a lane in registers; longer rows are
// read twice.
constexpr int kHeld = 8;
template <int DT, int WPR>
__device__ __forceinline__ void quantize_row(const char* x, uint64_t width, char* q, uint64_t pitch, float* scale,
                                             uint32_t* red) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  constexpr uint64_t STEP = (uint64_t)64 * WPR * V;
  u32x4 held[kHeld];
  uint32_t top = 0;
  auto load = [&](uint64_t c) {
    const int64_t left = (int64_t)width - (int64_t)c;
    return load_n<DT, false>(x + c * SZ, left < V ? (int)(left > 0 ? left : 0) : V);
  };
  auto larger = [&](u32x4 w) {
    float v[V];
    unpack<DT>(w, v);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = b > top ? b : top;
    }
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    held[k] = load(k * STEP + (uint64_t)tid * V);
    larger(held[k]);
  }
  for (uint64_t c = kHeld * STEP + (uint64_t)tid * V; c < width; c += STEP) larger(load(c));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) top = red[k] > top ? red[k] : top;
  }
  const bool nan = top >= 0x7f800000u;
  const float s = nan ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
  // a scale whose reciprocal is not normal: an estimate of infinity or NaN, which float64 decides
  const float inv = s >= 0x1p-100f ? __builtin_amdgcn_rcpf(s) : __uint_as_float(0x7fc00000u);
  auto put = [&](uint64_t c, u32x4 w) {
    float v[V], r[V];
    unpack<DT>(w, v);
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = nan || s == 0.0f ? 0.0f : nearest(v[i], s, inv);
    const int64_t left = (int64_t)width - (int64_t)c, room = (int64_t)pitch - (int64_t)c;
    if (room > 0) put_bytes<V>(q + c, r, (int)(left < V ? left : V), (int)(room < V ? room : V));
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k) put(k * STEP + (uint64_t)tid * V, held[k]);
  for (uint64_t c = kHeld * STEP + (uint64_t)tid * V; c < pitch; c += STEP) put(c, load(c));
  if (tid == 0) *scale = s;
}

// Plain rows: blockIdx.y the rank, 4 / WPR rows a workgroup.
template <int DT, int WPR>
__global__ __launch_bounds__(256) void k_int8_rows(RowsArgs a) {
  __shared__ uint32_t red[4];
  const uint64_t r = blockIdx.y, row = (uint64_t)blockIdx.x * (4 / WPR) + (WPR == 1 ? threadIdx.x >> 6 : 0);
  if (row >= a.rows) return;   // a whole wave, or (WPR 4) the workgroup
  quantize_row<DT, WPR>(a.x + r * a.x_stride + row * a.width * Ty<DT>::SZ, a.width, a.q + r * a.q_stride + row * a.q_pitch,
                        a.q_pitch, (float*)(a.s + r * a.s_stride) + row, red);
}

// The experts' kept rows: four workgroups a tile of 64 rows.
constexpr int kTileRows = 16;
template <int DT, int WPR>
__global__ __launch_bounds__(256) void k_int8_kept(RowsArgs a) {
  __shared__ uint32_t red[4];
  const int2 at = a.mtab[blockIdx.x / 4];
  const int stop = a.start[at.x + 1], first = at.y + (int)(blockIdx.x % 4) * kTileRows;
  const int end = first + kTileRows < stop ? first + kTileRows : stop;
  const char* x = a.x + (uint64_t)(at.x / a.per) * a.x_stride;
  for (int l = first + (WPR == 1 ? threadIdx.x >> 6 : 0); l < end; l += 4 / WPR) {
    quantize_row<DT, WPR>(x + (uint64_t)(uint32_t)a.map[l] * a.width * Ty<DT>::SZ, a.width,
                          a.q + (uint64_t)l * a.q_pitch, a.q_pitch, (float*)a.s + l, red);
    if constexpr (WPR > 1) __syncthreads();   // `red` is read
  }
}

template <int DT, int WPR>
hipError_t run_rows(const RowsArgs& a, const Int8Rows& L) {
  if (L.map) {
    CC_LAUNCH((k_int8_kept<DT, WPR>), dim3((unsigned)(4 * L.tiles)), dim3(256), 0, L.st, a);
  } else {
    const uint64_t per = 4 / WPR;
    CC_LAUNCH((k_int8_rows<DT, WPR>), dim3((unsigned)((L.rows + per - 1) / per), (unsigned)L.N), dim3(256), 0, L.st, a);
  }
  return hipGetLastError();
}
template <int DT>
hipError_t pick_rows(const RowsArgs& a, const Int8Rows& L) {
  return L.width <= (uint64_t)64 * Ty<DT>::V * kHeld ? run_rows<DT, 1>(a, L) : run_rows<DT, 4>(a, L);
}

// ------------------------------------------------------------------ products

uint64_t up256(uint64_t v) { return (v + 255) / 256 * 256; }

template <int KIND, int OT>
hipError_t run_int8(I8Args g, const Int8Launch& L, bool fast, bool vec) {
  const int cus = dev_info().cus > 0 ? dev_info().cus : 256, cols = KIND == K_GATEUP ? g.F : g.N;
  const int k = ffn_pick_tile(L.s, KIND, 0, cols, fast, cus);
  const FfnGrid tiles = ffn_grid(L.s, KIND, 0, cols, k);
  if (tiles.blocks == 0) return hipSuccess;
  g.mtiles = (int)tiles.mt;
  g.ntiles = (int)tiles.nt;
  g.mtab = (const int2*)(L.ws + L.o.plan.mtab[k]);
  const dim3 grid((unsigned)tiles.blocks);
  if (fast && vec) return launch_tile<DT_I8, KIND, true, OT>(g, k, grid, L.st);
  if (fast) return launch_tile<DT_I8, KIND, false, OT>(g, k, grid, L.st);
  if (k == 1) CC_LAUNCH((k_ffn_any<DT_I8, KIND, 128, 128, 64, 64, OT>), grid, dim3(256), 0, L.st, g);
  else CC_LAUNCH((k_ffn_any<DT_I8, KIND, 64, 64, 32, 64, OT>), grid, dim3(128), 0, L.st, g);
  return hipGetLastError();
}
template <int KIND>
hipError_t pick_int8(const I8Args& g, const Int8Launch& L, bool fast, bool vec) {
  return L.dt == DT_F32 ? run_int8<KIND, DT_F32>(g, L, fast, vec) : run_int8<KIND, DT_BF16>(g, L, fast, vec);
}

I8Args int8_args(const Int8Launch& L) {
  I8Args g = {};
  g.start = (const int*)(L.ws + L.o.plan.start);
  g.map = (const int*)(L.ws + L.o.plan.rowmap);
  g.E = L.s.E;
  g.per = L.s.E / L.s.N;
  g.F = (int)L.s.F;
  g.act = L.s.act;
  return g;
}

// `lines` rows of `cols` weights an expert
void weights_of(I8Args* g, const Side& w, const Side& s, uint64_t lines, uint64_t cols) {
  g->b = WtSide{w.base, w.stride, lines * cols, cols};
  g->sw = s.base;
  g->sw_stride = s.stride;
  g->M = (int)lines;
}

}  // namespace

hipError_t launch_int8_rows(const Int8Rows& L) {
  if (L.rows == 0) return hipSuccess;
  const RowsArgs a{L.x, L.x_stride, L.q, L.q_stride, L.q_pitch, L.s, L.s_stride, L.rows, L.width,
                   L.start, L.mtab, L.map, L.per};
  return L.dt == DT_F32 ? pick_rows<DT_F32>(a, L) : pick_rows<DT_BF16>(a, L);
}

Int8Ws int8_ws(const FfnShape& s, int block, int out_es) {
  Int8Ws o = {};
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t p = at;
    at += up256(bytes);
    return p;
  };
  o.plan.kept = take((uint64_t)s.N * s.E * 4);
  o.plan.start = take(((uint64_t)s.E + 1) * 4);
  for (int k = 0; k < kFfnTiles; ++k) o.plan.mtab[k] = take(s.mtiles[k] * 8);
  o.plan.rowmap = take(s.rows * 4);
  if (block) {
    o.xq_pitch = line_pitch(s, s.W);
    o.hq_pitch = line_pitch(s, s.F);
    o.xq = take(s.rows * o.xq_pitch);
    o.xs = take(s.rows * 4);
    o.h = take(s.rows * s.F * out_es);
    o.hq = take(s.rows * o.hq_pitch);
    o.hs = take(s.rows * 4);
  }
  o.bytes = at;
  return o;
}

hipError_t launch_int8(const Int8Launch& L) {
  const uint64_t W = L.s.W, C = L.s.F, es = elem_size(L.dt), side = (uint64_t)L.s.E * L.s.cap;
  hipError_t e = launch_ffn_plan(L.s, L.o.plan, L.ws, L.kept, L.st);
  if (e != hipSuccess) return e;
  I8Args g = int8_args(L);
  g.K = (int)W;
  g.N = (int)C;
  g.a = RowSide{L.x.base, L.x.stride, W, g.map, side * W};
  weights_of(&g, L.w_in, L.s_in, C, W);
  g.sx = L.xs.base;
  g.sx_stride = L.xs.stride;
  g.sx_map = g.map;
  g.out = RowSide{L.y.base, L.y.stride, C * es, g.map, side * C * es};
  const bool fast = L.x_ok && L.w_in_ok && side * W <= kMaxSpan && C * W <= kMaxSpan;
  return pick_int8<K_DOWN>(g, L, fast, L.y_ok);
}

hipError_t launch_int8_ffn(const Int8Launch& L) {
  const uint64_t W = L.s.W, F = L.s.F, es = elem_size(L.dt);
  hipError_t e = launch_ffn_plan(L.s, L.o.plan, L.ws, L.kept, L.st);
  if (e != hipSuccess) return e;
  I8Args g = int8_args(L);
  Int8Rows q = {};
  q.x = L.x.base; q.x_stride = L.x.stride;
  q.q = L.ws + L.o.xq; q.q_pitch = L.o.xq_pitch;
  q.s = L.ws + L.o.xs;
  q.rows = L.s.rows; q.width = W;
  q.start = g.start; q.mtab = (const int2*)(L.ws + L.o.plan.mtab[kFfnTiles - 1]); q.map = g.map;
  q.tiles = L.s.mtiles[kFfnTiles - 1]; q.per = g.per;
  q.N = 1; q.dt = L.dt; q.st = L.st;
  if ((e = launch_int8_rows(q)) != hipSuccess) return e;
  g.K = (int)W;
  g.N = (int)(2 * F);
  g.a = RowSide{q.q, 0, L.o.xq_pitch, nullptr, L.s.most * L.o.xq_pitch};
  weights_of(&g, L.w_in, L.s_in, 2 * F, W);
  g.sx = q.s;
  g.out = RowSide{L.ws + L.o.h, 0, F * es, nullptr, L.s.most * F * es};
  const bool rows_fit = L.s.most * std::max(L.o.xq_pitch, L.o.hq_pitch) <= kMaxSpan;
  if ((e = pick_int8<K_GATEUP>(g, L, L.w_in_ok && rows_fit && 2 * F * W <= kMaxSpan, F * es % 16 == 0)) != hipSuccess)
    return e;
  q.x = L.ws + L.o.h; q.x_stride = 0;
  q.q = L.ws + L.o.hq; q.q_pitch = L.o.hq_pitch;
  q.s = L.ws + L.o.hs;
  q.width = F;
  q.map = nullptr;
  if ((e = launch_int8_rows(q)) != hipSuccess) return e;
  g.K = (int)F;
  g.N = (int)W;
  g.a = RowSide{q.q, 0, L.o.hq_pitch, nullptr, L.s.most * L.o.hq_pitch};
  weights_of(&g, L.w_out, L.s_out, W, F);
  g.sx = q.s;
  g.out = RowSide{L.y.base, L.y.stride, W * es, g.map, (uint64_t)L.s.E * L.s.cap * W * es};
  return pick_int8<K_DOWN>(g, L, L.w_out_ok && rows_fit && F * W <= kMaxSpan, L.y_ok);
}

}  // namespace cc
