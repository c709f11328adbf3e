// Products of 8-bit integers with a scale for each row (token) and each column
// (channel), grouped by experts.
//
// A row v becomes the integers q nearest v / s (ties to even) with s = max|v| / 127
// rounded to float32 (or the product with float32(1 / 127), where the caller wants
// the rows that such code keeps), cut to [-127, 127]; q = 0 where s = 0, and s = NaN,
// q = 0 where the row holds a NaN or an infinity.  A product's sums of q's are exact
// in int32; float32 takes a sum, its row's scale and its column's.

#include <algorithm>

#include "cc_ffn_tile.h"
#include "cc_wave.h"

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
  uint64_t row0;         // of a launch
  int product;           // the scale is a product
};

// The integer nearest |u| / s, ties to even, for s of 2^-100 and more: k or k + 1,
// by the sign of |u| - (k + 1/2) s, which one rounding of a fused multiply-add
// keeps (the difference is 0 or a multiple of 2^-26 s).  `est` lies within 1/4 of
// the quotient.
__device__ __forceinline__ float nearest(float u, float s, float est) {
  const float k = __builtin_truncf(est), rem = __builtin_fmaf(-(k + 0.5f), s, u);
  const int up = (int)(rem > 0.0f) | ((int)(rem == 0.0f) & (int)k & 1);
  return k + (float)up;
}

typedef uint32_t u32_byte __attribute__((aligned(1)));
typedef uint32_t u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// the largest magnitude's bits so far, of a type's own width
template <int DT>
struct Top;
template <>
struct Top<DT_F32> {
  uint32_t m = 0;
  __device__ __forceinline__ void take(u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = w[i] & 0x7fffffffu;
      m = b > m ? b : m;
    }
  }
  __device__ __forceinline__ uint32_t bits() const { return m; }
};
template <>
struct Top<DT_BF16> {
  u16x2 m = {0, 0};
  __device__ __forceinline__ void take(u32x4 w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
  }
  __device__ __forceinline__ uint32_t bits() const { return (uint32_t)(m.x > m.y ? m.x : m.y) << 16; }
};

// V quantised values, in V / 4 words.  u times the hardware reciprocal of s is within
// 2.3e-5 of the quotient (127 at most; the reciprocal is off by 2^-23 and the product
// by 2^-24 of it), so that both round to the same integer unless the product
// lies closer than that to a half-integer: those are decided by `nearest`.
// The product plus 1.5 2^23 is that integer, in its lowest bits.
template <int DT, int V>
__device__ __forceinline__ void quantized(u32x4 in, float s, float inv, uint32_t* w) {
  constexpr float kMagic = 12582912.0f;
  float v[V], far = 0.0f;
  uint32_t b[V];
  unpack<DT>(in, v);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float est = v[i] * inv, t = est + kMagic;
    far = fmaxf(far, fabsf(est - (t - kMagic)));
    b[i] = __float_as_uint(t);
  }
  if (__builtin_expect(far > 0.499975f, 0)) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float q = nearest(fabsf(v[i]), s, fabsf(v[i] * inv));
      b[i] = __float_as_uint((v[i] < 0.0f ? -q : q) + kMagic);
    }
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    w[i] = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400u) |
           __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x04000c0cu);
}
// The same for scales below 2^-100, whose reciprocal need not be a number: by the
// quotient in float64, which is exact enough (off by 2^-46, and not closer than
// 2^-26 to a half-integer it does not equal).
template <int DT, int V>
__device__ __forceinline__ void quantized_small(u32x4 in, float s, uint32_t* w) {
  float v[V];
  unpack<DT>(in, v);
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double q = __builtin_rint((double)v[4 * i + j] / (double)s);
      w[i] |= ((uint32_t)(int)(q > 127.0 ? 127.0 : q < -127.0 ? -127.0 : q) & 0xffu) << (8 * j);
    }
  }
}

// A row by WPR waves (1 or 4), R vectors a lane in registers; longer rows (WPR 4)
// are read twice.  Bound by memory: 81920 rows of 2048 bf16, 503 MB in and out, 90 us
// (at best 79), 5.6 TB/s; 60.7k kept rows 76 (69), as many compact ones 59 (56); float32
// 163 (153), 839 MB, 5.1 TB/s, 135 (125) and 116 (112).  (With a branch to the float64
// quotient behind every element 150 and 168 for the first two.)
template <int DT, int WPR, int R>
__device__ __forceinline__ void quantize_row(const char* x, uint64_t width, char* q, uint64_t pitch, float* scale,
                                             int product, uint32_t* red) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  constexpr uint64_t STEP = (uint64_t)64 * WPR * V;
  u32x4 held[R];
  Top<DT> best;
  // this lane's vector of the STEP elements from b on; whether all of them are inside is the same on all lanes
  auto load = [&](uint64_t b) {
    const uint64_t c = b + (uint64_t)tid * V;
    if (b + STEP <= width) return (u32x4) * (const u32x4_any*)(x + c * SZ);
    if (b < width) {
      const int64_t left = (int64_t)width - (int64_t)c;
      return load_n<DT, false>(x + c * SZ, (int)(left < V ? left > 0 ? left : 0 : V));
    }
    return u32x4{0u, 0u, 0u, 0u};
  };
#pragma unroll
  for (int k = 0; k < R; ++k) held[k] = load(k * STEP);
#pragma unroll
  for (int k = 0; k < R; ++k) best.take(held[k]);
  if constexpr (WPR > 1)
    for (uint64_t b = R * STEP; b < width; b += STEP) best.take(load(b));
  uint32_t top = wave_umax(best.bits());
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WPR; ++k) top = red[k] > top ? red[k] : top;
    top = (uint32_t)__builtin_amdgcn_readfirstlane((int)top);
  }
  const bool nan = top >= 0x7f800000u;
  const float most = __uint_as_float(top);
  const float s = nan ? __uint_as_float(0x7fc00000u) : product ? most * (1.0f / 127.0f) : most / 127.0f;
  auto put = [&](uint64_t b, const uint32_t* w) {
    const uint64_t c = b + (uint64_t)tid * V;
    char* o = q + c;
    if (b + STEP <= pitch || c + V <= pitch) {
      if constexpr (V == 8) *(u32x2_byte*)o = u32x2_byte{w[0], w[1]};
      else *(u32_byte*)o = w[0];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < pitch) o[i] = (char)(w[i / 4] >> (8 * (i & 3)));
    }
  };
  uint32_t w[V / 4];
  if (s >= 0x1p-100f) {
    const float inv = __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (k * STEP < pitch) {
        quantized<DT, V>(held[k], s, inv, w);
        put(k * STEP, w);
      }
    if constexpr (WPR > 1)
      for (uint64_t b = R * STEP; b < pitch; b += STEP) {
        quantized<DT, V>(load(b), s, inv, w);
        put(b, w);
      }
  } else {   // a small scale, zeros, or (NaN) a marked row
#pragma unroll 1
    for (uint64_t b = 0; b < pitch; b += STEP) {
      if (s > 0.0f) {
        quantized_small<DT, V>(load(b), s, w);
      } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = 0;
      }
      put(b, w);
    }
  }
  if (tid == 0) *scale = s;
}

// Plain rows: blockIdx.y the rank, 4 / WPR rows a workgroup.  (One row a wave: in a
// loop over rows the compiler keeps the masks of a row's end for the next one.)
constexpr uint64_t kRowsGrid = 1u << 22;   // workgroups of 256 threads whose work-items fit 32 bits
template <int DT, int WPR, int R>
__global__ __launch_bounds__(256) void k_int8_rows(RowsArgs a) {
  __shared__ uint32_t red[4];
  const uint64_t r = blockIdx.y;
  const int wave = WPR == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const uint64_t row = a.row0 + (uint64_t)blockIdx.x * (4 / WPR) + wave;
  if (row < a.rows)   // the same on the wave, or (WPR 4) the workgroup
    quantize_row<DT, WPR, R>(a.x + r * a.x_stride + row * a.width * Ty<DT>::SZ, a.width,
                             a.q + r * a.q_stride + row * a.q_pitch, a.q_pitch, (float*)(a.s + r * a.s_stride) + row,
                             a.product, red);
}

// The experts' kept rows, compact.
struct TileArgs {
  RowsArgs r;
  const int* start;
  const int2* mtab;
  const int* map;
  int per;
};
template <int DT, int WPR, int R>
__global__ __launch_bounds__(256) void k_int8_tiles(TileArgs a) {
  __shared__ uint32_t red[4];
  auto row = [&](uint32_t l, uint32_t place, int e) {
    quantize_row<DT, WPR, R>(a.r.x + (uint64_t)(e / a.per) * a.r.x_stride + (uint64_t)place * a.r.width * Ty<DT>::SZ,
                             a.r.width, a.r.q + (uint64_t)l * a.r.q_pitch, a.r.q_pitch, (float*)a.r.s + l, a.r.product, red);
  };
  if constexpr (WPR == 1) {
    table_rows(a.start, a.mtab, a.map, row);
  } else {   // a row of the tile's a workgroup
    const int2 at = a.mtab[blockIdx.x];
    const int l = at.y + (int)blockIdx.y;
    if (l < a.start[at.x + 1]) row((uint32_t)l, (uint32_t)a.map[l], at.x);
  }
}

struct Plain {
  RowsArgs a;
  unsigned ranks;
  hipStream_t st;
  template <int DT, int WPR, int R>
  hipError_t run() const {
    const uint64_t per = 4 / WPR;
    RowsArgs b = a;
    for (b.row0 = 0; b.row0 < a.rows; b.row0 += kRowsGrid * per) {
      const uint64_t blocks = std::min((a.rows - b.row0 + per - 1) / per, kRowsGrid);
      CC_LAUNCH((k_int8_rows<DT, WPR, R>), dim3((unsigned)blocks, ranks), dim3(256), 0, st, b);
    }
    return hipGetLastError();
  }
};
struct Tiled {
  TileArgs a;
  unsigned tiles;
  hipStream_t st;
  template <int DT, int WPR, int R>
  hipError_t run() const {
    const dim3 grid(tiles, WPR == 1 ? kTileParts : kFfnTile[kFfnTiles - 1]);
    CC_LAUNCH((k_int8_tiles<DT, WPR, R>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
  }
};
// the least registers that hold a row
template <int DT, class L>
hipError_t pick_rows(uint64_t width, const L& launch) {
  const uint64_t one = (uint64_t)64 * Ty<DT>::V;
  if (width <= one) return launch.template run<DT, 1, 1>();
  if (width <= 2 * one) return launch.template run<DT, 1, 2>();
  if (width <= 4 * one) return launch.template run<DT, 1, 4>();
  if (width <= 8 * one) return launch.template run<DT, 1, 8>();
  return launch.template run<DT, 4, 8>();
}

// ------------------------------------------------------------------ copies

// Lines of at least 16 bytes that start at any byte into lines of whole 16-byte
// chunks, zeros past their end.
__device__ __forceinline__ u32x4 line_chunk(const char* from, uint64_t cols, uint64_t c) {
  if (c + 16 <= cols) return *(const u32x4_byte*)(from + c);
  if (c < cols) return line_tail(from + cols, (int)(cols - c));
  return u32x4{0u, 0u, 0u, 0u};
}

// An expert's weights (z), 16 lines a workgroup, 4 a wave at a time; y: which of
// them.  Bound by memory: 16 experts of 2047 x 2047 30 us, 4.5 TB/s (53 with the last
// bytes of a line loaded one by one).
struct WeightCopy {
  const int* start;
  int per;
  struct {
    const char* from;
    uint64_t rank_stride;
    uint64_t each, cols;   // lines of an expert
    char* to;
    uint64_t pitch;
  } job[2];
};
constexpr int kCopyLines = 16;
__global__ __launch_bounds__(256) void k_int8_copy_weights(WeightCopy a) {
  const auto& j = a.job[blockIdx.y];
  const int lane = threadIdx.x & 63, e = blockIdx.z, r = e / a.per;
  if (a.start[e] == a.start[e + 1]) return;   // no rows: never read
  const uint64_t first = (uint64_t)blockIdx.x * kCopyLines + 4 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const char* from = j.from + (uint64_t)r * j.rank_stride + ((uint64_t)(e - r * a.per) * j.each + first) * j.cols;
  char* to = j.to + ((uint64_t)e * j.each + first) * j.pitch;
  for (uint64_t c = (uint64_t)lane * 16; c < j.pitch; c += 1024) {
    u32x4 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (first + k < j.each) w[k] = line_chunk(from + k * j.cols, j.cols, c);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (first + k < j.each) *(u32x4*)(to + k * j.pitch + c) = w[k];
  }
}

// The kept rows of a product, compact.
__global__ __launch_bounds__(256) void k_int8_copy_rows(TileArgs a) {
  table_rows(a.start, a.mtab, a.map, [&](uint32_t l, uint32_t place, int e) {
    const char* from = a.r.x + (uint64_t)(e / a.per) * a.r.x_stride + (uint64_t)place * a.r.width;
    char* to = a.r.q + (uint64_t)l * a.r.q_pitch;
    for (uint64_t c0 = (uint64_t)(threadIdx.x & 63) * 16; c0 < a.r.q_pitch; c0 += 4 * 1024) {   // four loads under way
      u32x4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = line_chunk(from, a.r.width, c0 + q * 1024);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c0 + q * 1024 < a.r.q_pitch) *(u32x4*)(to + c0 + q * 1024) = w[q];
    }
  });
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

hipError_t copy_weights(const Int8Launch& L, bool block) {
  const uint64_t W = L.s.W, F = L.s.F, in = block ? 2 * F : F;
  WeightCopy a = {};
  a.start = (const int*)(L.ws + L.o.plan.start);
  a.per = L.s.E / L.s.N;
  int jobs = 0;
  uint64_t lines = 0;
  auto add = [&](const Side& w, uint64_t each, uint64_t cols, uint64_t to) {
    a.job[jobs++] = {w.base, w.stride, each, cols, L.ws + to, line_pitch(L.s, cols)};
    lines = std::max(lines, each);
  };
  if (L.o.copied_in) add(L.w_in, in, W, L.o.w_in);
  if (L.o.copied_out) add(L.w_out, W, F, L.o.w_out);
  if (jobs == 0) return hipSuccess;
  const dim3 grid((unsigned)((lines + kCopyLines - 1) / kCopyLines), (unsigned)jobs, (unsigned)L.s.E);
  CC_LAUNCH(k_int8_copy_weights, grid, dim3(256), 0, L.st, a);
  return hipGetLastError();
}

TileArgs tile_args(const Int8Launch& L, const RowsArgs& r) {
  return TileArgs{r, (const int*)(L.ws + L.o.plan.start), (const int2*)(L.ws + L.o.plan.mtab[kFfnTiles - 1]),
                  (const int*)(L.ws + L.o.plan.rowmap), L.s.E / L.s.N};
}

// the plan, and the kept rows quantised
hipError_t planned_rows(const Int8Launch& L, const RowsArgs& r) {
  const hipError_t e = launch_ffn_plan(L.s, L.o.plan, L.ws, L.kept, L.st);
  if (e != hipSuccess) return e;
  const Tiled t{tile_args(L, r), (unsigned)L.s.mtiles[kFfnTiles - 1], L.st};
  return L.dt == DT_F32 ? pick_rows<DT_F32>(r.width, t) : pick_rows<DT_BF16>(r.width, t);
}

// `lines` rows of `cols` weights an expert, the caller's or their copies
void weights_of(I8Args* g, const Int8Launch& L, const Side& w, const Side& s, uint64_t lines, uint64_t cols, int copied,
                uint64_t copy) {
  const uint64_t p = copied ? line_pitch(L.s, cols) : cols;
  g->b = copied ? WtSide{L.ws + copy, (uint64_t)g->per * lines * p, lines * p, p}
                : WtSide{w.base, w.stride, lines * p, p};
  g->sw = s.base;
  g->sw_stride = s.stride;
  g->M = (int)lines;
}

}  // namespace

hipError_t launch_int8_rows(const Int8Rows& L) {
  if (L.rows == 0) return hipSuccess;
  const Plain p{{L.x, L.x_stride, L.q, L.q_stride, L.q_pitch, L.s, L.s_stride, L.rows, L.width, 0, L.product},
                (unsigned)L.N, L.st};
  return L.dt == DT_F32 ? pick_rows<DT_F32>(L.width, p) : pick_rows<DT_BF16>(L.width, p);
}

// Whether weights of rows that are no whole 16-byte vectors are copied into lines
// that direct loads take, so that the same tiles run on them.  The block's rows x
// and h lie in such lines anyway; a product on its own copies its rows too.
// Measured on 16 experts, bf16, through registers and copied: block 2047 x 2047 512
// rows an expert 273 us and 289, 1024 418 and 397, 4096 1505 and 1059; 201 x 333 512 rows
// 42 and 45, 1024 62 and 60, 4096 161 and 140; product 2047 x 2047 1024 rows 188 and
// 161, 4096 679 and 486, 1001 x 733 1024 rows 61 and 61, 517 x 300 4096 rows 108 and 119.
constexpr uint64_t kCopyInt8Rows = 1024, kCopyInt8BlockCols = 192, kCopyInt8ProductCols = 512;
static_assert(kCopyInt8BlockCols >= 16 && kCopyInt8ProductCols >= 16, "line_chunk's lines");
static int int8_copied(const FfnShape& s, bool block, uint64_t lines, uint64_t cols) {
  const uint64_t p = line_pitch(s, cols);
  return cols % 16 != 0 && s.rows >= kCopyInt8Rows * s.E &&
         std::min(lines, cols) >= (block ? kCopyInt8BlockCols : kCopyInt8ProductCols) && s.most * p <= kMaxSpan &&
         lines * p <= kMaxSpan;
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
  o.xq_pitch = line_pitch(s, s.W);
  o.hq_pitch = line_pitch(s, s.F);
  o.copied_in = int8_copied(s, block, block ? 2 * s.F : s.F, s.W);
  o.copied_out = block && int8_copied(s, true, s.W, s.F);
  if (block || o.copied_in) o.xq = take(s.rows * o.xq_pitch);
  if (block) {
    o.xs = take(s.rows * 4);
    o.h = take(s.rows * s.F * out_es);
    o.hq = take(s.rows * o.hq_pitch);
    o.hs = take(s.rows * 4);
  }
  if (o.copied_in) o.w_in = take((uint64_t)s.E * (block ? 2 : 1) * s.F * o.xq_pitch);
  if (o.copied_out) o.w_out = take((uint64_t)s.E * s.W * o.hq_pitch);
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
  bool fast = L.x_ok && L.w_in_ok && side * W <= kMaxSpan && C * W <= kMaxSpan;
  g.a = RowSide{L.x.base, L.x.stride, W, g.map, side * W};
  if (L.o.copied_in) {
    const RowsArgs r{L.x.base, L.x.stride, L.ws + L.o.xq, 0, L.o.xq_pitch, nullptr, 0, L.s.rows, W, 0, 0};
    CC_LAUNCH(k_int8_copy_rows, dim3((unsigned)L.s.mtiles[kFfnTiles - 1], kTileParts), dim3(256), 0, L.st, tile_args(L, r));
    if ((e = hipGetLastError()) != hipSuccess || (e = copy_weights(L, false)) != hipSuccess) return e;
    g.a = RowSide{r.q, 0, r.q_pitch, nullptr, L.s.most * r.q_pitch};
    fast = true;
  }
  weights_of(&g, L, L.w_in, L.s_in, C, W, L.o.copied_in, L.o.w_in);
  g.sx = L.xs.base;
  g.sx_stride = L.xs.stride;
  g.sx_map = g.map;
  g.out = RowSide{L.y.base, L.y.stride, C * es, g.map, side * C * es};
  return pick_int8<K_DOWN>(g, L, fast, L.y_ok);
}

hipError_t launch_int8_ffn(const Int8Launch& L) {
  const uint64_t W = L.s.W, F = L.s.F, es = elem_size(L.dt);
  const RowsArgs r{L.x.base, L.x.stride, L.ws + L.o.xq, 0, L.o.xq_pitch, L.ws + L.o.xs, 0, L.s.rows, W, 0,
                   L.product};
  hipError_t e = planned_rows(L, r);
  if (e != hipSuccess || (e = copy_weights(L, true)) != hipSuccess) return e;
  I8Args g = int8_args(L);
  g.K = (int)W;
  g.N = (int)(2 * F);
  g.a = RowSide{r.q, 0, L.o.xq_pitch, nullptr, L.s.most * L.o.xq_pitch};
  weights_of(&g, L, L.w_in, L.s_in, 2 * F, W, L.o.copied_in, L.o.w_in);
  g.sx = r.s;
  g.out = RowSide{L.ws + L.o.h, 0, F * es, nullptr, L.s.most * F * es};
  const bool rows_fit = L.s.most * std::max(L.o.xq_pitch, L.o.hq_pitch) <= kMaxSpan;
  if ((e = pick_int8<K_GATEUP>(g, L, L.o.copied_in || (L.w_in_ok && rows_fit && 2 * F * W <= kMaxSpan),
                                F * es % 16 == 0)) != hipSuccess)
    return e;
  Int8Rows q = {};
  q.x = L.ws + L.o.h;
  q.q = L.ws + L.o.hq; q.q_pitch = L.o.hq_pitch;
  q.s = L.ws + L.o.hs;
  q.rows = L.s.rows; q.width = F;
  q.N = 1; q.dt = L.dt; q.product = L.product; q.st = L.st;
  if ((e = launch_int8_rows(q)) != hipSuccess) return e;
  g.K = (int)F;
  g.N = (int)W;
  g.a = RowSide{q.q, 0, L.o.hq_pitch, nullptr, L.s.most * L.o.hq_pitch};
  weights_of(&g, L, L.w_out, L.s_out, W, F, L.o.copied_out, L.o.w_out);
  g.sx = q.s;
  g.out = RowSide{L.y.base, L.y.stride, W * es, g.map, (uint64_t)L.s.E * L.s.cap * W * es};
  return pick_int8<K_DOWN>(g, L, L.o.copied_out || (L.w_out_ok && rows_fit && F * W <= kMaxSpan), L.y_ok);
}

}  // namespace cc
