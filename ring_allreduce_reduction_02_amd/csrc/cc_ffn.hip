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

#include "cc_ffn_tile.h"

namespace cc {
namespace {

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
  const uint32_t* kept;   // in memory (ARGS: v)
  int N, E;
  uint64_t cap;
  int* start;
  int2* mtab[kFfnTiles];
  int* rowmap;
};

// Workgroup e writes expert e's first compact row, its row tiles and its rows'
// places in the rank's buffer.  ARGS: the counts are the launch's arguments, which lie in
// the host's memory: read once, side by side (8 ranks' of 64 experts 4.8 us, one after
// another 5.6).
template <bool ARGS>
__global__ __launch_bounds__(256) void k_ffn_plan(PlanArgs a) {
  __shared__ uint32_t red[1 + kFfnTiles][4];
  __shared__ uint32_t counts[ARGS ? kPlanCounts : 1];
  const int e = blockIdx.x, tid = threadIdx.x, N = a.N;
  if constexpr (ARGS) {
    constexpr int Q = (kPlanCounts + 255) / 256;
    const int n = (e + 1) * N;
    uint32_t v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = tid + q * 256 < n ? a.v[tid + q * 256] : 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (tid + q * 256 < n) counts[tid + q * 256] = v[q];
    __syncthreads();
  }
  auto kept = [&](int i) { return ARGS ? counts[i] : a.kept[i]; };
  uint32_t sum[1 + kFfnTiles] = {};
  for (int x = tid; x < e; x += 256) {
    uint32_t n = 0;
    for (int i = 0; i < N; ++i) n += kept(x * N + i);
    sum[0] += n;
#pragma unroll
    for (int k = 0; k < kFfnTiles; ++k) sum[1 + k] += (n + kFfnTile[k] - 1) / kFfnTile[k];
  }
#pragma unroll
  for (int k = 0; k <= kFfnTiles; ++k) {
    const uint32_t s = group_usum<64>(sum[k]);
    if ((tid & 63) == 0) red[k][tid >> 6] = s;
  }
  __syncthreads();
  auto before = [&](int k) { return red[k][0] + red[k][1] + red[k][2] + red[k][3]; };
  const uint32_t r0 = before(0);
  const int per = a.E / N, l = e % per;
  uint32_t at = r0;
  for (int i = 0; i < N; ++i) {
    const uint32_t n = kept(e * N + i);
    const uint32_t src = (uint32_t)(((uint64_t)i * per + l) * a.cap);
    for (uint32_t s = tid; s < n; s += 256) a.rowmap[at + s] = (int)(src + s);
    at += n;
  }
#pragma unroll
  for (int k = 0; k < kFfnTiles; ++k) {
    const uint32_t nt = (at - r0 + kFfnTile[k] - 1) / kFfnTile[k], t0 = before(1 + k);
    for (uint32_t t = tid; t < nt; t += 256) a.mtab[k][t0 + t] = make_int2(e, (int)(r0 + t * kFfnTile[k]));
  }
  if (tid == 0) {
    a.start[e] = (int)r0;
    if (e == a.E - 1) a.start[a.E] = (int)at;
  }
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

constexpr int kCopyLines = kFfnTile[kFfnTiles - 1], kCopyParts = 4;

// Workgroup (x, y, z) copies part z of 64 lines of job y.  Bound by memory: the
// weights of 16 experts of 2047 x 2047 bf16 and 60.7k rows, 1.3 GB in and out, 248 us,
// 5.2 TB/s (all 64 lines a workgroup 300, and with one load of a lane under way 350;
// 6 experts of 515 x 331 and 1.4k rows 11 us and 31).
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
  constexpr uint64_t PART = kCopyLines / kCopyParts;
  first += blockIdx.z * PART;
  end = first + PART < end ? first + PART : end;
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
        w[q] = load_line<DT>(p, j.cols, c + q * 64 * V);
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

hipError_t plan(const FfnShape& s, const FfnWs& o, char* ws, const uint32_t* kept, hipStream_t st) {
  PlanArgs a;
  const int n = s.N * s.E;
  a.kept = nullptr;
  if (n <= kPlanCounts) {
    for (int i = 0; i < n; ++i) a.v[i] = kept[i];
  } else {
    uint32_t* to = (uint32_t*)(ws + o.kept);
    for (int i = 0; i < n; i += kPlanCounts) {
      PutArgs p;
      p.n = n - i < kPlanCounts ? n - i : kPlanCounts;
      for (int k = 0; k < p.n; ++k) p.v[k] = kept[i + k];
      p.to = to + i;
      CC_LAUNCH(k_ffn_put, dim3(1), dim3(256), 0, st, p);
    }
    a.kept = to;
  }
  a.N = s.N; a.E = s.E; a.cap = s.cap;
  a.start = (int*)(ws + o.start);
  for (int k = 0; k < kFfnTiles; ++k) a.mtab[k] = (int2*)(ws + o.mtab[k]);
  a.rowmap = (int*)(ws + o.rowmap);
  if (a.kept) CC_LAUNCH(k_ffn_plan<false>, dim3((unsigned)s.E), dim3(256), 0, st, a);
  else CC_LAUNCH(k_ffn_plan<true>, dim3((unsigned)s.E), dim3(256), 0, st, a);
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

CkArgs ckpt_args(const FfnLaunch& L, const GemmArgs& g) {
  CkArgs a;
  (GemmArgs&)a = g;
  a.at = ckpt_row(L.s.W, L.s.F);
  const uint64_t pitch = (uint64_t)a.at.pitch;
  a.ck = RowSide{L.ckpt.base, L.ckpt.stride, pitch, (const int*)(L.ws + L.o.rowmap), (uint64_t)L.s.E * L.s.cap * pitch};
  return a;
}

hipError_t copy_operands(const FfnLaunch& L, int grad) {
  const uint64_t W = L.s.W, F = L.s.F, n = L.s.E, tiles = L.s.mtiles[kFfnTiles - 1];
  CopyArgs a = {};
  a.start = (const int*)(L.ws + L.o.start);
  a.mtab = (const int2*)(L.ws + L.o.mtab[kFfnTiles - 1]);
  a.map = (const int*)(L.ws + L.o.rowmap);
  a.per = L.s.E / L.s.N;
  // rows x that a checkpoint holds are unpacked there (ckpt_unpack_x)
  a.job[0] = {L.x.base, L.x.stride, grad && L.ckpt.base ? 0 : tiles, 0, L.ws + L.o.x, W, line_pitch(L.s, W)};
  a.job[1] = {L.w_in.base, L.w_in.stride, n * 2 * F, 2 * F, L.ws + L.o.w_in, W, line_pitch(L.s, W)};
  a.job[2] = {L.w_out.base, L.w_out.stride, n * W, W, L.ws + L.o.w_out, F, line_pitch(L.s, F)};
  if (grad) a.job[3] = {L.dy.base, L.dy.stride, tiles, 0, L.ws + L.o.dy, W, line_pitch(L.s, W)};
  a.h = L.ws + L.o.h;
  a.dgu = grad ? L.ws + L.o.dgu : nullptr;
  a.F = F;
  a.h_pitch = line_pitch(L.s, F);
  a.dgu_pitch = line_pitch(L.s, 2 * F);
  const uint64_t blocks = std::max(tiles, (n * std::max(2 * F, W) + kCopyLines - 1) / kCopyLines);
  const dim3 grid((unsigned)blocks, grad ? 4 : 3, kCopyParts), blk(256);
  if (L.s.dt == DT_F32) CC_LAUNCH(k_ffn_copy<DT_F32>, grid, blk, 0, L.st, a);
  else CC_LAUNCH(k_ffn_copy<DT_BF16>, grid, blk, 0, L.st, a);
  return hipGetLastError();
}

hipError_t prepare(const FfnLaunch& L, int grad) {
  const hipError_t e = plan(L.s, L.o, L.ws, L.kept, L.st);
  return e == hipSuccess && L.o.copied ? copy_operands(L, grad) : e;
}

}  // namespace

FfnWs ffn_ws(const FfnShape& s, int grad, int ckpt) {
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
    if (grad && ckpt) o.x = take(s.rows * s.W * es);
  }
  o.bytes = at;
  return o;
}

hipError_t launch_ffn_plan(const FfnShape& s, const FfnWs& o, char* ws, const uint32_t* kept, hipStream_t st) {
  return plan(s, o, ws, kept, st);
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
  if (L.ckpt.base) {
    if ((e = ckpt_pack_x(L)) != hipSuccess || (e = ckpt_gateup(ckpt_args(L, g), L)) != hipSuccess) return e;
  } else {
    g.pre = rows_of(L, L.pre, 2 * F);
    if ((e = pick_gemm<K_GATEUP>(g, L)) != hipSuccess) return e;
  }
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
  if (L.ckpt.base) {
    if ((e = ckpt_unpack_x(L)) != hipSuccess || (e = ckpt_dhid(ckpt_args(L, g), L)) != hipSuccess) return e;
  } else {
    g.pre = rows_of(L, L.pre, 2 * F);
    if ((e = pick_gemm<K_DHID>(g, L)) != hipSuccess) return e;
  }
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
  g.b_rows = L.ckpt.base ? compact(L, L.o.x, W) : rows_in(L, L.x, L.o.x);
  g.wout = wts(L, L.dw_in, 2 * F, W);
  return pick_gemm<K_DW>(g, L);
}

}  // namespace cc