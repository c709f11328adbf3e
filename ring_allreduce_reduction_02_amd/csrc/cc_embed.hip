// Embedding lookup with scaling, and the table's gradient from the sorted
// tokens: of each rank, or summed over the ranks onto every rank.
//
//   out[t, :] = scale * table[ids[t], :]            (zeros where ids[t] is no row)
//   d[v, :]   = scale * sum over t with ids[t] = v of grad[t, :]
//
// Both are one pass over memory: the lookup reads and writes tokens * width
// elements, the gradient reads tokens * width and writes all vocab * width
// (most rows are zeros: a batch holds few of a vocabulary's words).

#include <algorithm>

#include "cc_device.h"
#include "cc_llm.h"

namespace cc {
namespace {

constexpr int kEmbedBlock = 256;

struct EmbedArgs {
  const char* table;
  uint64_t ts;
  const char* ids;
  uint64_t is;
  char* out;
  uint64_t os;
  uint64_t vocab, tokens, width;
  float scale;
};

// 16 bytes of a row: with VEC rows are 16-byte aligned; otherwise they start
// anywhere (global memory takes whole vectors at any element), and the row's
// last vector, `left` elements short of V, goes by elements.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <int DT, bool VEC>
__device__ __forceinline__ u32x4 load_part(const char* p, int64_t left) {
  if constexpr (VEC) {
    return left > 0 ? *(const u32x4*)p : u32x4{0u, 0u, 0u, 0u};
  } else {
    if (left >= Ty<DT>::V) return *(const u32x4_any*)p;
    float x[Ty<DT>::V] = {};
#pragma unroll
    for (int i = 0; i < Ty<DT>::V; ++i)
      if (i < left) x[i] = ld1<DT>(p + i * Ty<DT>::SZ);
    return pack<DT>(x);   // widened and packed again: the same bits
  }
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_part(char* p, u32x4 w, int64_t left) {
  if constexpr (VEC) {
    if (left > 0) stg(p, w);
  } else {
    if (left >= Ty<DT>::V) {
      *(u32x4_any*)p = w;
      return;
    }
    float x[Ty<DT>::V];
    unpack<DT>(w, x);
#pragma unroll
    for (int i = 0; i < Ty<DT>::V; ++i)
      if (i < left) st1<DT>(p + i * Ty<DT>::SZ, x[i]);
  }
}

// One workgroup a token row and rank.  Bound by memory: 8 ranks x 4096 tokens
// of 2048 float32 (537 MB of rows in and out) take 68 us, 7.8 TB/s (words that
// repeat are read from the cache); 4 tokens a rank 3 us, the launch.
template <int DT, bool VEC>
__global__ __launch_bounds__(kEmbedBlock) void k_embed(EmbedArgs a) {
  const uint64_t t = blockIdx.x, r = blockIdx.y;
  const int id = ((const int*)(a.ids + r * a.is))[t];
  const bool in = (uint32_t)id < a.vocab;
  char* o = a.out + r * a.os + t * a.width * Ty<DT>::SZ;
  const char* s = a.table + r * a.ts + (in ? (uint64_t)id : 0) * a.width * Ty<DT>::SZ;
  constexpr int V = Ty<DT>::V;
  for (uint64_t c = (uint64_t)threadIdx.x * V; c < a.width; c += kEmbedBlock * V) {
    const int64_t left = (int64_t)(a.width - c);
    u32x4 w = {0u, 0u, 0u, 0u};
    if (in) {
      float x[V];
      unpack<DT>(load_part<DT, VEC>(s + c * Ty<DT>::SZ, left), x);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] *= a.scale;
      w = pack<DT>(x);
    }
    store_part<DT, VEC>(o + c * Ty<DT>::SZ, w, left);
  }
}

struct EmbedGradArgs {
  const char* grad;
  uint64_t gs;
  char* out;
  uint64_t os;
  const int* keys;   // each rank's sorted ids and their positions, [N][tokens]
  const int* vals;
  float* partial;    // [N][pieces][pitch]
  uint64_t vocab, tokens, width, pitch;
  uint64_t pieces;   // of kEmbedPiece sorted positions per rank; 0: no partial sums
  float scale;
  int N;
};

// A wave's columns: CB blocks of 64 lanes, V consecutive elements a lane, as
// many (1, 2 or 4) as a row has, so that a row of 2048 bf16 takes one walk over
// its tokens and a narrow one has more token rows under way (4 ranks x 2000
// tokens, 2000 x 512 bf16: 28 us with one block and 16 rows, 50 with four blocks and 4).
template <int DT, int B>
struct Cols {
  static constexpr int V = Ty<DT>::V;
  static constexpr int CB = B;
  static constexpr int STEP = 64 * V * CB;
  static constexpr int BATCH = 16 / CB;   // token rows under way per wave
};

// acc += Q token rows, the first n of them; g is the lane's first byte of row 0,
// `mine` a position a lane, from lane k on.
template <int DT, bool VEC, int B, int Q>
__device__ __forceinline__ void add_batch(const char* g, uint64_t pitch, int64_t left, int mine, int k, int n,
                                          float (&acc)[Cols<DT, B>::CB][Cols<DT, B>::V]) {
  constexpr int V = Ty<DT>::V;
  u32x4 w[Q][B];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const uint32_t t = (uint32_t)__builtin_amdgcn_readlane(mine, q < n ? k + q : k);
#pragma unroll
    for (int i = 0; i < B; ++i) w[q][i] = load_part<DT, VEC>(g + t * pitch + i * 64 * V * Ty<DT>::SZ, left - i * 64 * V);
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (q >= n) break;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      float x[V];
      unpack<DT>(w[q][i], x);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[i][e] += x[e];
    }
  }
}

// acc += the rows of grad at the sorted positions [lo, hi) of rank r, columns
// c0 + 64 V i + V lane.  Positions are fetched 64 at a time, their rows BATCH
// at a time, so that a lane has 16 loads under way, and the last few by 4.
template <int DT, bool VEC, int B>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, uint64_t r, uint64_t lo, uint64_t hi, uint64_t c0,
                                         int lane, float (&acc)[Cols<DT, B>::CB][Cols<DT, B>::V]) {
  constexpr int V = Ty<DT>::V, BATCH = Cols<DT, B>::BATCH, SZ = Ty<DT>::SZ;
  const int* vals = a.vals + r * a.tokens;
  const char* base = a.grad + r * a.gs + (c0 + lane * V) * SZ;
  const int64_t left = (int64_t)(a.width - c0) - lane * V;
  for (uint64_t p0 = lo; p0 < hi; p0 += 64) {
    const int n = (int)(hi - p0 < 64 ? hi - p0 : 64);
    const int mine = lane < n ? vals[p0 + lane] : 0;
    int k = 0;
    if constexpr (BATCH > 4)
      for (; k + BATCH <= n; k += BATCH)
        add_batch<DT, VEC, B, BATCH>(base, a.width * SZ, left, mine, k, BATCH, acc);
    for (; k < n; k += 4) add_batch<DT, VEC, B, 4>(base, a.width * SZ, left, mine, k, n - k, acc);
  }
}

// first sorted position whose key is at least k
__device__ __forceinline__ uint32_t lower_bound(const int* keys, uint32_t n, uint32_t k) {
  uint32_t lo = 0, hi = n;
  while (lo < hi) {
    const uint32_t mid = (lo + hi) >> 1;
    if ((uint32_t)keys[mid] < k) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// Partial sums of the pieces (kEmbedPiece sorted positions) that lie inside
// one word's run of kEmbedLong or more, one wave each, so that a frequent word
// is summed by many.
template <int DT, bool VEC, int B>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_pieces(EmbedGradArgs a) {
  typedef Cols<DT, B> C;
  const int lane = threadIdx.x & 63;
  const uint64_t piece = (uint64_t)blockIdx.x * (kEmbedBlock / 64) + (threadIdx.x >> 6), r = blockIdx.y;
  if (piece >= a.pieces) return;
  const uint64_t p0 = piece * kEmbedPiece;
  const int* keys = a.keys + r * a.tokens;
  const uint32_t k = (uint32_t)keys[p0];
  if (k >= a.vocab || k != (uint32_t)keys[p0 + kEmbedPiece - 1]) return;
  const uint32_t end = lower_bound(keys, (uint32_t)a.tokens, k + (lane & 1));   // the run's first and last + 1
  if (__builtin_amdgcn_readlane(end, 1) - __builtin_amdgcn_readlane(end, 0) < kEmbedLong) return;
  float* o = a.partial + (r * a.pieces + piece) * a.pitch;
  for (uint64_t c0 = 0; c0 < a.width; c0 += C::STEP) {
    float acc[C::CB][C::V] = {};
    add_rows<DT, VEC, B>(a, r, p0, p0 + kEmbedPiece, c0, lane, acc);
#pragma unroll
    for (int i = 0; i < C::CB; ++i) {
      const uint64_t c = c0 + (uint64_t)(i * 64 + lane) * C::V;
      if (c < a.width) stw_vec<DT>((char*)(o + c), acc[i]);
    }
  }
}

// acc += the sorted positions [lo, hi) of rank r, part of a run of `run`
// positions: of a long run, whole pieces come as their partial sums.
template <int DT, bool VEC, int B>
__device__ __forceinline__ void add_run(const EmbedGradArgs& a, uint64_t r, uint64_t lo, uint64_t hi, uint64_t run,
                                        uint64_t c0, int lane, float (&acc)[Cols<DT, B>::CB][Cols<DT, B>::V]) {
  typedef Cols<DT, B> C;
  const uint64_t f = (lo + kEmbedPiece - 1) / kEmbedPiece, l = hi / kEmbedPiece;
  if (a.pieces == 0 || run < kEmbedLong || f >= l) {
    add_rows<DT, VEC, B>(a, r, lo, hi, c0, lane, acc);
    return;
  }
  add_rows<DT, VEC, B>(a, r, lo, f * kEmbedPiece, c0, lane, acc);
  const float* part = a.partial + (r * a.pieces + f) * a.pitch + c0 + lane * C::V;
  for (uint64_t p = f; p < l; ++p, part += a.pitch)
#pragma unroll
    for (int k = 0; k < C::CB; ++k) {
      if (c0 + (uint64_t)(k * 64 + lane) * C::V >= a.width) continue;
      float x[C::V];
      ldw_vec<DT>((const char*)(part + k * 64 * C::V), x);
#pragma unroll
      for (int e = 0; e < C::V; ++e) acc[k][e] += x[e];
    }
  add_rows<DT, VEC, B>(a, r, l * kEmbedPiece, hi, c0, lane, acc);
}

// columns of acc, scaled, to the ranks [r0, r0 + nr)
template <int DT, bool VEC, int B>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, char* o, int r0, int nr, uint64_t c0, int lane,
                                        float (&acc)[Cols<DT, B>::CB][Cols<DT, B>::V]) {
  typedef Cols<DT, B> C;
#pragma unroll
  for (int k = 0; k < C::CB; ++k) {
    const uint64_t c = c0 + (uint64_t)(k * 64 + lane) * C::V;
    if (c >= a.width) continue;
#pragma unroll
    for (int e = 0; e < C::V; ++e) acc[k][e] *= a.scale;
    for (int r = r0; r < r0 + nr; ++r) {
      store_part<DT, VEC>(o + (uint64_t)r * a.os + c * Ty<DT>::SZ, pack<DT>(acc[k]), (int64_t)(a.width - c));
    }
  }
}

// a row of zeros: whole vectors wherever the row starts
template <int DT>
__device__ __forceinline__ void zero_row(char* o, uint64_t bytes, int lane) {
  const uint64_t head = (16 - ((uintptr_t)o & 15u)) & 15u, h = head < bytes ? head : bytes;
  constexpr int SZ = Ty<DT>::SZ;
  if ((uint64_t)lane * SZ < h) st1<DT>(o + lane * SZ, 0.0f);
  const uint64_t body = (bytes - h) / 16 * 16;
  for (uint64_t c = (uint64_t)lane * 16; c < body; c += 1024) stg(o + h + c, u32x4{0u, 0u, 0u, 0u});
  const uint64_t tail = h + body + (uint64_t)lane * SZ;
  if (tail < bytes) st1<DT>(o + tail, 0.0f);
}

// A workgroup takes every gridDim.x-th table row, up to 16 or 32 of them (frequent
// words have neighbouring ids and so fall to different workgroups).  Where a
// row's tokens lie in the sorted ids is found by binary search, all rows (and
// ranks) of the workgroup at once.  Most rows have none and are written as
// zeros; a wave sums a row of a few tokens by itself, and the four waves a
// row of kEmbedShared or more, each a quarter of them.  SUM: the tokens of all
// ranks, rank by rank, and the row on every rank; else of the workgroup's rank.
//
// Bound by the table's writes, and by the latency of the rows that have
// tokens: 8 ranks x 4096 tokens, 32000 x 2048 bf16, written 1.05 GB: the sum
// 233 us (and 28 us of sort and partial sums), 4.5 TB/s; with no token at all
// 200-215 us.  A fill of the same memory takes 153 us.
// Rows: 32 of one rank, 16 of a sum (8 ranks x 4096 tokens, 32000 x 2048 bf16:
// each rank's 275 us against 321 with 16 rows, the sum 288 against 319 with 32).
template <bool SUM>
constexpr int embed_rows() {
  return SUM ? 16 : 32;
}
constexpr uint32_t kEmbedShared = 16;
constexpr int kEmbedWaves = kEmbedBlock / 64;

template <int DT, bool VEC, bool SUM, int B>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_grad(EmbedGradArgs a) {
  typedef Cols<DT, B> C;
  constexpr int SZ = Ty<DT>::SZ, ROWS = embed_rows<SUM>();
  extern __shared__ uint32_t runs[];   // [nr][ROWS] begin, then end
  uint32_t(*const begin)[ROWS] = (uint32_t(*)[ROWS])runs;
  __shared__ uint32_t total[ROWS];
  __shared__ float part[2][C::STEP];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r0 = SUM ? 0 : (int)blockIdx.y, nr = SUM ? a.N : 1;
  uint32_t(*const end)[ROWS] = begin + nr;
  const uint64_t v0 = blockIdx.x, dv = gridDim.x;
  const int rows = (int)((a.vocab - v0 + dv - 1) / dv);
  for (int i = threadIdx.x; i < nr * 2 * ROWS; i += kEmbedBlock) {
    const int r = i / (2 * ROWS), row = (i / 2) % ROWS;
    const uint32_t at = row < rows ? lower_bound(a.keys + (uint64_t)(r0 + r) * a.tokens, (uint32_t)a.tokens,
                                                 (uint32_t)(v0 + row * dv) + (i & 1))
                                   : 0u;
    if (i & 1) end[r][row] = at; else begin[r][row] = at;
  }
  __syncthreads();
  if (threadIdx.x < ROWS) {
    uint32_t n = 0;
    for (int r = 0; r < nr; ++r) n += end[r][threadIdx.x] - begin[r][threadIdx.x];
    total[threadIdx.x] = n;
  }
  __syncthreads();
  for (int i = wave; i < rows; i += kEmbedWaves) {
    if (total[i] >= kEmbedShared) continue;
    char* const o = a.out + (v0 + i * dv) * a.width * SZ;
    if (total[i] == 0) {
      for (int r = r0; r < r0 + nr && blockIdx.z == 0; ++r) zero_row<DT>(o + (uint64_t)r * a.os, a.width * SZ, lane);
      continue;
    }
    for (uint64_t c0 = blockIdx.z * C::STEP; c0 < a.width; c0 += gridDim.z * C::STEP) {
      float acc[C::CB][C::V] = {};
      for (int r = 0; r < nr; ++r)
        if (begin[r][i] < end[r][i]) add_rows<DT, VEC, B>(a, r0 + r, begin[r][i], end[r][i], c0, lane, acc);
      put_row<DT, VEC, B>(a, o, r0, nr, c0, lane, acc);
    }
  }
  for (int i = 0; i < rows; ++i) {
    if (total[i] < kEmbedShared) continue;
    // this wave's quarter of the tokens, counted over the ranks
    const uint32_t w0 = (uint32_t)((uint64_t)total[i] * wave / kEmbedWaves);
    const uint32_t w1 = (uint32_t)((uint64_t)total[i] * (wave + 1) / kEmbedWaves);
    for (uint64_t c0 = blockIdx.z * C::STEP; c0 < a.width; c0 += gridDim.z * C::STEP) {
      float acc[C::CB][C::V] = {};
      uint32_t before = 0;
      for (int r = 0; r < nr; ++r) {
        const uint32_t lo = begin[r][i], n = end[r][i] - lo;
        const uint32_t f = w0 > before ? w0 - before : 0, l = w1 > before ? w1 - before : 0;
        if (f < n && l) add_run<DT, VEC, B>(a, r0 + r, lo + f, lo + (l < n ? l : n), n, c0, lane, acc);
        before += n;
      }
      // join: waves 2 and 3 into 0 and 1, then 1 into 0
      for (int half = kEmbedWaves / 2; half; half >>= 1) {
        __syncthreads();   // the last parts are read
        if (wave >= half && wave < 2 * half)
#pragma unroll
          for (int k = 0; k < C::CB; ++k)
#pragma unroll
            for (int e = 0; e < C::V; ++e) part[wave - half][(k * C::V + e) * 64 + lane] = acc[k][e];
        __syncthreads();
        if (wave < half)
#pragma unroll
          for (int k = 0; k < C::CB; ++k)
#pragma unroll
            for (int e = 0; e < C::V; ++e) acc[k][e] += part[wave][(k * C::V + e) * 64 + lane];
      }
      if (wave == 0)
        put_row<DT, VEC, B>(a, a.out + (v0 + i * dv) * a.width * SZ, r0, nr, c0, lane, acc);
    }
  }
}

int compute_units() { return dev_info().cus > 0 ? dev_info().cus : 256; }

// A small table has fewer rows a workgroup, so that all compute units have some
// (8 ranks x 4096 tokens, 300 x 400 float32: 43 us against 58, the sum 54
// against 155).  Where that makes less than two workgroups a unit, a row's
// columns go to several too (the sum of 8 x 4096 tokens, 400 x 2048 bf16: 75 us
// against 121, of 8 x 100 tokens, 300 x 2048: 16 against 20).
unsigned embed_blocks(const EmbedGradArgs& a, const EmbedGradLaunch& L) {
  const uint64_t rows = L.summed ? embed_rows<true>() : embed_rows<false>();
  const uint64_t fill = (uint64_t)(4 * compute_units() / (L.summed ? 1 : L.N));
  return (unsigned)std::max((a.vocab + rows - 1) / rows, std::min(a.vocab, fill));
}
bool few_rows(const EmbedGradArgs& a, const EmbedGradLaunch& L) {
  return (uint64_t)embed_blocks(a, L) * (L.summed ? 1 : L.N) < (uint64_t)2 * compute_units();
}

template <int DT, bool VEC, int B>
hipError_t run_embed_grad(const EmbedGradArgs& a, const EmbedGradLaunch& L) {
  if (a.pieces) {
    const unsigned blocks = (unsigned)((a.pieces + kEmbedBlock / 64 - 1) / (kEmbedBlock / 64));
    CC_LAUNCH((k_embed_pieces<DT, VEC, B>), dim3(blocks, (unsigned)L.N), dim3(kEmbedBlock), 0, L.st, a);
  }
  const int rows = L.summed ? embed_rows<true>() : embed_rows<false>();
  const unsigned blocks = embed_blocks(a, L);
  const unsigned z = few_rows(a, L) ? (unsigned)std::min<uint64_t>((a.width - 1) / Cols<DT, B>::STEP + 1, 64) : 1;
  const unsigned need = (L.summed ? L.N : 1) * 2 * rows * 4;
  // A sum of wide rows written to more than 4 ranks streams best from one
  // workgroup a compute unit, once its table gives a workgroup two rows or
  // more (8 ranks x 1000 tokens, 10000 x 2048 bf16: 85 us against 99 uncapped; 4096
  // tokens, 32000 words 254 against 248; to 4 ranks of a fourth of the tokens
  // 110 either way, float32 x 1024 to 2 ranks 93 against 86).  Narrow rows and
  // small tables wait for their loads instead, and need all that fit (8 x 4096
  // tokens, 32000 x 512: 84 us against 123 with one, 400 x 2048: 75 against
  // 101; 8 x 100 tokens, 1500 x 2048: 22 against 30).  Rows of two blocks lie
  // between (10000 x 1024 bf16, 1000 tokens: 5 ranks 38 against 44, 16 ranks 107
  // against 94).
  const bool one = L.summed && L.N > 4 && B == 4 && a.vocab >= 2 * (uint64_t)blocks;
  const int blocks_per_cu = L.blocks_per_cu > 0 ? L.blocks_per_cu : one ? 1 : 0;
  const unsigned cap = lds_for_blocks_per_cu(blocks_per_cu), fixed = sizeof(float) * (2 * Cols<DT, B>::STEP + rows);
  const unsigned lds = std::max(need, cap > fixed ? cap - fixed : 0u);
  if (L.summed) CC_LAUNCH((k_embed_grad<DT, VEC, true, B>), dim3(blocks, 1, z), dim3(kEmbedBlock), lds, L.st, a);
  else CC_LAUNCH((k_embed_grad<DT, VEC, false, B>), dim3(blocks, (unsigned)L.N, z), dim3(kEmbedBlock), lds, L.st, a);
  return hipGetLastError();
}

template <int DT, bool VEC>
hipError_t pick_embed_grad(const EmbedGradArgs& a, const EmbedGradLaunch& L) {
  if (a.width <= (uint64_t)Cols<DT, 1>::STEP || few_rows(a, L)) return run_embed_grad<DT, VEC, 1>(a, L);
  if (a.width <= (uint64_t)Cols<DT, 2>::STEP) return run_embed_grad<DT, VEC, 2>(a, L);
  return run_embed_grad<DT, VEC, 4>(a, L);
}

}  // namespace

hipError_t launch_embed(const EmbedLaunch& L) {
  EmbedArgs a{L.table, L.table_stride, L.ids, L.ids_stride, L.out, L.out_stride, L.vocab, L.tokens, L.width, L.scale};
  const dim3 grid((unsigned)L.tokens, (unsigned)L.N), blk(kEmbedBlock);
  const unsigned lds = lds_for_blocks_per_cu(L.blocks_per_cu);
  if (L.dt == DT_F32) {
    if (L.vec_ok) CC_LAUNCH((k_embed<DT_F32, true>), grid, blk, lds, L.st, a);
    else CC_LAUNCH((k_embed<DT_F32, false>), grid, blk, lds, L.st, a);
  } else {
    if (L.vec_ok) CC_LAUNCH((k_embed<DT_BF16, true>), grid, blk, lds, L.st, a);
    else CC_LAUNCH((k_embed<DT_BF16, false>), grid, blk, lds, L.st, a);
  }
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradLaunch& L) {
  EmbedGradArgs a{L.grad, L.grad_stride, L.out, L.out_stride, L.keys, L.vals, L.partial,
                  L.vocab, L.tokens, L.width, embed_partial_pitch(L.width), embed_pieces(L.tokens), L.scale, L.N};
  if (L.dt == DT_F32) return L.vec_ok ? pick_embed_grad<DT_F32, true>(a, L) : pick_embed_grad<DT_F32, false>(a, L);
  return L.vec_ok ? pick_embed_grad<DT_BF16, true>(a, L) : pick_embed_grad<DT_BF16, false>(a, L);
}

}  // namespace cc
