// Embedding lookup with scaling, and the table's gradient from the sorted
// tokens: of each rank, or summed over the ranks onto every rank.
//
//   out[t, :] = scale * table[ids[t], :]            (zeros where ids[t] is no row)
//   d[v, :]   = scale * sum over t with ids[t] = v of grad[t, :]
//
// Both are one pass over memory: the lookup reads and writes tokens * width
// elements, the gradient reads tokens * width and writes all vocab * width
// (most rows are zeros: a batch holds few of a vocabulary's words).

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

// One workgroup a token row and rank.
template <int DT, bool VEC>
__global__ __launch_bounds__(kEmbedBlock) void k_embed(EmbedArgs a) {
  const uint64_t t = blockIdx.x, r = blockIdx.y;
  const int id = ((const int*)(a.ids + r * a.is))[t];
  const bool in = (uint32_t)id < a.vocab;
  char* o = a.out + r * a.os + t * a.width * Ty<DT>::SZ;
  const char* s = a.table + r * a.ts + (in ? (uint64_t)id : 0) * a.width * Ty<DT>::SZ;
  constexpr int V = VEC ? Ty<DT>::V : 1;
  for (uint64_t c = (uint64_t)threadIdx.x * V; c < a.width; c += kEmbedBlock * V) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = 0.0f;
    if constexpr (VEC) {
      if (in) {
        unpack<DT>(*(const u32x4*)(s + c * Ty<DT>::SZ), x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] *= a.scale;
      }
      *(u32x4*)(o + c * Ty<DT>::SZ) = pack<DT>(x);
    } else {
      if (in) x[0] = ld1<DT>(s + c * Ty<DT>::SZ) * a.scale;
      st1<DT>(o + c * Ty<DT>::SZ, x[0]);
    }
  }
}

struct EmbedGradArgs {
  const char* grad;
  uint64_t gs;
  char* out;
  uint64_t os;
  const int* keys;
  const int* vals;
  float* partial;
  uint64_t n;
  uint64_t vocab, tokens, width;
  uint64_t pieces;   // n / kEmbedPiece
  float scale;
  int N;
};

// The grad row of sorted position p in segment seg: a summed segment holds
// all ranks' tokens, rank by rank.
template <int DT, bool SUM>
__device__ __forceinline__ const char* grad_row(const EmbedGradArgs& a, uint64_t seg, int val) {
  uint64_t r = seg, t = (uint32_t)val;
  if constexpr (SUM) {
    r = (uint32_t)val / (uint32_t)a.tokens;
    t = (uint32_t)val - (uint32_t)r * (uint32_t)a.tokens;
  }
  return a.grad + r * a.gs + t * a.width * Ty<DT>::SZ;
}

template <int DT, bool VEC, bool SUM>
__device__ __forceinline__ void add_rows(const EmbedGradArgs& a, uint64_t seg, uint64_t lo, uint64_t hi, uint64_t c,
                                         float* acc) {
  constexpr int V = VEC ? Ty<DT>::V : 1;
  const int* vals = a.vals + seg * a.n;
  for (uint64_t p = lo; p < hi; ++p) {
    const char* g = grad_row<DT, SUM>(a, seg, vals[p]) + c * Ty<DT>::SZ;
    if constexpr (VEC) {
      float x[V];
      unpack<DT>(*(const u32x4*)g, x);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += x[i];
    } else {
      acc[0] += ld1<DT>(g);
    }
  }
}

// Partial sums of the pieces (kEmbedPiece sorted positions) that lie inside
// one word's run, so that a frequent word is summed by many workgroups.
template <int DT, bool VEC, bool SUM>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_pieces(EmbedGradArgs a) {
  const uint64_t piece = blockIdx.x, seg = blockIdx.y;
  const uint64_t p0 = piece * kEmbedPiece;
  const int* keys = a.keys + seg * a.n;
  const uint32_t k = (uint32_t)keys[p0];
  if (k >= a.vocab || k != (uint32_t)keys[p0 + kEmbedPiece - 1]) return;
  float* o = a.partial + (seg * a.pieces + piece) * a.width;
  constexpr int V = VEC ? Ty<DT>::V : 1;
  for (uint64_t c = (uint64_t)threadIdx.x * V; c < a.width; c += kEmbedBlock * V) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    add_rows<DT, VEC, SUM>(a, seg, p0, p0 + kEmbedPiece, c, acc);
#pragma unroll
    for (int i = 0; i < V; ++i) o[c + i] = acc[i];
  }
}

// first sorted position whose key is at least k
__device__ __forceinline__ uint64_t lower_bound(const int* keys, uint64_t n, uint32_t k) {
  uint64_t lo = 0, hi = n;
  while (lo < hi) {
    const uint64_t mid = (lo + hi) >> 1;
    if ((uint32_t)keys[mid] < k) lo = mid + 1; else hi = mid;
  }
  return lo;
}

constexpr int kEmbedRows = 8;   // table rows per workgroup

template <int DT, bool VEC, bool SUM>
__global__ __launch_bounds__(kEmbedBlock) void k_embed_grad(EmbedGradArgs a) {
  __shared__ uint64_t begin[kEmbedRows + 1];
  const uint64_t seg = blockIdx.y, v0 = (uint64_t)blockIdx.x * kEmbedRows;
  if (threadIdx.x <= kEmbedRows) begin[threadIdx.x] = lower_bound(a.keys + seg * a.n, a.n, (uint32_t)(v0 + threadIdx.x));
  __syncthreads();
  const int rows = (int)(a.vocab - v0 < kEmbedRows ? a.vocab - v0 : kEmbedRows);
  constexpr int V = VEC ? Ty<DT>::V : 1;
  for (int i = 0; i < rows; ++i) {
    const uint64_t lo = begin[i], hi = begin[i + 1];
    // whole pieces of a long run come as their partial sums
    const uint64_t f = (lo + kEmbedPiece - 1) / kEmbedPiece, l = hi / kEmbedPiece;
    for (uint64_t c = (uint64_t)threadIdx.x * V; c < a.width; c += kEmbedBlock * V) {
      float acc[V];
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = 0.0f;
      if (f < l) {
        add_rows<DT, VEC, SUM>(a, seg, lo, f * kEmbedPiece, c, acc);
        for (uint64_t p = f; p < l; ++p)
#pragma unroll
          for (int q = 0; q < V; ++q) acc[q] += a.partial[(seg * a.pieces + p) * a.width + c + q];
        add_rows<DT, VEC, SUM>(a, seg, l * kEmbedPiece, hi, c, acc);
      } else {
        add_rows<DT, VEC, SUM>(a, seg, lo, hi, c, acc);
      }
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] *= a.scale;
      const uint64_t at = ((v0 + i) * a.width + c) * Ty<DT>::SZ;
      const int r0 = SUM ? 0 : (int)seg, r1 = SUM ? a.N : r0 + 1;
      for (int r = r0; r < r1; ++r) {
        char* o = a.out + (uint64_t)r * a.os + at;
        if constexpr (VEC) *(u32x4*)o = pack<DT>(acc);
        else st1<DT>(o, acc[0]);
      }
    }
  }
}

template <int DT, bool VEC, bool SUM>
hipError_t run_embed_grad(const EmbedGradArgs& a, const EmbedGradLaunch& L) {
  const unsigned segs = SUM ? 1 : (unsigned)L.N;
  if (a.pieces)
    CC_LAUNCH((k_embed_pieces<DT, VEC, SUM>), dim3((unsigned)a.pieces, segs), dim3(kEmbedBlock), 0, L.st, a);
  const unsigned blocks = (unsigned)((a.vocab + kEmbedRows - 1) / kEmbedRows);
  CC_LAUNCH((k_embed_grad<DT, VEC, SUM>), dim3(blocks, segs), dim3(kEmbedBlock), 0, L.st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedLaunch& L) {
  EmbedArgs a{L.table, L.table_stride, L.ids, L.ids_stride, L.out, L.out_stride, L.vocab, L.tokens, L.width, L.scale};
  const dim3 grid((unsigned)L.tokens, (unsigned)L.N), blk(kEmbedBlock);
  if (L.dt == DT_F32) {
    if (L.vec_ok) CC_LAUNCH((k_embed<DT_F32, true>), grid, blk, 0, L.st, a);
    else CC_LAUNCH((k_embed<DT_F32, false>), grid, blk, 0, L.st, a);
  } else {
    if (L.vec_ok) CC_LAUNCH((k_embed<DT_BF16, true>), grid, blk, 0, L.st, a);
    else CC_LAUNCH((k_embed<DT_BF16, false>), grid, blk, 0, L.st, a);
  }
  return hipGetLastError();
}

hipError_t launch_embed_grad(const EmbedGradLaunch& L) {
  EmbedGradArgs a{L.grad, L.grad_stride, L.out, L.out_stride, L.keys, L.vals, L.partial, L.n,
                  L.vocab, L.tokens, L.width, L.n / kEmbedPiece, L.scale, L.N};
  if (L.dt == DT_F32) {
    if (L.vec_ok) return L.summed ? run_embed_grad<DT_F32, true, true>(a, L) : run_embed_grad<DT_F32, true, false>(a, L);
    return L.summed ? run_embed_grad<DT_F32, false, true>(a, L) : run_embed_grad<DT_F32, false, false>(a, L);
  }
  if (L.vec_ok) return L.summed ? run_embed_grad<DT_BF16, true, true>(a, L) : run_embed_grad<DT_BF16, true, false>(a, L);
  return L.summed ? run_embed_grad<DT_BF16, false, true>(a, L) : run_embed_grad<DT_BF16, false, false>(a, L);
}

}  // namespace cc
