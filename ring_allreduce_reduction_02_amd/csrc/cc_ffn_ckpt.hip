// The experts' feed-forward block with its activations kept in 8 bits
// (cc_ckpt.h): the products that write and read them, and the rows x.

#include "cc_ffn_tile.h"

namespace cc {
namespace {

struct XRows {
  char* ck;
  uint64_t ck_stride;
  CkptRow at;
  char* x;               // in the ranks' buffers (pack), compact (unpack)
  uint64_t x_stride, pitch;
  uint64_t W;
  // unpack, where the products read padded copies: the padding of the rows between them (NULL: none)
  char* h;
  char* dgu;
  uint64_t F, h_pitch, dgu_pitch;
  int per;               // experts a rank
  const int* start;
  const int2* mtab;
  const int* map;
};

// A kept row x into the checkpoint, by a wave.  A lane takes V consecutive
// elements, so that 32 / V lanes hold a block.
template <int DT>
__device__ __forceinline__ void pack_x(const XRows& a, uint64_t rank, uint32_t row) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int lane = threadIdx.x & 63;
  const char* x = a.x + rank * a.x_stride + (uint64_t)row * a.W * SZ;
  char* ck = a.ck + rank * a.ck_stride + (uint64_t)row * (uint64_t)a.at.pitch;
  for (uint64_t c0 = 0; c0 < a.W; c0 += 4 * 64 * V) {   // four loads under way
    u32x4 w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t c = c0 + (uint64_t)(q * 64 + lane) * V;
      w[q] = load_line<DT>(x, a.W, c);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t c = c0 + (uint64_t)(q * 64 + lane) * V;
      const int64_t left = (int64_t)a.W - (int64_t)c;
      float v[V];
      unpack<DT>(w[q], v);
      if (c0 + q * 64 * V < a.W)   // the same on all lanes
        kept_store<V, kCkptBlock / V>(v, (int)(left < V ? left : V), lane, ck + a.at.x + c, ck + a.at.xe + c / kCkptBlock);
    }
  }
}

// A row's kept values as one of the matrix products' type, exact in either (7
// significant bits, no exponent below -126); zeros up to the pitch.
template <int DT>
__device__ __forceinline__ void unpack_x(const XRows& a, uint64_t rank, uint32_t row, uint64_t to) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int lane = threadIdx.x & 63;
  const char* ck = a.ck + rank * a.ck_stride + (uint64_t)row * (uint64_t)a.at.pitch;
  char* x = a.x + to * a.pitch;
  for (uint64_t c0 = (uint64_t)lane * V; c0 * SZ < a.pitch; c0 += 4 * 64 * V) {   // four loads under way
    Kept<V> k[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t c = c0 + q * 64 * V;
      if (c < a.W) k[q] = kept_load<V>(ck + a.at.x + c, ck + a.at.xe + c / kCkptBlock);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t c = c0 + q * 64 * V;
      const int64_t left = (int64_t)a.W - (int64_t)c, room = (int64_t)(a.pitch / SZ) - (int64_t)c;
      float v[V] = {};
      if (left > 0) {
        kept_unpack<V>(k[q], v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < left ? v[i] : 0.0f;
      }
      if (room > 0) store_n<DT, false, V>(x + c * SZ, v, (int)(room < V ? room : V));
    }
  }
  if (a.h) {
    for (uint64_t c = a.F * SZ + lane * SZ; c < a.h_pitch; c += 64 * SZ) st1<DT>(a.h + to * a.h_pitch + c, 0.0f);
    for (uint64_t c = 2 * a.F * SZ + lane * SZ; c < a.dgu_pitch; c += 64 * SZ)
      st1<DT>(a.dgu + to * a.dgu_pitch + c, 0.0f);
  }
}

// Both are bound by memory: 60.7k rows of 2048 bf16 83 and 65 us, at best 73 and 63, 5.2
// and 6.0 TB/s.
// (In one kernel with the plan, whose counts lie in the host's memory, the whole
// step of 64 to 32768 rows took 0-4% less where few rows, 0-2% more where many.)
template <int DT, bool UNPACK>
__global__ __launch_bounds__(256) void k_ckpt_x(XRows a) {
  table_rows(a.start, a.mtab, a.map, [&](uint32_t l, uint32_t row, int e) {
    if constexpr (UNPACK) unpack_x<DT>(a, (uint64_t)(e / a.per), row, l);
    else pack_x<DT>(a, (uint64_t)(e / a.per), row);
  });
}

template <bool UNPACK>
hipError_t run_x(const XRows& a, const FfnLaunch& L) {
  const uint64_t tiles = L.s.mtiles[kFfnTiles - 1];
  if (tiles == 0) return hipSuccess;
  const dim3 grid((unsigned)tiles, kTileParts), blk(256);
  if (L.s.dt == DT_F32) CC_LAUNCH((k_ckpt_x<DT_F32, UNPACK>), grid, blk, 0, L.st, a);
  else CC_LAUNCH((k_ckpt_x<DT_BF16, UNPACK>), grid, blk, 0, L.st, a);
  return hipGetLastError();
}

XRows x_rows(const FfnLaunch& L, const Side& x) {
  XRows a = {};
  a.ck = L.ckpt.base;
  a.ck_stride = L.ckpt.stride;
  a.at = ckpt_row(L.s.W, L.s.F);
  a.x = x.base;
  a.x_stride = x.stride;
  a.W = L.s.W;
  a.per = L.s.E / L.s.N;
  a.start = (const int*)(L.ws + L.o.start);
  a.mtab = (const int2*)(L.ws + L.o.mtab[kFfnTiles - 1]);
  a.map = (const int*)(L.ws + L.o.rowmap);
  return a;
}

}  // namespace

hipError_t ckpt_gateup(const CkArgs& g, const FfnLaunch& L) { return pick_gemm<K_GATEUP_CK>(g, L); }
hipError_t ckpt_dhid(const CkArgs& g, const FfnLaunch& L) { return pick_gemm<K_DHID_CK>(g, L); }

hipError_t ckpt_pack_x(const FfnLaunch& L) { return run_x<false>(x_rows(L, L.x), L); }

hipError_t ckpt_unpack_x(const FfnLaunch& L) {
  XRows a = x_rows(L, Side{L.ws + L.o.x, 0});
  a.pitch = L.o.copied ? line_pitch(L.s, L.s.W) : L.s.W * elem_size(L.s.dt);
  if (L.o.copied) {
    a.h = L.ws + L.o.h;
    a.dgu = L.ws + L.o.dgu;
    a.F = L.s.F;
    a.h_pitch = line_pitch(L.s, L.s.F);
    a.dgu_pitch = line_pitch(L.s, 2 * L.s.F);
  }
  return run_x<true>(a, L);
}

}  // namespace cc
