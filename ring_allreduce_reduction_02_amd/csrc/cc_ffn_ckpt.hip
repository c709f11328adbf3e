// The experts' feed-forward block with its activations kept in 8 bits
// (cc_ckpt.h): the products that write and read them, and the rows x.

#include "cc_ffn_tile.h"

namespace cc {
namespace {

struct XArgs {
  const int* start;
  const int2* mtab;      // row tiles of 64
  const int* map;
  int per;
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
};

constexpr int kXParts = 16, kXRows = kFfnTile[kFfnTiles - 1] / kXParts;   // workgroups of a tile of 64 rows

// The compact rows of a workgroup, a wave each.
struct XRows {
  int first, end, rank;
};
__device__ __forceinline__ XRows rows_of_block(const XArgs& a) {
  const int2 at = a.mtab[blockIdx.x / kXParts];
  const int stop = a.start[at.x + 1], first = at.y + (int)(blockIdx.x % kXParts) * kXRows;
  return XRows{first, first + kXRows < stop ? first + kXRows : stop, at.x / a.per};
}

// A lane takes V consecutive elements, so that 32 / V lanes hold a block.
template <int DT>
__global__ __launch_bounds__(256) void k_ckpt_pack(XArgs a) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const XRows b = rows_of_block(a);
  for (int l = b.first + wave; l < b.end; l += 4) {
    const uint64_t row = (uint64_t)(uint32_t)a.map[l];
    const char* x = a.x + (uint64_t)b.rank * a.x_stride + row * a.W * SZ;
    char* ck = a.ck + (uint64_t)b.rank * a.ck_stride + row * (uint64_t)a.at.pitch;
    for (uint64_t c0 = 0; c0 < a.W; c0 += 64 * V) {
      const uint64_t c = c0 + (uint64_t)lane * V;
      const int left = (int)((int64_t)a.W - (int64_t)c < V ? (int64_t)a.W - (int64_t)c : V);
      float v[V];
      unpack<DT>(load_n<DT, false>(x + c * SZ, left), v);
      kept_store<V, kCkptBlock / V>(v, left, lane, ck + a.at.x + c, ck + a.at.xe + c / kCkptBlock);
    }
  }
}

// The kept values as rows of the matrix products' type, exact in either (7
// significant bits, no exponent below -126); zeros up to the pitch.
template <int DT>
__global__ __launch_bounds__(256) void k_ckpt_unpack(XArgs a) {
  constexpr int V = Ty<DT>::V, SZ = Ty<DT>::SZ;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const XRows b = rows_of_block(a);
  for (int l = b.first + wave; l < b.end; l += 4) {
    const uint64_t row = (uint64_t)(uint32_t)a.map[l];
    const char* ck = a.ck + (uint64_t)b.rank * a.ck_stride + row * (uint64_t)a.at.pitch;
    char* x = a.x + (uint64_t)l * a.pitch;
    for (uint64_t c = (uint64_t)lane * V; c * SZ < a.pitch; c += 64 * V) {
      const int64_t left = (int64_t)a.W - (int64_t)c;
      float v[V] = {};
      if (left > 0) {
        kept_unpack<V>(kept_load<V>(ck + a.at.x + c, ck + a.at.xe + c / kCkptBlock), v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < left ? v[i] : 0.0f;
      }
      const int64_t room = (int64_t)(a.pitch / SZ) - (int64_t)c;
      store_n<DT, false, V>(x + c * SZ, v, (int)(room < V ? room : V));
    }
    if (a.h) {
      for (uint64_t c = a.F * SZ + lane * SZ; c < a.h_pitch; c += 64 * SZ) st1<DT>(a.h + l * a.h_pitch + c, 0.0f);
      for (uint64_t c = 2 * a.F * SZ + lane * SZ; c < a.dgu_pitch; c += 64 * SZ)
        st1<DT>(a.dgu + l * a.dgu_pitch + c, 0.0f);
    }
  }
}

XArgs x_args(const FfnLaunch& L, const Side& x) {
  XArgs a = {};
  a.start = (const int*)(L.ws + L.o.start);
  a.mtab = (const int2*)(L.ws + L.o.mtab[kFfnTiles - 1]);
  a.map = (const int*)(L.ws + L.o.rowmap);
  a.per = L.s.E / L.s.N;
  a.ck = L.ckpt.base;
  a.ck_stride = L.ckpt.stride;
  a.at = ckpt_row(L.s.W, L.s.F);
  a.x = x.base;
  a.x_stride = x.stride;
  a.W = L.s.W;
  return a;
}

}  // namespace

hipError_t ckpt_gateup(const CkArgs& g, const FfnLaunch& L) { return pick_gemm<K_GATEUP_CK>(g, L); }
hipError_t ckpt_dhid(const CkArgs& g, const FfnLaunch& L) { return pick_gemm<K_DHID_CK>(g, L); }

hipError_t ckpt_pack_x(const FfnLaunch& L) {
  const uint64_t tiles = L.s.mtiles[kFfnTiles - 1];
  if (tiles == 0) return hipSuccess;
  const XArgs a = x_args(L, L.x);
  const dim3 grid((unsigned)(kXParts * tiles)), blk(256);
  if (L.s.dt == DT_F32) CC_LAUNCH(k_ckpt_pack<DT_F32>, grid, blk, 0, L.st, a);
  else CC_LAUNCH(k_ckpt_pack<DT_BF16>, grid, blk, 0, L.st, a);
  return hipGetLastError();
}

hipError_t ckpt_unpack_x(const FfnLaunch& L) {
  const uint64_t tiles = L.s.mtiles[kFfnTiles - 1];
  if (tiles == 0) return hipSuccess;
  XArgs a = x_args(L, Side{L.ws + L.o.x, 0});
  a.pitch = L.o.copied ? line_pitch(L.s, L.s.W) : L.s.W * elem_size(L.s.dt);
  if (L.o.copied) {
    a.h = L.ws + L.o.h;
    a.dgu = L.ws + L.o.dgu;
    a.F = L.s.F;
    a.h_pitch = line_pitch(L.s, L.s.F);
    a.dgu_pitch = line_pitch(L.s, 2 * L.s.F);
  }
  const dim3 grid((unsigned)(kXParts * tiles)), blk(256);
  if (L.s.dt == DT_F32) CC_LAUNCH(k_ckpt_unpack<DT_F32>, grid, blk, 0, L.st, a);
  else CC_LAUNCH(k_ckpt_unpack<DT_BF16>, grid, blk, 0, L.st, a);
  return hipGetLastError();
}

}  // namespace cc
