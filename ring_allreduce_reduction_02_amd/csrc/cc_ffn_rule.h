// Which form the products of the expert feed-forward block run in: on the
// caller's operands, on padded copies of them, or through registers, and in
// tiles of which size.  Free of HIP, so that a host test can compile it and
// see which kernels its cases reach.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace cc {

constexpr int kFfnTiles = 3;            // tile sizes (rows and columns) of the products
constexpr int kFfnTile[kFfnTiles] = {256, 128, 64};
struct FfnShape {
  int N, E;              // ranks, experts
  uint64_t cap;
  uint64_t W, F;         // width, hidden
  uint64_t rows, most;   // kept rows of all experts, and of the one with most
  uint64_t mtiles[kFfnTiles];   // row tiles of all experts, of each size
  int dt, es, act;       // element type, its bytes, activation
};

enum Kind { K_GATEUP = 0, K_DOWN = 1, K_DHID = 2, K_DX = 3, K_DW = 4 };

constexpr uint64_t kMaxSpan = 0xfff00000ull;   // bytes that the direct loads' 32-bit offsets reach

inline uint64_t line_pitch(const FfnShape& s, uint64_t cols) {   // whole cache lines
  return (cols * s.es + 127) / 128 * 128;
}

// Whether the operands are first copied into rows that direct loads can take:
// whole 16-byte vectors, padded with zeros, the experts' rows compact.  For
// rows that are none, or a side that 32-bit offsets do not reach.  (Rows of
// whole vectors on a base or rank stride that is none are not copied: they go
// through registers.)
// Gradients of such rows always: 1.04 to 2.7 times faster than the tiles through
// registers over 1 to 8192 rows an expert and 201 x 333 to 2047 x 2047 of both
// types (16 experts, 2047 x 2047 bf16, 4 rows an expert 461 us against 747, 4096
// rows 3605 against 10002).  The forward pass reads every operand once along
// its rows, where the tiles through registers do better, so that the copies
// pay from about 1024 rows an expert and 512 columns on: 2047 x 2047 bf16 128
// rows 378 us against 285, 512 rows 504 against 507, 2048 rows 1072 against 1665;
// 300 x 517 bf16 2048 rows 118 against 121, 201 x 333 float32 236 against 213.
constexpr uint64_t kCopyRows = 1024, kCopyCols = 512;
inline bool ffn_copied(const FfnShape& s, int grad) {
  const uint64_t es = s.es, w = line_pitch(s, s.W), f = line_pitch(s, s.F), f2 = line_pitch(s, 2 * s.F);
  if (s.rows == 0 || (s.W * es % 16 == 0 && s.F * es % 16 == 0 && s.E * s.cap * s.W * es <= kMaxSpan)) return false;
  if (s.most * std::max(w, f2) > kMaxSpan || 2 * s.F * w > kMaxSpan || s.W * f > kMaxSpan) return false;
  return grad || (s.rows >= kCopyRows * s.E && std::min(s.W, s.F) >= kCopyCols);
}

// Whether the products run as tiles by direct loads: on copies, or on rows of
// whole 16-byte vectors (`vec_ok`, bases and rank strides too) that 32-bit
// offsets reach.
inline bool ffn_tiled(const FfnShape& s, bool copied, bool vec_ok) {
  if (copied) return true;
  const uint64_t es = s.es, row = std::max(s.W, 2 * s.F) * es;
  return vec_ok && (uint64_t)s.E * s.cap * s.W * es <= kMaxSpan && s.most * row <= kMaxSpan &&
         2 * s.F * s.W * es <= kMaxSpan;
}

// A product's tiles of size kFfnTile[k]: mt x nt, and (K_DW, an M x N result of
// every expert) of all experts.  `cols`: the result's columns; K_GATEUP: of each
// half, half a tile of them in a tile.
struct FfnGrid {
  uint64_t mt, nt, blocks;
};
inline FfnGrid ffn_grid(const FfnShape& s, int kind, uint64_t M, uint64_t cols, int k) {
  const uint64_t t = kFfnTile[k], bn = kind == K_GATEUP ? t / 2 : t;
  FfnGrid g;
  g.nt = (cols + bn - 1) / bn;
  g.mt = kind == K_DW ? (M + t - 1) / t : s.mtiles[k];
  g.blocks = g.mt * g.nt * (kind == K_DW ? s.E : 1);
  return g;
}

// The tile whose workgroups, dealt out over the compute units, take least: a
// larger tile moves fewer bytes for a product, a smaller one leaves fewer
// units idle.  Cost of equal areas, measured on all six products of 60.7k rows:
// bf16 2048 x 2048 1, 1.21 and 1.92 (4.62, 5.62 and 8.87 ms), float32, whose
// products take eight times as long, 1024 x 1024 1, 1 and 1.25 (9.79, 9.81 and
// 12.24 ms; the weight gradients alone 1, 1 and 1.35, which is counted).  The
// tiles through registers have the last two sizes.
inline int ffn_pick_tile(const FfnShape& s, int kind, uint64_t M, uint64_t cols, bool fast, int cus) {
  constexpr double kArea[2][kFfnTiles] = {{16.0, 4.0 * 1.21, 1.92}, {16.0, 4.0, 1.35}};
  const int first = fast ? 0 : 1;
  int best = first;
  double least = 0.0;
  for (int k = first; k < kFfnTiles; ++k) {
    const double t = (double)((ffn_grid(s, kind, M, cols, k).blocks + cus - 1) / cus) * kArea[s.es == 4][k];
    if (k == first || t < least) {
      least = t;
      best = k;
    }
  }
  return best;
}

}  // namespace cc
