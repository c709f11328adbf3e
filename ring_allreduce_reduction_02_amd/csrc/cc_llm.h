// Internal interface between the C ABI of the model-side operators
// (cc_model.cpp) and their kernels (cc_sort.hip, cc_embed.hip, cc_route.hip,
// cc_ffn.hip).  Host-side only; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cc_ffn_rule.h"
#include "cc_launch.h"

namespace cc {

// ---- stable sort of each rank's n int32 keys with their positions.  Keys
// outside [0, nkeys) sort last, as the key nkeys.
struct SortPlan {
  int N;
  uint64_t n;        // keys per rank, < 2^31
  uint32_t nkeys;
  int passes;        // of 8 bits
  uint64_t tiles;    // per rank and pass; 0: one workgroup sorts a rank's keys in LDS
  uint64_t bytes;    // of workspace
};
SortPlan sort_plan(int N, uint64_t n, uint32_t nkeys);
struct SortLaunch {
  SortPlan p;
  const char* keys;      // rank-strided
  uint64_t key_stride;
  char* ws;              // p.bytes, 16-byte aligned
  // Without `counts`: sorted keys and their positions, [N][n] int32 inside ws
  const int* sorted_keys;
  const int* sorted_vals;
  // With it (both rank-strided): the positions, -1 for keys outside [0, nkeys), and
  // the number of each key
  char* order;
  uint64_t order_stride;
  char* counts;
  uint64_t counts_stride;
  hipStream_t st;
};
hipError_t launch_sort(SortLaunch* L);

// ---- embedding
struct EmbedLaunch {
  const char* table;
  uint64_t table_stride;
  const char* ids;
  uint64_t ids_stride;
  char* out;
  uint64_t out_stride;
  uint64_t vocab, tokens, width;
  float scale;
  int N, dt, vec_ok, blocks_per_cu;
  hipStream_t st;
};
hipError_t launch_embed(const EmbedLaunch& L);

// Sorted positions per partial sum of a long run, the shortest run that has
// them, and how many a rank's tokens have; none up to 1024 tokens, where a
// workgroup sums a whole run itself in the time of the extra launch.
constexpr int kEmbedPiece = 32;
constexpr uint32_t kEmbedLong = 128;
inline uint64_t embed_partial_pitch(uint64_t width) { return (width + 7) / 8 * 8; }
inline uint64_t embed_pieces(uint64_t tokens) { return tokens > 1024 ? tokens / kEmbedPiece : 0; }
struct EmbedGradLaunch {
  const char* grad;
  uint64_t grad_stride;
  char* out;
  uint64_t out_stride;
  const int* keys;       // sorted, [N][tokens]
  const int* vals;
  float* partial;        // [N][embed_pieces][embed_partial_pitch]
  uint64_t vocab, tokens, width;
  float scale;
  int N, dt, vec_ok, blocks_per_cu;
  int summed;            // over all ranks, the result on every rank
  hipStream_t st;
};
hipError_t launch_embed_grad(const EmbedGradLaunch& L);

// ---- MoE routing
constexpr int kMaxRouteExperts = 1024;
struct RouteLaunch {
  const char* logits;
  uint64_t logits_stride;
  char* experts;         // int32 [tokens][topk]
  uint64_t experts_stride;
  char* weights;         // float32 [tokens][topk]; dweights of the gradient
  uint64_t weights_stride;
  char* dlogits;
  uint64_t dlogits_stride;
  uint64_t tokens;
  int nexperts, topk, normalize;
  int N, dt;
  hipStream_t st;
};
hipError_t launch_route(const RouteLaunch& L);
hipError_t launch_route_grad(const RouteLaunch& L);

// ---- gated feed-forward block of the experts.  Compact rows: the kept rows
// of all experts back to back, expert by expert, source by source.
// Workspace: row starts [E + 1], row tiles of each size (expert, first row), row
// map [rows] (row in the rank's buffer), kept counts [N * E], h [rows][F],
// and for the gradient d(gate | up) [rows][2F].  Where rows are no whole
// 16-byte vectors it may hold aligned copies, lines padded with zeros to 128
// bytes (h and d(gate | up) then too): x and dy by compact rows, the weights.
struct FfnWs {
  uint64_t kept, start, mtab[kFfnTiles], rowmap, h, dgu, bytes;
  int copied;
  uint64_t x, dy, w_in, w_out;
};
FfnWs ffn_ws(const FfnShape& s, int grad);
struct FfnLaunch {
  FfnShape s;
  FfnWs o;
  char* ws;
  const uint32_t* kept;  // host, [E][N]: kept rows of expert e from source i
  Side x, w_in, w_out, pre, y;      // pre.base may be NULL (forward)
  Side dy, dx, dw_in, dw_out;       // gradient
  int vec_ok;
  hipStream_t st;
};
hipError_t launch_ffn(const FfnLaunch& L);
hipError_t launch_ffn_grad(const FfnLaunch& L);

}  // namespace cc
