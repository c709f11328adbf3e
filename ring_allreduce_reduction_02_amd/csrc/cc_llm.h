// Internal interface between the C ABI of the model-side operators
// (cc_model.cpp) and their kernels (cc_sort.hip, cc_embed.hip, cc_route.hip,
// cc_balance.hip, cc_ffn.hip, cc_ffn_ckpt.hip, cc_int8.hip).  Host-side only; not
// installed.
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

// ---- balance loss of the routing
constexpr int kBalanceBlock = 256;
struct BalanceLaunch {
  const char* logits;
  uint64_t logits_stride;
  const char* counts;    // int32 [nexperts]
  uint64_t counts_stride;
  char* total;           // int32 [nexperts + 1]; the gradient's input
  uint64_t total_stride;
  char* prob;            // float32 [nexperts]
  uint64_t prob_stride;
  char* loss;            // float32; dloss of the gradient
  uint64_t loss_stride;
  const char* base;      // the gradient's addend, or NULL
  uint64_t base_stride;
  char* dlogits;
  uint64_t dlogits_stride;
  char* ws;
  uint64_t tokens;
  int nexperts, summed;
  int N, dt;
  hipStream_t st;
};
uint64_t balance_ws(int N, uint64_t tokens, int nexperts);
hipError_t launch_balance(const BalanceLaunch& L);
hipError_t launch_balance_grad(const BalanceLaunch& L);

// ---- a checkpoint row: x, gate and up integers, each part on a multiple of 16
// bytes, then the exponents of their blocks
constexpr int kCkptBlock = 32;
struct CkptRow {
  int x, g, u, xe, ge, ue, pitch;
};
inline CkptRow ckpt_row(uint64_t W, uint64_t F) {
  auto up = [](uint64_t v) { return (int)((v + 15) / 16 * 16); };
  auto blocks = [](uint64_t v) { return (int)((v + kCkptBlock - 1) / kCkptBlock); };
  CkptRow r;
  r.x = 0;
  r.g = up(W);
  r.u = r.g + up(F);
  r.xe = r.u + up(F);
  r.ge = r.xe + blocks(W);
  r.ue = r.ge + blocks(F);
  r.pitch = up((uint64_t)r.ue + blocks(F));
  return r;
}

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
// `ckpt`: the gradient's rows x come from checkpoints, unpacked into the workspace
FfnWs ffn_ws(const FfnShape& s, int grad, int ckpt = 0);
struct FfnLaunch {
  FfnShape s;
  FfnWs o;
  char* ws;
  const uint32_t* kept;  // host, [E][N]: kept rows of expert e from source i
  Side x, w_in, w_out, pre, y;      // pre.base may be NULL (forward)
  Side dy, dx, dw_in, dw_out;       // gradient
  Side ckpt;                        // checkpoint rows in x's layout (base NULL: none)
  int vec_ok;
  hipStream_t st;
};
hipError_t launch_ffn(const FfnLaunch& L);
hipError_t launch_ffn_grad(const FfnLaunch& L);
// the plan alone: o.kept, o.start, o.mtab and o.rowmap
hipError_t launch_ffn_plan(const FfnShape& s, const FfnWs& o, char* ws, const uint32_t* kept, hipStream_t st);

// the parts of the block that keep or read a checkpoint (cc_ffn_ckpt.hip)
struct CkArgs;
hipError_t ckpt_gateup(const CkArgs& g, const FfnLaunch& L);
hipError_t ckpt_dhid(const CkArgs& g, const FfnLaunch& L);
hipError_t ckpt_pack_x(const FfnLaunch& L);
hipError_t ckpt_unpack_x(const FfnLaunch& L);   // into the workspace

// ---- 8-bit integers: rows and their scales, grouped products
struct Int8Rows {
  const char* x;         // rows of `width` elements, rank-strided
  uint64_t x_stride;
  char* q;               // rows of q_pitch bytes, zeros past the width
  uint64_t q_stride, q_pitch;
  char* s;               // a float32 a row
  uint64_t s_stride;
  uint64_t rows, width;
  int N, dt;
  int product;           // the scale: max|x| times 1 / 127 (1), or max|x| / 127 (0)
  hipStream_t st;
};
hipError_t launch_int8_rows(const Int8Rows& L);
// Workspace: the plan's tables; of the block the rows x and h in 8 bits (lines
// padded with zeros to 128 bytes), their scales and h; and where a product's rows
// are no whole 16-byte vectors it may hold copies in such lines: of the weights,
// and of the product's rows.
struct Int8Ws {
  FfnWs plan;
  uint64_t xq, xs, h, hq, hs, bytes;
  uint64_t xq_pitch, hq_pitch;
  int copied_in, copied_out;
  uint64_t w_in, w_out;
};
Int8Ws int8_ws(const FfnShape& s, int block, int out_es);
struct Int8Launch {
  FfnShape s;            // element size 1; W summed, F the product's columns, or the block's hidden size
  Int8Ws o;
  char* ws;
  const uint32_t* kept;
  Side x, xs;            // the product: 8-bit rows and scales; the block: rows of type dt
  Side w_in, s_in, w_out, s_out, y;
  int w_in_ok, w_out_ok, x_ok, y_ok;   // whole 16-byte vectors
  int dt;                // of the results
  int product;           // the block's rows, as in Int8Rows
  hipStream_t st;
};
hipError_t launch_int8(const Int8Launch& L);
hipError_t launch_int8_ffn(const Int8Launch& L);


}  // namespace cc
