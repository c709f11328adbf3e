// C ABI of the model-side operators: embedding and its gradients, MoE routing
// and its gradient, the routing's balance loss and its gradient, the experts' gated
// feed-forward block and its gradients, with 8-bit checkpoints too, and the
// experts' products in 8-bit integers.
// Declared in include/cc.h.

#include <algorithm>
#include <new>
#include <vector>

#include "cc_api_internal.h"
#include "cc_llm.h"

using namespace cc;
using namespace cc::api;

namespace {

typedef unsigned __int128 u128;
constexpr uint64_t kByteLimit = 1ull << 62;
constexpr uint64_t kMaxBlocks = 1ull << 24;   // workgroups of 256 threads whose work-items fit 32 bits

// host allocations are the only thing that may throw here
template <class F>
cc_status_t guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(CC_ERR_INVALID_ARG, "no host memory for the counts");
  }
}

cc_status_t model_checks(int nranks, cc_dtype_t dtype, const cc_config_t& cfg) {
  cc_status_t s = common_checks(CC_COLL_ALL_REDUCE, nranks, dtype, &cfg);
  if (s) return s;
  if (dtype != CC_FLOAT32 && dtype != CC_BFLOAT16)
    return fail(CC_ERR_UNSUPPORTED, "the model-side operators take float32 or bf16");
  if (cfg.algo != CC_ALGO_RING || cfg.fuse_depth != 0)
    return fail(CC_ERR_UNSUPPORTED, "the model-side operators have no schedules (algo ring, fuse_depth 0)");
  return CC_OK;
}

// One buffer of a call: n bytes per rank, `ranks` of them (1 for a shared one).
struct Buf {
  const cc_rankbuf_t* b;
  u128 n;
  const char* name;
  bool out;
  int ranks;
};

bool al(const cc_rankbuf_t& b) { return al16p(b.base) && al16(b.rank_stride_bytes); }

// Bases, strides and sizes, then outputs against everything else and the
// workspace against everything.
cc_status_t check_bufs(const Buf* b, int n, const cc_config_t& cfg, uint64_t need, const char* sizer) {
  cc_status_t s;
  for (int i = 0; i < n; ++i) {
    if (b[i].n >= kByteLimit) return fail(CC_ERR_INVALID_ARG, "%s is too large", b[i].name);
    if ((s = check_side(*b[i].b, (uint64_t)b[i].n, b[i].ranks, b[i].name))) return s;
  }
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((b[i].out || b[j].out) &&
          sides_overlap(*b[i].b, (uint64_t)b[i].n, b[i].ranks, *b[j].b, (uint64_t)b[j].n, b[j].ranks))
        return fail(CC_ERR_INVALID_ARG, "%s and %s overlap", b[i].name, b[j].name);
  if (need == 0) return CC_OK;
  if (cfg.workspace == nullptr || cfg.workspace_bytes < need)
    return fail(CC_ERR_INVALID_ARG, "this call needs %llu bytes of workspace (%s); got %zu", (unsigned long long)need,
                sizer, cfg.workspace ? cfg.workspace_bytes : (size_t)0);
  if (!al16p(cfg.workspace)) return fail(CC_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
  const cc_rankbuf_t ws{cfg.workspace, (size_t)need};
  for (int i = 0; i < n; ++i)
    if (sides_overlap(ws, need, 1, *b[i].b, (uint64_t)b[i].n, b[i].ranks))
      return fail(CC_ERR_INVALID_ARG, "the workspace overlaps %s", b[i].name);
  return CC_OK;
}

// elements that start on a multiple of their size
bool elems_aligned(const cc_rankbuf_t& b, int es) {
  return ((uint64_t)(uintptr_t)b.base % es) == 0 && b.rank_stride_bytes % es == 0;
}
cc_status_t check_elems(const cc_rankbuf_t& b, int es, const char* name) {
  if (!elems_aligned(b, es))
    return fail(CC_ERR_INVALID_ARG, "%s must start on a multiple of its elements' %d bytes on every rank", name, es);
  return CC_OK;
}

// ------------------------------------------------------------------ embedding

cc_status_t embed_sizes(int nranks, uint64_t vocab, uint64_t tokens, uint64_t width) {
  if (nranks < 1 || nranks > CC_MAX_RANKS)
    return fail(CC_ERR_INVALID_ARG, "nranks=%d outside [1, %d]", nranks, CC_MAX_RANKS);
  if (vocab == 0 || width == 0) return fail(CC_ERR_INVALID_ARG, "vocab and width must be positive");
  if (vocab >= (1ull << 27)) return fail(CC_ERR_INVALID_ARG, "vocab too large for one launch");
  if (tokens >= kMaxBlocks) return fail(CC_ERR_INVALID_ARG, "tokens too large for one launch");
  if (width >= (1ull << 40)) return fail(CC_ERR_INVALID_ARG, "width too large");
  return CC_OK;
}

// the sort of each rank's ids and the partial sums of its pieces
struct EmbedWs {
  SortPlan sort;
  uint64_t partial, bytes;
};
EmbedWs embed_ws(int N, uint64_t vocab, uint64_t tokens, uint64_t width) {
  EmbedWs w;
  w.sort = sort_plan(N, tokens, (uint32_t)vocab);
  w.partial = w.sort.bytes;
  w.bytes = tokens ? w.partial + rup((uint64_t)N * embed_pieces(tokens) * embed_partial_pitch(width) * 4, 256) : 0;
  return w;
}

cc_status_t embed_grad(cc_rankbuf_t grad, cc_rankbuf_t ids, cc_rankbuf_t dtable, uint64_t vocab, uint64_t tokens,
                       uint64_t width, float scale, cc_dtype_t dtype, int N, const cc_config_t& cfg, bool summed,
                       hipStream_t st) {
  cc_status_t s = model_checks(N, dtype, cfg);
  if (s || (s = embed_sizes(N, vocab, tokens, width))) return s;
  const int es = elem_size((int)dtype);
  const Buf b[] = {{&grad, (u128)tokens * width * es, "grad", false, N},
                   {&ids, (u128)tokens * 4, "ids", false, N},
                   {&dtable, (u128)vocab * width * es, "dtable", true, N}};
  const u128 whole = (u128)N * tokens * width * 4 + (u128)N * tokens * 64;
  if (whole >= kByteLimit) return fail(CC_ERR_INVALID_ARG, "grad is too large");
  const EmbedWs w = embed_ws(N, vocab, tokens, width);
  if ((s = check_bufs(b, 3, cfg, w.bytes, "cc_embedding_grad_workspace_size")) ||
      (s = check_elems(grad, es, "grad")) || (s = check_elems(ids, 4, "ids")) || (s = check_elems(dtable, es, "dtable")))
    return s;
  if ((s = device_ready())) return s;
  SortLaunch so = {};
  so.p = w.sort;
  so.keys = (const char*)ids.base;
  so.key_stride = ids.rank_stride_bytes;
  so.ws = (char*)cfg.workspace;
  so.st = st;
  if (tokens) {
    hipError_t e = launch_sort(&so);
    if (e != hipSuccess) return hip_status(e, "embedding gradient (sort)");
  }
  EmbedGradLaunch L = {};
  L.grad = (const char*)grad.base; L.grad_stride = grad.rank_stride_bytes;
  L.out = (char*)dtable.base; L.out_stride = dtable.rank_stride_bytes;
  L.keys = so.sorted_keys; L.vals = so.sorted_vals;
  L.partial = (float*)((char*)cfg.workspace + w.partial);
  L.vocab = vocab; L.tokens = tokens; L.width = width;
  L.scale = scale;
  L.N = N; L.dt = (int)dtype; L.blocks_per_cu = cfg.blocks_per_cu;
  L.vec_ok = (tokens == 0 || al(grad)) && al(dtable) && al16(width * es);
  L.summed = summed;
  L.st = st;
  return hip_status(launch_embed_grad(L), "embedding gradient");
}

// ------------------------------------------------------------------ routing

cc_status_t route_sizes(int nranks, uint64_t tokens, int nexperts, int topk, int normalize) {
  if (nranks < 1 || nranks > CC_MAX_RANKS)
    return fail(CC_ERR_INVALID_ARG, "nranks=%d outside [1, %d]", nranks, CC_MAX_RANKS);
  if (nexperts < 1 || nexperts > CC_MAX_ROUTE_EXPERTS)
    return fail(CC_ERR_INVALID_ARG, "nexperts=%d outside [1, %d]", nexperts, CC_MAX_ROUTE_EXPERTS);
  if (topk < 1 || topk > 64 || topk > nexperts)
    return fail(CC_ERR_INVALID_ARG, "topk=%d outside [1, %d]", topk, std::min(64, nexperts));
  if (normalize != 0 && normalize != 1) return fail(CC_ERR_INVALID_ARG, "normalize=%d is neither 0 nor 1", normalize);
  if (tokens >= kMaxBlocks) return fail(CC_ERR_INVALID_ARG, "tokens too large for one launch");
  return CC_OK;
}

// ------------------------------------------------------------------ feed-forward

constexpr int kMaxFfnExperts = 8192;   // the plan's workgroups each sum the counts of the experts before theirs

// What a call launches: the block's products and its weights' gradients, the
// block's products alone, or one product of F columns.
enum Launches { BLOCK_AND_GRADIENTS, BLOCK, PRODUCT };

// Counts [N][E] as the caller gives them -> kept rows [E][N], totals and
// limits.  Row numbers are int32 on the device.
cc_status_t ffn_shape(const size_t* counts, int E, uint64_t cap, uint64_t W, uint64_t F, cc_dtype_t dtype, int N,
                      FfnShape* sh, std::vector<uint32_t>* kept, Launches what = BLOCK_AND_GRADIENTS) {
  if (N < 1 || N > CC_MAX_RANKS) return fail(CC_ERR_INVALID_ARG, "nranks=%d outside [1, %d]", N, CC_MAX_RANKS);
  if (!counts) return fail(CC_ERR_INVALID_ARG, "counts is NULL");
  if (E < N || E % N) return fail(CC_ERR_INVALID_ARG, "nexperts=%d must be a positive multiple of nranks=%d", E, N);
  if (E > kMaxFfnExperts) return fail(CC_ERR_INVALID_ARG, "nexperts=%d is above %d", E, kMaxFfnExperts);
  if (W == 0 || F == 0) return fail(CC_ERR_INVALID_ARG, "width and hidden must be positive");
  if (W >= (1ull << 24) || F >= (1ull << 24)) return fail(CC_ERR_INVALID_ARG, "width or hidden too large");
  if ((u128)E * cap >= (1ull << 31)) return fail(CC_ERR_INVALID_ARG, "nexperts * capacity must be below 2^31 rows");
  kept->assign((size_t)E * N, 0);
  uint64_t rows = 0, most = 0, tiles[kFfnTiles] = {};
  for (int e = 0; e < E; ++e) {
    uint64_t n = 0;
    for (int i = 0; i < N; ++i) {
      if (counts[(size_t)i * E + e] > SIZE_MAX / 2)
        return fail(CC_ERR_INVALID_ARG, "counts[%d][%d] is negative", i, e);
      const uint64_t k = std::min<uint64_t>(counts[(size_t)i * E + e], cap);
      (*kept)[(size_t)e * N + i] = (uint32_t)k;
      n += k;
    }
    rows += n;
    most = std::max(most, n);
    for (int k = 0; k < kFfnTiles; ++k) tiles[k] += (n + kFfnTile[k] - 1) / kFfnTile[k];
    if (rows >= (1ull << 31)) return fail(CC_ERR_INVALID_ARG, "2^31 rows or more in one call");
  }
  // columns of the smallest tiles
  const uint64_t wt = ((what == PRODUCT ? F : 2 * F) + 63) / 64, wn = what == PRODUCT ? 0 : (W + 63) / 64;
  if ((u128)tiles[kFfnTiles - 1] * std::max(wt, wn) >= kMaxBlocks ||
      (what == BLOCK_AND_GRADIENTS && (u128)E * wt * wn >= kMaxBlocks))
    return fail(CC_ERR_INVALID_ARG, "too many tiles for one launch");
  *sh = FfnShape{N, E, cap, W, F, rows, most, {tiles[0], tiles[1], tiles[2]}, (int)dtype, elem_size((int)dtype), 0};
  return CC_OK;
}

struct FfnBufs {
  cc_rankbuf_t x, w_in, w_out, pre, y, dy, dx, dw_in, dw_out;
  cc_rankbuf_t ckpt;   // in place of pre, and for the gradients of x
  bool kept8;
};

Side side(const cc_rankbuf_t& b) { return Side{(char*)b.base, (uint64_t)b.rank_stride_bytes}; }

cc_status_t run_ffn(const FfnBufs& f, const size_t* counts, int E, uint64_t cap, uint64_t W, uint64_t F, cc_act_t act,
                    cc_dtype_t dtype, int N, const cc_config_t& cfg, bool grad, hipStream_t st) {
  cc_status_t s = model_checks(N, dtype, cfg);
  if (s) return s;
  if ((int)act != CC_ACT_SILU && (int)act != CC_ACT_GELU)
    return fail(CC_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  FfnLaunch L = {};
  std::vector<uint32_t> kept;
  if ((s = ffn_shape(counts, E, cap, W, F, dtype, N, &L.s, &kept))) return s;
  const int es = elem_size((int)dtype);
  L.s.act = (int)act;
  L.o = ffn_ws(L.s, grad, f.kept8);
  const u128 side_n = (u128)E * cap * W * es, pre_n = (u128)E * cap * 2 * F * es;
  const u128 wi_n = (u128)(E / N) * 2 * F * W * es, wo_n = (u128)(E / N) * W * F * es;
  const u128 ckpt_n = (u128)E * cap * (unsigned)ckpt_row(W, F).pitch;
  const bool keep = !f.kept8 && (grad || f.pre.base != nullptr);
  std::vector<Buf> b;
  if (!grad || !f.kept8) b.push_back({&f.x, side_n, "x", false, N});
  b.push_back({&f.w_in, wi_n, "w_in", false, N});
  b.push_back({&f.w_out, wo_n, "w_out", false, N});
  if (f.kept8) b.push_back({&f.ckpt, ckpt_n, "ckpt", !grad, N});
  if (keep) b.push_back({&f.pre, pre_n, "pre", !grad, N});
  if (grad) {
    b.push_back({&f.dy, side_n, "dy", false, N});
    b.push_back({&f.dx, side_n, "dx", true, N});
    b.push_back({&f.dw_in, wi_n, "dw_in", true, N});
    b.push_back({&f.dw_out, wo_n, "dw_out", true, N});
  } else {
    b.push_back({&f.y, side_n, "y", true, N});
  }
  if ((s = check_bufs(b.data(), (int)b.size(), cfg, L.o.bytes,
                      f.kept8 ? "cc_moe_ffn_checkpoint_workspace_size" : "cc_moe_ffn_workspace_size")))
    return s;
  if (f.kept8 && ckpt_n != 0 && !al(f.ckpt))
    return fail(CC_ERR_INVALID_ARG, "ckpt must start on a multiple of 16 bytes on every rank");
  L.vec_ok = al16(W * es) && al16(F * es);
  for (const Buf& x : b) {
    if (x.n == 0 || x.b == &f.ckpt) continue;   // no rows: never touched
    if ((s = check_elems(*x.b, es, x.name))) return s;
    L.vec_ok = L.vec_ok && al(*x.b);
  }
  if (L.s.rows == 0 && !grad) return ok();
  if ((s = device_ready())) return s;
  L.ws = (char*)cfg.workspace;
  L.kept = kept.data();
  L.x = side(f.x); L.w_in = side(f.w_in); L.w_out = side(f.w_out);
  L.pre = keep ? side(f.pre) : Side{nullptr, 0};
  L.y = side(f.y);
  L.ckpt = f.kept8 ? side(f.ckpt) : Side{nullptr, 0};
  L.dy = side(f.dy); L.dx = side(f.dx); L.dw_in = side(f.dw_in); L.dw_out = side(f.dw_out);
  L.st = st;
  return hip_status(grad ? launch_ffn_grad(L) : launch_ffn(L), grad ? "expert feed-forward gradient" : "expert feed-forward");
}

// ------------------------------------------------------------------ balance loss

cc_status_t balance_sizes(int nranks, uint64_t tokens, int nexperts) {
  return route_sizes(nranks, tokens, nexperts, 1, 0);
}

// ------------------------------------------------------------------ 8-bit integers

constexpr uint64_t kMaxInt8Sum = 1ull << 17;   // 2^14 a product: sums below 2^31

// The shape of a product (cols, block 0) or of the block (hidden, block 1).
cc_status_t int8_shape(const size_t* counts, int E, uint64_t cap, uint64_t W, uint64_t F, int N, bool block,
                       FfnShape* sh, std::vector<uint32_t>* kept) {
  if (W >= kMaxInt8Sum || (block && F >= kMaxInt8Sum))
    return fail(CC_ERR_INVALID_ARG, "a summed axis must be shorter than %llu", (unsigned long long)kMaxInt8Sum);
  cc_status_t s = ffn_shape(counts, E, cap, W, F, CC_BFLOAT16, N, sh, kept, block ? BLOCK : PRODUCT);
  sh->es = 1;
  return s;
}

bool rows16(const cc_rankbuf_t& b, uint64_t row_bytes) { return al(b) && al16(row_bytes); }

struct Int8Bufs {
  cc_rankbuf_t x, xs, w_in, s_in, w_out, s_out, y;
};

cc_status_t check_scale(int scale) {
  return scale == CC_SCALE_QUOTIENT || scale == CC_SCALE_PRODUCT ? CC_OK
                                                                 : fail(CC_ERR_INVALID_ARG, "unknown scale %d", scale);
}

cc_status_t run_int8(const Int8Bufs& f, const size_t* counts, int E, uint64_t cap, uint64_t W, uint64_t F, int act,
                     int scale, cc_dtype_t dtype, int N, const cc_config_t& cfg, bool block, hipStream_t st) {
  cc_status_t s = model_checks(N, dtype, cfg);
  if (s) return s;
  if (act != CC_ACT_SILU && act != CC_ACT_GELU) return fail(CC_ERR_INVALID_ARG, "unknown activation %d", act);
  if ((s = check_scale(scale))) return s;
  Int8Launch L = {};
  std::vector<uint32_t> kept;
  if ((s = int8_shape(counts, E, cap, W, F, N, block, &L.s, &kept))) return s;
  const int es = elem_size((int)dtype);
  L.s.act = act;
  L.o = int8_ws(L.s, block, es);
  const u128 side_n = (u128)E * cap, per = (unsigned)(E / N), lines = block ? 2 * F : F;
  const uint64_t ycols = block ? W : F;
  std::vector<Buf> b = {{&f.x, side_n * W * (block ? es : 1), "x", false, N},
                        {&f.w_in, per * lines * W, block ? "w_in" : "w", false, N},
                        {&f.s_in, per * lines * 4, block ? "s_in" : "sw", false, N},
                        {&f.y, side_n * ycols * es, "y", true, N}};
  const int elems[] = {block ? es : 1, 1, 4, es, block ? 1 : 4, 4};
  if (block) {
    b.push_back({&f.w_out, per * W * F, "w_out", false, N});
    b.push_back({&f.s_out, per * W * 4, "s_out", false, N});
  } else {
    b.push_back({&f.xs, side_n * 4, "sx", false, N});
  }
  if ((s = check_bufs(b.data(), (int)b.size(), cfg, L.o.bytes,
                      block ? "cc_moe_ffn_int8_workspace_size" : "cc_moe_matmul_int8_workspace_size")))
    return s;
  for (size_t i = 0; i < b.size(); ++i)
    if (b[i].n && (s = check_elems(*b[i].b, elems[i], b[i].name))) return s;
  if (L.s.rows == 0) return ok();
  if ((s = device_ready())) return s;
  L.ws = (char*)cfg.workspace;
  L.kept = kept.data();
  L.x = side(f.x); L.xs = side(f.xs);
  L.w_in = side(f.w_in); L.s_in = side(f.s_in); L.w_out = side(f.w_out); L.s_out = side(f.s_out);
  L.y = side(f.y);
  L.x_ok = rows16(f.x, W);
  L.w_in_ok = rows16(f.w_in, W);
  L.w_out_ok = block && rows16(f.w_out, F);
  L.y_ok = rows16(f.y, ycols * es);
  L.dt = (int)dtype;
  L.product = scale == CC_SCALE_PRODUCT;
  L.st = st;
  return hip_status(block ? launch_int8_ffn(L) : launch_int8(L),
                    block ? "expert feed-forward in 8-bit integers" : "product in 8-bit integers");
}

}  // namespace

extern "C" {

cc_status_t cc_embedding(cc_rankbuf_t table, cc_rankbuf_t ids, cc_rankbuf_t out, size_t vocab, size_t tokens,
                         size_t width, float scale, cc_dtype_t dtype, int nranks, const cc_config_t* cfgp,
                         cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = embed_sizes(nranks, vocab, tokens, width))) return s;
  if (tokens == 0) return ok();
  const int N = nranks, es = elem_size((int)dtype);
  const Buf b[] = {{&table, (u128)vocab * width * es, "table", false, table.rank_stride_bytes == 0 ? 1 : N},
                   {&ids, (u128)tokens * 4, "ids", false, N},
                   {&out, (u128)tokens * width * es, "out", true, N}};
  if ((s = check_bufs(b, 3, cfg, 0, "")) || (s = check_elems(table, es, "table")) ||
      (s = check_elems(ids, 4, "ids")) || (s = check_elems(out, es, "out")))
    return s;
  if ((s = device_ready())) return s;
  const int vec_ok = al(table) && al(out) && al16(width * es);
  return hip_status(launch_embed(EmbedLaunch{(const char*)table.base, table.rank_stride_bytes, (const char*)ids.base,
                                             ids.rank_stride_bytes, (char*)out.base, out.rank_stride_bytes, vocab,
                                             tokens, width, scale, N, (int)dtype, vec_ok, cfg.blocks_per_cu,
                                             (hipStream_t)stream}),
                    "embedding lookup");
}

cc_status_t cc_embedding_grad(cc_rankbuf_t grad, cc_rankbuf_t ids, cc_rankbuf_t dtable, size_t vocab, size_t tokens,
                              size_t width, float scale, cc_dtype_t dtype, int nranks, const cc_config_t* cfgp,
                              cc_stream_t stream) {
  return embed_grad(grad, ids, dtable, vocab, tokens, width, scale, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, false,
                    (hipStream_t)stream);
}

cc_status_t cc_all_reduce_embedding_grad(cc_rankbuf_t grad, cc_rankbuf_t ids, cc_rankbuf_t dtable, size_t vocab,
                                         size_t tokens, size_t width, float scale, cc_dtype_t dtype, int nranks,
                                         const cc_config_t* cfgp, cc_stream_t stream) {
  return embed_grad(grad, ids, dtable, vocab, tokens, width, scale, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, true,
                    (hipStream_t)stream);
}

cc_status_t cc_embedding_grad_workspace_size(int nranks, size_t vocab, size_t tokens, size_t width, size_t* bytes) {
  cc_status_t s = embed_sizes(nranks, vocab, tokens, width);
  if (s) return s;
  if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
  if ((u128)nranks * tokens * width * 4 + (u128)nranks * tokens * 64 >= kByteLimit)
    return fail(CC_ERR_INVALID_ARG, "grad is too large");
  *bytes = (size_t)embed_ws(nranks, vocab, tokens, width).bytes;
  return ok();
}

cc_status_t cc_moe_route(cc_rankbuf_t logits, cc_rankbuf_t experts, cc_rankbuf_t weights, cc_rankbuf_t order,
                         cc_rankbuf_t counts, size_t tokens, int nexperts, int topk, int normalize, cc_dtype_t dtype,
                         int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = route_sizes(nranks, tokens, nexperts, topk, normalize))) return s;
  const int N = nranks, es = elem_size((int)dtype);
  const u128 slots = (u128)tokens * (unsigned)topk * 4;
  const Buf b[] = {{&logits, (u128)tokens * (unsigned)nexperts * es, "logits", false, N},
                   {&experts, slots, "experts", true, N},
                   {&weights, slots, "weights", true, N},
                   {&order, slots, "order", true, N},
                   {&counts, (u128)(unsigned)nexperts * 4, "counts", true, N}};
  const SortPlan p = sort_plan(N, (uint64_t)tokens * topk, (uint32_t)nexperts);
  if ((s = check_bufs(b, 5, cfg, tokens ? p.bytes : 0, "cc_moe_route_workspace_size"))) return s;
  for (int i = 0; i < 5; ++i)
    if (b[i].n && (s = check_elems(*b[i].b, i ? 4 : es, b[i].name))) return s;
  if ((s = device_ready())) return s;
  RouteLaunch L = {};
  L.logits = (const char*)logits.base; L.logits_stride = logits.rank_stride_bytes;
  L.experts = (char*)experts.base; L.experts_stride = experts.rank_stride_bytes;
  L.weights = (char*)weights.base; L.weights_stride = weights.rank_stride_bytes;
  L.tokens = tokens; L.nexperts = nexperts; L.topk = topk; L.normalize = normalize;
  L.N = N; L.dt = (int)dtype; L.st = (hipStream_t)stream;
  hipError_t e = tokens ? launch_route(L) : hipSuccess;
  if (e != hipSuccess) return hip_status(e, "MoE routing");
  SortLaunch so = {};
  so.p = p;
  so.keys = (const char*)experts.base;
  so.key_stride = experts.rank_stride_bytes;
  so.ws = (char*)cfg.workspace;
  so.order = (char*)order.base; so.order_stride = order.rank_stride_bytes;
  so.counts = (char*)counts.base; so.counts_stride = counts.rank_stride_bytes;
  so.st = (hipStream_t)stream;
  return hip_status(launch_sort(&so), "MoE routing (order)");
}

cc_status_t cc_moe_route_workspace_size(int nranks, size_t tokens, int nexperts, int topk, size_t* bytes) {
  cc_status_t s = route_sizes(nranks, tokens, nexperts, topk, 0);
  if (s) return s;
  if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = tokens == 0 ? 0 : (size_t)sort_plan(nranks, (uint64_t)tokens * topk, (uint32_t)nexperts).bytes;
  return ok();
}

cc_status_t cc_moe_route_grad(cc_rankbuf_t logits, cc_rankbuf_t experts, cc_rankbuf_t dweights, cc_rankbuf_t dlogits,
                              size_t tokens, int nexperts, int topk, int normalize, cc_dtype_t dtype, int nranks,
                              const cc_config_t* cfgp, cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = route_sizes(nranks, tokens, nexperts, topk, normalize))) return s;
  if (tokens == 0) return ok();
  const int N = nranks, es = elem_size((int)dtype);
  const u128 slots = (u128)tokens * (unsigned)topk * 4, lg = (u128)tokens * (unsigned)nexperts * es;
  const Buf b[] = {{&logits, lg, "logits", false, N},
                   {&experts, slots, "experts", false, N},
                   {&dweights, slots, "dweights", false, N},
                   {&dlogits, lg, "dlogits", true, N}};
  if ((s = check_bufs(b, 4, cfg, 0, ""))) return s;
  for (int i = 0; i < 4; ++i)
    if ((s = check_elems(*b[i].b, i == 1 || i == 2 ? 4 : es, b[i].name))) return s;
  if ((s = device_ready())) return s;
  RouteLaunch L = {};
  L.logits = (const char*)logits.base; L.logits_stride = logits.rank_stride_bytes;
  L.experts = (char*)experts.base; L.experts_stride = experts.rank_stride_bytes;
  L.weights = (char*)dweights.base; L.weights_stride = dweights.rank_stride_bytes;
  L.dlogits = (char*)dlogits.base; L.dlogits_stride = dlogits.rank_stride_bytes;
  L.tokens = tokens; L.nexperts = nexperts; L.topk = topk; L.normalize = normalize;
  L.N = N; L.dt = (int)dtype; L.st = (hipStream_t)stream;
  return hip_status(launch_route_grad(L), "MoE routing gradient");
}

cc_status_t cc_moe_ffn(cc_rankbuf_t x, cc_rankbuf_t w_in, cc_rankbuf_t w_out, cc_rankbuf_t pre, cc_rankbuf_t y,
                       const size_t* counts, int nexperts, size_t capacity, size_t width, size_t hidden, cc_act_t act,
                       cc_dtype_t dtype, int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_ffn(FfnBufs{x, w_in, w_out, pre, y, none, none, none, none, none, false}, counts, nexperts, capacity, width, hidden,
                   act, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, false, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_grad(cc_rankbuf_t x, cc_rankbuf_t w_in, cc_rankbuf_t w_out, cc_rankbuf_t pre, cc_rankbuf_t dy,
                            cc_rankbuf_t dx, cc_rankbuf_t dw_in, cc_rankbuf_t dw_out, const size_t* counts,
                            int nexperts, size_t capacity, size_t width, size_t hidden, cc_act_t act, cc_dtype_t dtype,
                            int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_ffn(FfnBufs{x, w_in, w_out, pre, none, dy, dx, dw_in, dw_out, none, false}, counts, nexperts, capacity, width, hidden,
                   act, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, true, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_workspace_size(const size_t* counts, int nexperts, size_t capacity, size_t width, size_t hidden,
                                      cc_dtype_t dtype, int nranks, int grad, size_t* bytes) {
  return guarded([&] {
    FfnShape sh;
    std::vector<uint32_t> kept;
    cc_status_t s = model_checks(nranks, dtype, kDefaultCfg);
    if (s || (s = ffn_shape(counts, nexperts, capacity, width, hidden, dtype, nranks, &sh, &kept))) return s;
    if (grad != 0 && grad != 1) return fail(CC_ERR_INVALID_ARG, "grad=%d is neither 0 nor 1", grad);
    if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)ffn_ws(sh, grad).bytes;
    return ok();
  });
}

cc_status_t cc_moe_balance_loss(cc_rankbuf_t logits, cc_rankbuf_t counts, cc_rankbuf_t total, cc_rankbuf_t prob,
                                cc_rankbuf_t loss, size_t tokens, int nexperts, int summed, cc_dtype_t dtype,
                                int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = balance_sizes(nranks, tokens, nexperts))) return s;
  if (summed != 0 && summed != 1) return fail(CC_ERR_INVALID_ARG, "summed=%d is neither 0 nor 1", summed);
  const int N = nranks, es = elem_size((int)dtype);
  const u128 E = (unsigned)nexperts;
  const Buf b[] = {{&logits, (u128)tokens * E * es, "logits", false, N},
                   {&counts, E * 4, "counts", false, N},
                   {&total, (E + 1) * 4, "total", true, N},
                   {&prob, E * 4, "prob", true, N},
                   {&loss, 4, "loss", true, N}};
  if ((s = check_bufs(b, 5, cfg, balance_ws(N, tokens, nexperts), "cc_moe_balance_loss_workspace_size"))) return s;
  for (int i = 0; i < 5; ++i)
    if (b[i].n && (s = check_elems(*b[i].b, i ? 4 : es, b[i].name))) return s;
  if ((s = device_ready())) return s;
  BalanceLaunch L = {};
  L.logits = (const char*)logits.base; L.logits_stride = logits.rank_stride_bytes;
  L.counts = (const char*)counts.base; L.counts_stride = counts.rank_stride_bytes;
  L.total = (char*)total.base; L.total_stride = total.rank_stride_bytes;
  L.prob = (char*)prob.base; L.prob_stride = prob.rank_stride_bytes;
  L.loss = (char*)loss.base; L.loss_stride = loss.rank_stride_bytes;
  L.ws = (char*)cfg.workspace;
  L.tokens = tokens; L.nexperts = nexperts; L.summed = summed;
  L.N = N; L.dt = (int)dtype; L.st = (hipStream_t)stream;
  return hip_status(launch_balance(L), "balance loss");
}

cc_status_t cc_moe_balance_loss_workspace_size(int nranks, size_t tokens, int nexperts, size_t* bytes) {
  cc_status_t s = balance_sizes(nranks, tokens, nexperts);
  if (s) return s;
  if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)balance_ws(nranks, tokens, nexperts);
  return ok();
}

cc_status_t cc_moe_balance_loss_grad(cc_rankbuf_t logits, cc_rankbuf_t total, cc_rankbuf_t dloss, cc_rankbuf_t base,
                                     cc_rankbuf_t dlogits, size_t tokens, int nexperts, cc_dtype_t dtype, int nranks,
                                     const cc_config_t* cfgp, cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = balance_sizes(nranks, tokens, nexperts))) return s;
  if (tokens == 0) return ok();
  const int N = nranks, es = elem_size((int)dtype);
  const u128 E = (unsigned)nexperts, lg = (u128)tokens * E * es;
  // in place: one buffer, read and written element by element
  const bool apart = base.base && !same_side(base, dlogits);
  const Buf b[] = {{&logits, lg, "logits", false, N},
                   {&total, (E + 1) * 4, "total", false, N},
                   {&dloss, 4, "dloss", false, N},
                   {&dlogits, lg, "dlogits", true, N},
                   {&base, lg, "base", false, N}};
  const int n = apart ? 5 : 4;
  if ((s = check_bufs(b, n, cfg, 0, ""))) return s;
  for (int i = 0; i < n; ++i)
    if ((s = check_elems(*b[i].b, i == 1 || i == 2 ? 4 : es, b[i].name))) return s;
  if ((s = device_ready())) return s;
  BalanceLaunch L = {};
  L.logits = (const char*)logits.base; L.logits_stride = logits.rank_stride_bytes;
  L.total = (char*)total.base; L.total_stride = total.rank_stride_bytes;
  L.loss = (char*)dloss.base; L.loss_stride = dloss.rank_stride_bytes;
  L.base = (const char*)base.base; L.base_stride = base.rank_stride_bytes;
  L.dlogits = (char*)dlogits.base; L.dlogits_stride = dlogits.rank_stride_bytes;
  L.tokens = tokens; L.nexperts = nexperts;
  L.N = N; L.dt = (int)dtype; L.st = (hipStream_t)stream;
  return hip_status(launch_balance_grad(L), "balance loss gradient");
}

cc_status_t cc_quantize_rows_scaled(cc_rankbuf_t x, cc_rankbuf_t q, cc_rankbuf_t scales, size_t rows, size_t width,
                                    cc_scale_t scale, cc_dtype_t dtype, int nranks, const cc_config_t* cfgp,
                                    cc_stream_t stream) {
  const cc_config_t& cfg = cfgp ? *cfgp : kDefaultCfg;
  cc_status_t s = model_checks(nranks, dtype, cfg);
  if (s || (s = check_scale((int)scale))) return s;
  if (width == 0) return fail(CC_ERR_INVALID_ARG, "width must be positive");
  if (width >= (1ull << 31) || rows >= (1ull << 31)) return fail(CC_ERR_INVALID_ARG, "width or rows too large");
  if (rows == 0) return ok();
  const int N = nranks, es = elem_size((int)dtype);
  const Buf b[] = {{&x, (u128)rows * width * es, "x", false, N},
                   {&q, (u128)rows * width, "q", true, N},
                   {&scales, (u128)rows * 4, "scales", true, N}};
  if ((s = check_bufs(b, 3, cfg, 0, "")) || (s = check_elems(x, es, "x")) || (s = check_elems(scales, 4, "scales")))
    return s;
  if ((s = device_ready())) return s;
  Int8Rows L = {};
  L.x = (const char*)x.base; L.x_stride = x.rank_stride_bytes;
  L.q = (char*)q.base; L.q_stride = q.rank_stride_bytes; L.q_pitch = width;
  L.s = (char*)scales.base; L.s_stride = scales.rank_stride_bytes;
  L.rows = rows; L.width = width; L.N = N; L.dt = (int)dtype; L.product = scale == CC_SCALE_PRODUCT;
  L.st = (hipStream_t)stream;
  return hip_status(launch_int8_rows(L), "quantisation of rows");
}

cc_status_t cc_quantize_rows(cc_rankbuf_t x, cc_rankbuf_t q, cc_rankbuf_t scales, size_t rows, size_t width,
                             cc_dtype_t dtype, int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return cc_quantize_rows_scaled(x, q, scales, rows, width, CC_SCALE_QUOTIENT, dtype, nranks, cfgp, stream);
}

cc_status_t cc_moe_matmul_int8(cc_rankbuf_t x, cc_rankbuf_t sx, cc_rankbuf_t w, cc_rankbuf_t sw, cc_rankbuf_t y,
                               const size_t* counts, int nexperts, size_t capacity, size_t width, size_t cols,
                               cc_dtype_t dtype, int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_int8(Int8Bufs{x, sx, w, sw, none, none, y}, counts, nexperts, capacity, width, cols, CC_ACT_SILU,
                    CC_SCALE_QUOTIENT, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, false, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_int8_scaled(cc_rankbuf_t x, cc_rankbuf_t w_in, cc_rankbuf_t s_in, cc_rankbuf_t w_out,
                                   cc_rankbuf_t s_out, cc_rankbuf_t y, const size_t* counts, int nexperts,
                                   size_t capacity, size_t width, size_t hidden, cc_act_t act, cc_scale_t scale,
                                   cc_dtype_t dtype, int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_int8(Int8Bufs{x, none, w_in, s_in, w_out, s_out, y}, counts, nexperts, capacity, width, hidden, (int)act,
                    (int)scale, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, true, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_int8(cc_rankbuf_t x, cc_rankbuf_t w_in, cc_rankbuf_t s_in, cc_rankbuf_t w_out,
                            cc_rankbuf_t s_out, cc_rankbuf_t y, const size_t* counts, int nexperts, size_t capacity,
                            size_t width, size_t hidden, cc_act_t act, cc_dtype_t dtype, int nranks,
                            const cc_config_t* cfgp, cc_stream_t stream) {
  return cc_moe_ffn_int8_scaled(x, w_in, s_in, w_out, s_out, y, counts, nexperts, capacity, width, hidden, act,
                                CC_SCALE_QUOTIENT, dtype, nranks, cfgp, stream);
}

cc_status_t cc_moe_matmul_int8_workspace_size(const size_t* counts, int nexperts, size_t capacity, size_t width,
                                              size_t cols, int nranks, size_t* bytes) {
  return guarded([&] {
    FfnShape sh;
    std::vector<uint32_t> kept;
    cc_status_t s = int8_shape(counts, nexperts, capacity, width, cols, nranks, false, &sh, &kept);
    if (s) return s;
    if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)int8_ws(sh, 0, 0).bytes;
    return ok();
  });
}

cc_status_t cc_moe_ffn_int8_workspace_size(const size_t* counts, int nexperts, size_t capacity, size_t width,
                                           size_t hidden, cc_dtype_t dtype, int nranks, size_t* bytes) {
  return guarded([&] {
    FfnShape sh;
    std::vector<uint32_t> kept;
    cc_status_t s = model_checks(nranks, dtype, kDefaultCfg);
    if (s || (s = int8_shape(counts, nexperts, capacity, width, hidden, nranks, true, &sh, &kept))) return s;
    if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)int8_ws(sh, 1, elem_size((int)dtype)).bytes;
    return ok();
  });
}

cc_status_t cc_moe_ffn_checkpoint(cc_rankbuf_t x, cc_rankbuf_t w_in, cc_rankbuf_t w_out, cc_rankbuf_t ckpt,
                                  cc_rankbuf_t y, const size_t* counts, int nexperts, size_t capacity, size_t width,
                                  size_t hidden, cc_act_t act, cc_dtype_t dtype, int nranks, const cc_config_t* cfgp,
                                  cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_ffn(FfnBufs{x, w_in, w_out, none, y, none, none, none, none, ckpt, true}, counts, nexperts, capacity,
                   width, hidden, act, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, false, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_checkpoint_grad(cc_rankbuf_t ckpt, cc_rankbuf_t w_in, cc_rankbuf_t w_out, cc_rankbuf_t dy,
                                       cc_rankbuf_t dx, cc_rankbuf_t dw_in, cc_rankbuf_t dw_out, const size_t* counts,
                                       int nexperts, size_t capacity, size_t width, size_t hidden, cc_act_t act,
                                       cc_dtype_t dtype, int nranks, const cc_config_t* cfgp, cc_stream_t stream) {
  return guarded([&] {
    const cc_rankbuf_t none{nullptr, 0};
    return run_ffn(FfnBufs{none, w_in, w_out, none, none, dy, dx, dw_in, dw_out, ckpt, true}, counts, nexperts,
                   capacity, width, hidden, act, dtype, nranks, cfgp ? *cfgp : kDefaultCfg, true, (hipStream_t)stream);
  });
}

cc_status_t cc_moe_ffn_checkpoint_row(size_t width, size_t hidden, size_t* bytes) {
  if (width == 0 || hidden == 0 || width >= (1ull << 24) || hidden >= (1ull << 24))
    return fail(CC_ERR_INVALID_ARG, "width or hidden outside [1, 2^24)");
  if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = (size_t)ckpt_row(width, hidden).pitch;
  return ok();
}

cc_status_t cc_moe_ffn_checkpoint_workspace_size(const size_t* counts, int nexperts, size_t capacity, size_t width,
                                                 size_t hidden, cc_dtype_t dtype, int nranks, int grad, size_t* bytes) {
  return guarded([&] {
    FfnShape sh;
    std::vector<uint32_t> kept;
    cc_status_t s = model_checks(nranks, dtype, kDefaultCfg);
    if (s || (s = ffn_shape(counts, nexperts, capacity, width, hidden, dtype, nranks, &sh, &kept))) return s;
    if (grad != 0 && grad != 1) return fail(CC_ERR_INVALID_ARG, "grad=%d is neither 0 nor 1", grad);
    if (!bytes) return fail(CC_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)ffn_ws(sh, grad, 1).bytes;
    return ok();
  });
}

}  // extern "C"
