// Host side of the router, the experts' forward pass and its epilogue's
// backward pass: argument validation, workspace planning and the launch
// sequences (the same conventions as the backward's entry points).
#include <cmath>

#include "lrm.h"
#include "api.h"
#include "common.h"
#include "launch.h"

using namespace lrm;

namespace {

// ---------------------------------------------------------------- router

lrm_status check_router(const lrm_router* r) {
  if (!r) return LRM_ERR_NULL;
  if (r->T < 0 || r->E < 1 || r->E > kMaxE) return LRM_ERR_SHAPE;
  if (r->k < 1 || r->k > r->E || r->k > 64) return LRM_ERR_SHAPE;
  if ((int64_t)r->T * r->k > 0x7fffffffll) return LRM_ERR_SHAPE;
  if (r->n_group < 1 || r->n_group > 64 || r->E % r->n_group != 0) return LRM_ERR_SHAPE;
  if (r->topk_group < 1 || r->topk_group > r->n_group) return LRM_ERR_SHAPE;
  if (r->dtype != LRM_F32 && r->dtype != LRM_BF16) return LRM_ERR_DTYPE;
  if (r->score != LRM_SOFTMAX && r->score != LRM_SIGMOID) return LRM_ERR_UNSUPPORTED;
  if (r->group_rule != LRM_GROUP_MAX && r->group_rule != LRM_GROUP_TOP2)
    return LRM_ERR_UNSUPPORTED;
  if (r->flags & ~LRM_ROUTE_RENORM) return LRM_ERR_UNSUPPORTED;
  if (!std::isfinite(r->scale)) return LRM_ERR_UNSUPPORTED;
  if (r->ld < r->E) return LRM_ERR_SHAPE;
  if (r->T > 0 && !r->logits) return LRM_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(r->logits) % esize(r->dtype) != 0) return LRM_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(r->bias) & 3u) != 0) return LRM_ERR_ALIGN;
  return LRM_OK;
}

bool rows16(const void* p, int64_t ld, int dtype) {
  return aligned16(p) && (ld * esize(dtype)) % 16 == 0;
}

RouteArgs route_args(const lrm_router* r) {
  RouteArgs a{};
  a.T = r->T; a.E = r->E; a.k = r->k;
  a.softmax = r->score == LRM_SOFTMAX;
  a.renorm = (r->flags & LRM_ROUTE_RENORM) != 0;
  a.n_group = r->n_group; a.topk_group = r->topk_group;
  a.group_top2 = r->group_rule == LRM_GROUP_TOP2;
  a.bf16 = r->dtype == LRM_BF16;
  a.vec = rows16(r->logits, r->ld, r->dtype);
  a.scale = r->scale;
  a.logits = r->logits; a.ld = r->ld;
  a.bias = r->bias; a.expert_mask = r->expert_mask; a.token_mask = r->token_mask;
  return a;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// ---------------------------------------------------------------- balance

lrm_status check_balance(const lrm_balance* b) {
  if (!b) return LRM_ERR_NULL;
  LRM_TRY(check_router(&b->router));
  if (b->S < 1 || b->S > (1 << 20) || (int64_t)b->S * b->router.E > 0x7fffffffll)
    return LRM_ERR_SHAPE;
  if (!b->seq && b->S != 1) return LRM_ERR_SHAPE;
  if (!std::isfinite(b->coef) || !std::isfinite(b->z_coef)) return LRM_ERR_UNSUPPORTED;
  if (b->z_coef != 0.f && b->router.score != LRM_SOFTMAX) return LRM_ERR_UNSUPPORTED;
  if (!aligned4(b->expert) || !aligned4(b->counts) || !aligned4(b->seq)) return LRM_ERR_ALIGN;
  return LRM_OK;
}

BalanceArgs carve_balance(Carve& c, const lrm_balance* b) {
  BalanceArgs g{};
  const int E = b->router.E, T = b->router.T;
  g.S = b->S;
  g.chunk = balance_chunk(T, E, b->router.k);
  g.chunks = (int)(((int64_t)T + g.chunk - 1) / g.chunk);
  g.rows = c.take<BalanceRow>((int64_t)g.chunks + b->S);
  g.blocks = c.take<double>((int64_t)balance_join_blocks(b->S) * 4);
  if (!b->counts) g.cnt = c.take<int32_t>((int64_t)b->S * E);
  return g;
}

// --------------------------------------------------------------- bucketing
// The pairs in expert order (every pair kept), as the backward's bucketing
// with LRM_KEEP_ALL makes it.
struct BucketWs {
  uint32_t* err;
  uint32_t* blkerr;
  int32_t* blkcnt;
  int32_t* cand_off;
  int32_t* offsets;
  int32_t* kept;
  int32_t* pos;
  int32_t* tokens;
  int32_t* tok_off;
  int32_t* mt_off;
};

// (err first: it is the workspace's error word)
BucketWs carve_bucket(Carve& c, const lrm_pairs* p) {
  BucketWs w;
  w.err = c.take<uint32_t>(64);
  w.blkerr = c.take<uint32_t>(bucket_blocks(p->N));
  w.blkcnt = c.take<int32_t>((int64_t)bucket_blocks(p->N) * p->E);
  w.cand_off = c.take<int32_t>(p->E + 1);
  w.offsets = c.take<int32_t>(p->E + 1);
  w.kept = c.take<int32_t>(p->N);
  w.pos = c.take<int32_t>(p->N);
  w.tokens = c.take<int32_t>(p->N);
  w.tok_off = c.take<int32_t>((int64_t)p->T + 1);
  w.mt_off = c.take<int32_t>(p->E + 1);
  return w;
}

hipError_t run_bucket(const lrm_pairs* p, const BucketWs& w, bool tok, int mt_bm, hipStream_t s) {
  BucketArgs b{};
  b.N = p->N; b.T = p->T; b.E = p->E; b.token = p->token; b.expert = p->expert;
  b.blkcnt = w.blkcnt; b.cand_off = w.cand_off; b.offsets = w.offsets; b.cand = w.kept;
  b.pos = w.pos; b.tokens = w.tokens; b.keep_all = 1; b.err = w.err; b.blkerr = w.blkerr;
  b.tok_off = tok && p->N > 0 ? w.tok_off : nullptr;
  b.mt_off = mt_bm > 0 ? w.mt_off : nullptr; b.mt_bm = mt_bm; b.max_kept = -1;
  hipError_t e = launch_bucket(b, s);
  if (e == hipSuccess && tok && p->N == 0) e = launch_token_offsets(0, p->T, p->token, w.tok_off, s);
  return e;
}

// ------------------------------------------------------------ forward pass

lrm_status check_forward(const lrm_forward* f, const lrm_forward_outputs* out) {
  if (!f) return LRM_ERR_NULL;
  LRM_TRY(check_pairs(&f->pairs));
  if (f->dtype != LRM_F32 && f->dtype != LRM_BF16) return LRM_ERR_DTYPE;
  const lrm_pairs* p = &f->pairs;
  const int q = 16 / esize(f->dtype);
  int d_out;
  if (f->kind == LRM_LINEAR) {
    if (f->act < LRM_ACT_NONE || f->act > LRM_ACT_SILU) return LRM_ERR_UNSUPPORTED;
    if (f->d_in <= 0 || f->d_out <= 0 || f->d_in > kMaxDim || f->d_out > kMaxDim)
      return LRM_ERR_SHAPE;
    LRM_TRY(check_mat(&f->X, p, f->dtype, f->d_in, -1));
    if (f->d_out % q) return LRM_ERR_UNSUPPORTED;
    if (!f->W) return LRM_ERR_NULL;
    if (!aligned16(f->W) || !aligned16(f->bias)) return LRM_ERR_ALIGN;
    if (f->w_stride < (int64_t)f->d_in * f->d_out) return LRM_ERR_SHAPE;
    if ((f->w_stride * esize(f->dtype)) % 16) return LRM_ERR_ALIGN;
    d_out = f->d_out;
  } else if (f->kind == LRM_SWIGLU) {
    if (f->act != LRM_ACT_NONE || f->bias) return LRM_ERR_UNSUPPORTED;
    if (f->H <= 0 || f->I <= 0 || f->H > kMaxDim || f->I > kMaxDim) return LRM_ERR_SHAPE;
    if (f->H % q || f->I % q) return LRM_ERR_UNSUPPORTED;
    LRM_TRY(check_mat(&f->X, p, f->dtype, f->H, LRM_ROWS_TOKEN));
    if (!f->W_gate || !f->W_up || !f->W_down) return LRM_ERR_NULL;
    if (!aligned16(f->W_gate) || !aligned16(f->W_up) || !aligned16(f->W_down))
      return LRM_ERR_ALIGN;
    d_out = f->H;
  } else {
    return LRM_ERR_UNSUPPORTED;
  }
  if (f->R.ptr) LRM_TRY(check_mat(&f->R, p, f->dtype, d_out, LRM_ROWS_TOKEN));
  if (out) {
    const bool glu = f->kind == LRM_SWIGLU;
    if (glu ? out->Z != nullptr : (out->A || out->B || out->h_sumsq)) return LRM_ERR_UNSUPPORTED;
    // (outputs of no rows may be null)
    if (p->N > 0 && !out->Y && !out->Yp && !out->Z && !out->A && !out->B && !out->h_sumsq)
      return LRM_ERR_NULL;
    if (f->R.ptr && !out->Y) return LRM_ERR_UNSUPPORTED;
    if (!aligned16(out->Y) || !aligned16(out->Yp) || !aligned16(out->Z) || !aligned16(out->A) ||
        !aligned16(out->B) || (reinterpret_cast<uintptr_t>(out->h_sumsq) & 7u))
      return LRM_ERR_ALIGN;
  }
  return LRM_OK;
}

// Few pairs: at most kFewPairs, and on average at most kFewRows an expert
// (Qwen3-shaped layer, 128 experts, top-8: 2 tokens 31 us against 45 with the
// tiles, 4 tokens 65 and 63, 8 tokens 110 and 116; a projection 1024 x 1408 of 8
// experts in fp32: 64 pairs 22 us and 54).
// (LRM_FWD_TILE keeps the tiles.)
constexpr int kFewRows = 8;
bool few_pairs(const lrm_pairs* p) {
  return p->N <= kFewPairs && p->T <= 65535 && p->N <= (int64_t)kFewRows * p->E;
}
// Few enough that a token's pairs are joined where they are multiplied, each
// token reading its experts' weights on its own, a block for 8 columns of every
// token (a token should bring two of its eight waves a pair, and one without
// pairs brings none: 2 T <= N; a lone token shares no expert).  Joined against the
// products and the sum apart, us, weights from memory:
//   128 experts, 2048/768: 1 token of 8 pairs 35 and 40, 2 tokens 51 and 57, 4
//     tokens 84 and 87; 4 tokens of 2 pairs 39 and 38, of 1 pair 31 and 27
//   32 experts, 4096/1408: 1 token of 8 pairs 70 and 75; 2 of 1 pair 42 and 37
//   64 experts, 1024/512: 4 tokens of 4 pairs 25 and 30
//   8 pairs among 4096 tokens (128 experts, 2048/768): 2392 and 30
bool few_join(const lrm_pairs* p) {
  return p->T == 1 || ((int64_t)p->N * 4 <= p->E && 2ll * p->T <= p->N);
}

struct FwdWs {
  BucketWs b;
  float* Yf;     // few pairs: y in fp32, [N][d_out]
  void* H;       // SWIGLU: packed silu(a) b, [N][I] (fp32 where few_join takes it)
  void* Yp;      // [N][d_out]
  int8_t* Ylo;   // bf16: [N][d_out]
  void* dump;    // 1 KB that lanes outside a tile store to
  void* Xp;      // X in packed order, where X is too large to gather from
};

int64_t x_bytes(const lrm_forward* f) {
  const int64_t rows = f->X.rows == LRM_ROWS_PAIR ? f->pairs.N : f->pairs.T;
  return rows > 0 ? ((rows - 1) * f->X.ld + f->X.cols) * esize(f->dtype) : 0;
}

FwdWs carve_forward(Carve& c, const lrm_forward* f) {
  FwdWs w{};
  const int64_t N = f->pairs.N;
  const int es = esize(f->dtype);
  const bool glu = f->kind == LRM_SWIGLU;
  const int64_t d = glu ? f->H : f->d_out;
  w.b = carve_bucket(c, &f->pairs);
  const bool h32 = few_pairs(&f->pairs) && few_join(&f->pairs);
  if (glu) w.H = c.take<char>(N * f->I * (h32 ? 4 : es));
  w.Yp = c.take<char>(N * d * es);
  if (f->dtype == LRM_BF16) w.Ylo = c.take<int8_t>(N * d);
  if (few_pairs(&f->pairs)) w.Yf = c.take<float>(N * d);
  w.dump = c.take<char>(1024);
  if (x_bytes(f) > kFwdGatherMax) w.Xp = c.take<char>(N * f->X.cols * es);
  return w;
}

lrm_status run_few(const lrm_forward* f, const lrm_forward_outputs* out, void* ws, hipStream_t s) {
  const lrm_pairs* p = &f->pairs;
  const bool glu = f->kind == LRM_SWIGLU;
  const bool joined = out->Y && glu && few_join(p);
  Carve c(ws);
  const FwdWs w = carve_forward(c, f);
  FwdFewArgs g{};
  g.N = p->N; g.T = p->T; g.E = p->E; g.bf16 = f->dtype == LRM_BF16;
  g.by_pair = p->N <= p->E;
  g.token = p->token; g.expert = p->expert; g.weight = p->weight;
  g.X = f->X.ptr; g.ldx = f->X.ld; g.x_pair = f->X.rows == LRM_ROWS_PAIR;
  g.err = w.b.err;
  if (p->N == 0) LRM_TRY_HIP(launch_fill_u32(w.b.err, 0u, 1, s));
  if (glu) {
    g.glu = 1; g.K = f->H; g.n = f->I;
    g.W0 = f->W_gate; g.W1 = f->W_up; g.w_stride = (int64_t)f->H * f->I;
    g.A = out->A; g.B = out->B; g.H = w.H;
    g.h32 = joined;
    LRM_TRY_HIP(launch_fwd_few(g, s));
    if (out->h_sumsq) LRM_TRY_HIP(launch_fwd_few_sumsq(g, out->h_sumsq, s));
    g.glu = 0; g.K = f->I; g.n = f->H; g.X = w.H; g.ldx = f->I; g.x_pair = 1;
    g.W0 = f->W_down; g.W1 = nullptr; g.err = nullptr;
  } else {
    g.K = f->d_in; g.n = f->d_out; g.act = f->act; g.W0 = f->W; g.w_stride = f->w_stride;
    g.bias = f->bias; g.Z = out->Z;
  }
  g.Y = out->Yp; g.out = out->Y; g.R = f->R.ptr; g.ldr = f->R.ld;
  // (the joining product reports no index errors: GLU's first product has, and
  // one projection without it takes the other way)
  if (joined) {
    LRM_TRY_HIP(launch_fwd_few_join(g, s));
    return LRM_OK;
  }
  if (out->Y) g.Yf = w.Yf;
  if (g.Y || g.Z || g.Yf) LRM_TRY_HIP(launch_fwd_few(g, s));
  if (out->Y) LRM_TRY_HIP(launch_fwd_few_sum(g, s));
  return LRM_OK;
}

lrm_status run_forward(const lrm_forward* f, const lrm_forward_outputs* out, void* ws,
                       hipStream_t s) {
  const lrm_pairs* p = &f->pairs;
  if (few_pairs(p) && !fwd_tile_forced()) return run_few(f, out, ws, s);
  const bool glu = f->kind == LRM_SWIGLU;
  const bool bf16 = f->dtype == LRM_BF16;
  Carve c(ws);
  const FwdWs w = carve_forward(c, f);
  FwdGemmArgs g{};
  g.N = p->N; g.E = p->E; g.bf16 = bf16;
  g.offsets = w.b.offsets; g.kept = w.b.kept; g.mt_off = w.b.mt_off; g.dump = w.dump;
  g.rows = f->X.rows == LRM_ROWS_PAIR ? w.b.kept : w.b.tokens;
  g.gather = 1; g.X = f->X.ptr; g.ldx = f->X.ld;
  LRM_TRY_HIP(run_bucket(p, w.b, out->Y != nullptr, fwd_tile_rows(g), s));
  g.x_bytes = x_bytes(f);
  if (w.Xp) {
    g.K = f->X.cols;
    LRM_TRY_HIP(launch_fwd_pack(g, w.Xp, s));
    g.gather = 0; g.X = w.Xp; g.ldx = g.K;
  }
  const bool y_wanted = out->Y || out->Yp;
  void* const Y = out->Yp ? out->Yp : (out->Y ? w.Yp : nullptr);
  int d;
  if (glu) {
    d = f->H;
    g.glu = 1; g.K = f->H; g.n = f->I;
    g.W0 = f->W_gate; g.W1 = f->W_up; g.w_stride = (int64_t)f->H * f->I;
    g.A = out->A; g.B = out->B; g.H = w.H;
    LRM_TRY_HIP(launch_fwd_gemm(g, s));
    if (out->h_sumsq) LRM_TRY_HIP(launch_fwd_sumsq(g, out->h_sumsq, s));
    g.glu = 0; g.K = f->I; g.n = f->H; g.gather = 0; g.X = w.H; g.ldx = f->I;
    g.W0 = f->W_down; g.W1 = nullptr;
  } else {
    d = f->d_out;
    g.K = f->d_in; g.n = f->d_out; g.act = f->act; g.W0 = f->W; g.w_stride = f->w_stride;
    g.bias = f->bias; g.Z = out->Z;
  }
  if (y_wanted || g.Z) {
    g.Y = Y;
    g.Ylo = bf16 && out->Y ? w.Ylo : nullptr;
    LRM_TRY_HIP(launch_fwd_gemm(g, s));
  }
  if (out->Y) {
    FwdJoinArgs j{};
    j.N = p->N; j.T = p->T; j.d = d; j.bf16 = bf16; j.tok_off = w.b.tok_off; j.pos = w.b.pos;
    j.weight = p->weight; j.Y = Y; j.Ylo = w.Ylo; j.R = f->R.ptr; j.ldr = f->R.ld; j.out = out->Y;
    LRM_TRY_HIP(launch_fwd_join(j, s));
  }
  return LRM_OK;
}

// ------------------------------------------------------ epilogue backward

lrm_status check_pair_grad(const lrm_pair_grad_problem* g, const lrm_pair_grad_outputs* out) {
  if (!g) return LRM_ERR_NULL;
  LRM_TRY(check_pairs(&g->pairs));
  if (g->dtype != LRM_F32 && g->dtype != LRM_BF16) return LRM_ERR_DTYPE;
  if (g->act < LRM_ACT_NONE || g->act > LRM_ACT_SILU) return LRM_ERR_UNSUPPORTED;
  if (g->Z.cols > kMaxDim) return LRM_ERR_SHAPE;
  LRM_TRY(check_mat(&g->Z, &g->pairs, g->dtype, -1, LRM_ROWS_PAIR));
  LRM_TRY(check_mat(&g->dY, &g->pairs, g->dtype, g->Z.cols, -1));
  if (out) {
    if (g->pairs.N > 0 && !out->dweight && !out->G && !out->dbias) return LRM_ERR_NULL;
    if (!aligned4(out->dweight) || !aligned16(out->G) || !aligned4(out->dbias))
      return LRM_ERR_ALIGN;
  }
  return LRM_OK;
}

struct PairGradWs {
  BucketWs b;
  float* part;
};

PairGradWs carve_pair_grad(Carve& c, const lrm_pair_grad_problem* g) {
  PairGradWs w;
  w.b = carve_bucket(c, &g->pairs);
  w.part = c.take<float>((int64_t)pair_grad_splits(g->pairs.N, g->pairs.E) * g->pairs.E * g->Z.cols);
  return w;
}

}  // namespace

extern "C" {

size_t lrm_route_workspace_size(const lrm_router* r) {
  if (check_router(r) != LRM_OK) return 0;
  Carve c(nullptr);
  c.take<int32_t>((int64_t)kRouteBlocks * r->E);
  return c.size();
}

lrm_status lrm_route(const lrm_router* r, int32_t* expert, float* weight, int32_t* token,
                     int32_t* counts, void* ws, size_t ws_bytes, void* stream) {
  LRM_TRY(check_router(r));
  if (r->T > 0 && (!expert || !weight)) return LRM_ERR_NULL;
  if (!aligned4(expert) || !aligned4(weight) || !aligned4(token) || !aligned4(counts))
    return LRM_ERR_ALIGN;
  if (counts && (!ws || ws_bytes < lrm_route_workspace_size(r))) return LRM_ERR_WORKSPACE;
  if (counts && !aligned4(ws)) return LRM_ERR_ALIGN;
  RouteArgs a = route_args(r);
  a.expert = expert; a.weight = weight; a.token = token;
  a.counts = static_cast<int32_t*>(ws);
  LRM_TRY_HIP(launch_route(a, counts, as_stream(stream)));
  return LRM_OK;
}

lrm_status lrm_route_bwd(const lrm_router* r, const int32_t* expert, const float* dweight,
                         void* dlogits, int64_t ldd, void* stream) {
  LRM_TRY(check_router(r));
  if (r->T > 0 && (!expert || !dweight || !dlogits)) return LRM_ERR_NULL;
  if (ldd < r->E) return LRM_ERR_SHAPE;
  if (!aligned4(expert) || !aligned4(dweight) ||
      reinterpret_cast<uintptr_t>(dlogits) % esize(r->dtype) != 0)
    return LRM_ERR_ALIGN;
  LRM_TRY_HIP(launch_route_bwd(route_args(r), expert, dweight, dlogits, ldd,
                               rows16(dlogits, ldd, r->dtype), as_stream(stream)));
  return LRM_OK;
}

size_t lrm_balance_workspace_size(const lrm_balance* b) {
  if (check_balance(b) != LRM_OK) return 0;
  Carve c(nullptr);
  carve_balance(c, b);
  return c.size();
}

lrm_status lrm_balance_loss(const lrm_balance* b, float* loss, float* saved, int32_t* counts,
                            void* ws, size_t ws_bytes, void* stream) {
  LRM_TRY(check_balance(b));
  if (!loss || !saved) return LRM_ERR_NULL;
  if (!b->counts && !b->expert && b->router.T > 0) return LRM_ERR_NULL;
  if (b->counts && counts) return LRM_ERR_UNSUPPORTED;
  if (!aligned4(loss) || !aligned4(saved) || !aligned4(counts)) return LRM_ERR_ALIGN;
  if (!ws || ws_bytes < lrm_balance_workspace_size(b)) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return LRM_ERR_ALIGN;
  Carve c(ws);
  BalanceArgs g = carve_balance(c, b);
  g.coef = b->coef; g.z_coef = b->z_coef;
  g.expert = b->expert; g.counts = b->counts; g.seq = b->seq;
  g.loss = loss; g.saved = saved; g.counts_out = counts;
  LRM_TRY_HIP(launch_balance(route_args(&b->router), g, as_stream(stream)));
  return LRM_OK;
}

lrm_status lrm_balance_bwd(const lrm_balance* b, const float* saved, const float* dloss,
                           const float* dweight, void* dlogits, int64_t ldd, void* stream) {
  LRM_TRY(check_balance(b));
  const lrm_router* r = &b->router;
  if (!saved || (r->T > 0 && (!dlogits || (dweight && !b->expert)))) return LRM_ERR_NULL;
  if (ldd < r->E) return LRM_ERR_SHAPE;
  if (!aligned4(saved) || !aligned4(dloss) || !aligned4(dweight) ||
      reinterpret_cast<uintptr_t>(dlogits) % esize(r->dtype) != 0)
    return LRM_ERR_ALIGN;
  BalanceBwdArgs g{};
  g.S = b->S; g.vec_out = rows16(dlogits, ldd, r->dtype); g.ldd = ldd;
  g.expert = b->expert; g.seq = b->seq; g.saved = saved; g.dloss = dloss;
  g.dweight = dweight; g.dlogits = dlogits;
  LRM_TRY_HIP(launch_balance_bwd(route_args(r), g, as_stream(stream)));
  return LRM_OK;
}

size_t lrm_route_share_workspace_size(int32_t T, int32_t k) {
  if (T < 0 || k < 1 || (int64_t)T * k > 0x7fffffffll) return 0;
  Carve c(nullptr);
  c.take<int32_t>(kShareBlocks);
  return c.size();
}

lrm_status lrm_route_share(int32_t T, int32_t k, const int32_t* expert, const float* weight,
                           int32_t e0, int32_t E, int32_t* out_token, int32_t* out_expert,
                           float* out_weight, int32_t* out_slot, int32_t* out_n, void* ws,
                           size_t ws_bytes, void* stream) {
  if (T < 0 || k < 1 || (int64_t)T * k > 0x7fffffffll) return LRM_ERR_SHAPE;
  if (e0 < 0 || E < 1 || E > kMaxE) return LRM_ERR_SHAPE;
  if (!out_n) return LRM_ERR_NULL;
  if (T > 0 && (!expert || !weight || !out_expert || !out_weight)) return LRM_ERR_NULL;
  if (!aligned4(expert) || !aligned4(weight) || !aligned4(out_token) || !aligned4(out_expert) ||
      !aligned4(out_weight) || !aligned4(out_slot) || !aligned4(out_n) || !aligned4(ws))
    return LRM_ERR_ALIGN;
  if (!ws || ws_bytes < lrm_route_share_workspace_size(T, k)) return LRM_ERR_WORKSPACE;
  LRM_TRY_HIP(launch_route_share((int64_t)T * k, k, expert, weight, e0, E, out_token, out_expert,
                                 out_weight, out_slot, out_n, static_cast<int32_t*>(ws),
                                 as_stream(stream)));
  return LRM_OK;
}

size_t lrm_forward_workspace_size(const lrm_forward* f) {
  if (check_forward(f, nullptr) != LRM_OK) return 0;
  Carve c(nullptr);
  carve_forward(c, f);
  return c.size();
}

lrm_status lrm_expert_forward(const lrm_forward* f, const lrm_forward_outputs* out, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!out) return LRM_ERR_NULL;
  LRM_TRY(check_forward(f, out));
  if (!ws || ws_bytes < lrm_forward_workspace_size(f)) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return LRM_ERR_ALIGN;
  return run_forward(f, out, ws, as_stream(stream));
}

size_t lrm_pair_grad_workspace_size(const lrm_pair_grad_problem* g) {
  if (check_pair_grad(g, nullptr) != LRM_OK) return 0;
  Carve c(nullptr);
  carve_pair_grad(c, g);
  return c.size();
}

lrm_status lrm_pair_grad(const lrm_pair_grad_problem* g, const lrm_pair_grad_outputs* out,
                         void* ws, size_t ws_bytes, void* stream) {
  if (!out) return LRM_ERR_NULL;
  LRM_TRY(check_pair_grad(g, out));
  if (!ws || ws_bytes < lrm_pair_grad_workspace_size(g)) return LRM_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return LRM_ERR_ALIGN;
  hipStream_t s = as_stream(stream);
  const lrm_pairs* p = &g->pairs;
  Carve c(ws);
  const PairGradWs w = carve_pair_grad(c, g);
  if (out->dbias) LRM_TRY_HIP(run_bucket(p, w.b, false, 0, s));
  PairGradArgs a{};
  a.N = p->N; a.T = p->T; a.E = p->E; a.d = g->Z.cols; a.bf16 = g->dtype == LRM_BF16;
  a.act = g->act; a.token = p->token; a.expert = p->expert; a.weight = p->weight;
  a.dY = g->dY.ptr; a.ldy = g->dY.ld; a.dy_pair = g->dY.rows == LRM_ROWS_PAIR;
  a.Z = g->Z.ptr; a.ldz = g->Z.ld;
  a.dweight = out->dweight; a.G = out->G; a.dbias = out->dbias;
  a.offsets = w.b.offsets; a.kept = w.b.kept; a.pos = w.b.pos; a.part = w.part; a.err = w.b.err;
  LRM_TRY_HIP(launch_pair_grad(a, s));
  return LRM_OK;
}

}  // extern "C"
