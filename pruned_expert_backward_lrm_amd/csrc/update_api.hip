// Host side of the update of the parameters: argument validation, the table of
// tensors and the launch sequences.
#include <cmath>

#include "lrm.h"
#include "api.h"
#include "update.h"

using namespace lrm;

namespace {

bool on(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// The descriptor and its tensors; step: they are to be updated, not only read.
// total: their chunks.
lrm_status check_params(const lrm_params* ps, bool step, int64_t* total) {
  if (!ps) return LRM_ERR_NULL;
  if (ps->n < 0 || ps->n > kMaxTensors) return LRM_ERR_SHAPE;
  if ((ps->p_dtype != LRM_F32 && ps->p_dtype != LRM_BF16) ||
      (ps->g_dtype != LRM_F32 && ps->g_dtype != LRM_BF16))
    return LRM_ERR_DTYPE;
  if (ps->moments != LRM_MOMENTS_F32 && ps->moments != LRM_MOMENTS_8BIT) return LRM_ERR_UNSUPPORTED;
  if (ps->masters != 0 && ps->masters != 1) return LRM_ERR_UNSUPPORTED;
  if (ps->masters && ps->p_dtype != LRM_BF16) return LRM_ERR_UNSUPPORTED;
  if (!ps->table || (ps->n > 0 && !ps->param)) return LRM_ERR_NULL;
  if (!on(ps->table, kAlign)) return LRM_ERR_ALIGN;
  const bool eight = ps->moments == LRM_MOMENTS_8BIT;
  int64_t chunks = 0;
  for (int i = 0; i < ps->n; ++i) {
    const lrm_param& q = ps->param[i];
    if (q.n < 0 || q.n > (1ll << 40)) return LRM_ERR_SHAPE;
    chunks += (q.n + kChunk - 1) / kChunk;
    if (!std::isfinite(q.lr) || q.lr < 0.f || !std::isfinite(q.weight_decay)) return LRM_ERR_UNSUPPORTED;
    if (q.n == 0) continue;
    if (!q.g) return LRM_ERR_NULL;
    if (!on(q.g, esize(ps->g_dtype))) return LRM_ERR_ALIGN;
    const bool reads = !q.p && !q.m && !q.v && !q.master && !q.m_exp && !q.v_exp;
    if (reads && !step) continue;
    if (!q.p || !q.m || !q.v) return LRM_ERR_NULL;
    if ((q.master != nullptr) != (ps->masters == 1)) return LRM_ERR_NULL;
    if ((q.m_exp != nullptr) != eight || (q.v_exp != nullptr) != eight) return LRM_ERR_NULL;
    if (!on(q.p, esize(ps->p_dtype)) || !on(q.master, 4)) return LRM_ERR_ALIGN;
    if (!eight && (!on(q.m, 4) || !on(q.v, 4))) return LRM_ERR_ALIGN;
  }
  *total = chunks;
  return LRM_OK;
}

ParamTable table_of(const lrm_params* ps) {
  ParamTable t;
  t.n = ps->n;
  t.entry = static_cast<const ParamEntry*>(ps->table);
  t.chunk0 = reinterpret_cast<const int64_t*>(t.entry + ps->n);
  return t;
}

}  // namespace

extern "C" {

size_t lrm_params_table_size(int32_t n) {
  if (n < 0 || n > kMaxTensors) return 0;
  Carve c(nullptr);
  c.take<char>((int64_t)n * (sizeof(ParamEntry) + sizeof(int64_t)) + sizeof(int64_t));
  return c.size();
}

lrm_status lrm_params_table(lrm_params* ps, size_t table_bytes, void* stream) {
  int64_t chunks = 0, blocks = 0;
  LRM_TRY(check_params(ps, false, &chunks));
  if (table_bytes < lrm_params_table_size(ps->n)) return LRM_ERR_WORKSPACE;
  const bool eight = ps->moments == LRM_MOMENTS_8BIT;
  ps->chunks = chunks;
  chunks = 0;
  for (int first = 0; first == 0 || first < ps->n; first += kTableBatch) {
    TableBatch b{};
    const int count = ps->n - first < kTableBatch ? ps->n - first : kTableBatch;
    for (int i = 0; i < count; ++i) {
      const lrm_param& q = ps->param[first + i];
      ParamEntry& e = b.entry[i];
      e.p = q.p; e.g = q.g; e.master = q.master; e.m = q.m; e.v = q.v;
      e.m_exp = q.m_exp; e.v_exp = q.v_exp;
      e.n = q.n; e.chunk0 = chunks; e.block0 = blocks;
      e.lr = q.lr; e.decay = q.weight_decay;
      e.vec = on(q.p, 16) && on(q.g, 16) && on(q.master, 16) && on(q.m, eight ? 8 : 16) &&
              on(q.v, eight ? 8 : 16);
      chunks += (q.n + kChunk - 1) / kChunk;
      blocks += (q.n + kMomentBlock - 1) / kMomentBlock;
    }
    LRM_TRY_HIP(launch_params_table(b, first, count, ps->n, ps->chunks, ps->table, as_stream(stream)));
  }
  return LRM_OK;
}

size_t lrm_sumsq_workspace_size(const lrm_params* ps) {
  int64_t chunks;
  if (check_params(ps, false, &chunks) != LRM_OK) return 0;
  Carve c(nullptr);
  c.take<double>(kSumBlocks);
  return c.size();
}

lrm_status lrm_grad_sumsq(const lrm_params* ps, double* sumsq, void* ws, size_t ws_bytes,
                          void* stream) {
  int64_t chunks;
  LRM_TRY(check_params(ps, false, &chunks));
  if (!sumsq) return LRM_ERR_NULL;
  if (!on(sumsq, 8)) return LRM_ERR_ALIGN;
  if (!ws || ws_bytes < kSumBlocks * sizeof(double)) return LRM_ERR_WORKSPACE;
  if (!on(ws, 8)) return LRM_ERR_ALIGN;
  if (ps->chunks != chunks) return LRM_ERR_SHAPE;  // (no table of these tensors)
  LRM_TRY_HIP(launch_grad_sumsq(table_of(ps), ps->chunks, ps->g_dtype == LRM_BF16,
                                static_cast<double*>(ws), sumsq, as_stream(stream)));
  return LRM_OK;
}

lrm_status lrm_adamw(const lrm_params* ps, const lrm_adamw_step* a, void* stream) {
  int64_t chunks;
  LRM_TRY(check_params(ps, true, &chunks));
  if (!a) return LRM_ERR_NULL;
  if (ps->chunks != chunks) return LRM_ERR_SHAPE;  // (no table of these tensors)
  if (!std::isfinite(a->lr) || a->lr < 0.0 || !std::isfinite(a->eps) || !(a->eps >= 1e-16) ||
      !std::isfinite(a->grad_scale) || !std::isfinite(a->max_norm) || a->max_norm < 0.0)
    return LRM_ERR_UNSUPPORTED;
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0) || !(a->beta2 >= 0.0 && a->beta2 < 1.0))
    return LRM_ERR_UNSUPPORTED;
  if (!a->steps && (a->step < 1 || a->step > (1ll << 53))) return LRM_ERR_SHAPE;
  if (a->n_sumsq < 0 || a->n_sumsq > 64 || (a->n_sumsq > 0) != (a->sumsq != nullptr))
    return LRM_ERR_SHAPE;
  if (a->max_norm > 0.0 && !a->sumsq) return LRM_ERR_NULL;
  if (!on(a->sumsq, 8) || !on(a->lr_dev, 4) || !on(a->steps, 8)) return LRM_ERR_ALIGN;
  AdamArgs g{};
  g.lr = (float)a->lr; g.grad_scale = a->grad_scale;
  g.over = a->max_norm > 0.0 ? a->max_norm / std::fabs(a->grad_scale) : HUGE_VAL;
  g.beta1 = a->beta1; g.beta2 = a->beta2;
  g.b1 = (float)a->beta1; g.d1 = (float)(1.0 - a->beta1);
  g.b2 = (float)a->beta2; g.d2 = (float)(1.0 - a->beta2);
  g.eps = (float)a->eps;
  g.ln1 = std::log(a->beta1); g.ln2 = std::log(a->beta2);
  g.bias = (float)(-1.0 / std::expm1((double)a->step * g.ln1));
  g.root = (float)(1.0 / std::sqrt(-std::expm1((double)a->step * g.ln2)));
  g.key = step_key(a->seed, (uint64_t)a->step);
  g.seed = a->seed; g.sumsq = a->sumsq; g.n_sumsq = a->n_sumsq;
  g.lr_dev = a->lr_dev; g.steps = a->steps;
  const int p = ps->masters ? 2 : (ps->p_dtype == LRM_BF16 ? 1 : 0);
  LRM_TRY_HIP(launch_adamw(table_of(ps), ps->chunks, p, ps->g_dtype == LRM_BF16,
                           ps->moments == LRM_MOMENTS_8BIT, g, a->steps, as_stream(stream)));
  return LRM_OK;
}

lrm_status lrm_moment_read(int64_t n, int32_t second, const void* codes, const uint8_t* exps,
                           int32_t dtype, void* out, void* stream) {
  if (n < 0 || n > (1ll << 40)) return LRM_ERR_SHAPE;
  if (second != 0 && second != 1) return LRM_ERR_UNSUPPORTED;
  if (dtype != LRM_F32 && dtype != LRM_BF16) return LRM_ERR_DTYPE;
  if (n > 0 && (!codes || !exps || !out)) return LRM_ERR_NULL;
  if (!on(out, esize(dtype))) return LRM_ERR_ALIGN;
  LRM_TRY_HIP(launch_moment_read(n, second, static_cast<const uint8_t*>(codes), exps,
                                 dtype == LRM_BF16, out, as_stream(stream)));
  return LRM_OK;
}

}  // extern "C"
