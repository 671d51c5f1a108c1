// Driver of the CPU-emulation build for the balance losses and the update of the
// parameters -- TEST INFRASTRUCTURE ONLY (see emu_driver.cpp).
//
//   emu_training IN OUT
//
// IN: 32 int64 (call, then the call's numbers, see main), then the arrays: each
// an int64 byte count and the bytes (-1: a NULL pointer).  Every array gets an
// allocation of exactly its bytes (behind `offset` elements of its own, where the
// call has one), so that any access past it is caught.  OUT: int32 status, int32
// 0, then every output array's bytes.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "lrm.h"

namespace {

std::vector<char> g_in;
size_t g_at = 0;

int64_t num() {
  int64_t v;
  std::memcpy(&v, g_in.data() + g_at, 8);
  g_at += 8;
  return v;
}
double real() {
  const int64_t v = num();
  double d;
  std::memcpy(&d, &v, 8);
  return d;
}

char* exact(size_t bytes) {
  char* p = static_cast<char*>(std::malloc(bytes ? bytes : 1));
  if (!p || (reinterpret_cast<uintptr_t>(p) & 15)) std::exit(3);
  return p;
}

struct Out {
  void* p;
  size_t n;
};
std::vector<Out> g_outs;

// an input, `skip` bytes behind the start of its allocation; out: written back
template <class T>
T* in(bool out = false, size_t skip = 0) {
  const int64_t n = num();
  if (n < 0) return nullptr;
  char* p = exact((size_t)n + skip) + skip;
  std::memcpy(p, g_in.data() + g_at, (size_t)n);
  g_at += (size_t)n;
  if (out) g_outs.push_back({p, (size_t)n});
  return reinterpret_cast<T*>(p);
}
template <class T>
T* outp(int64_t n) {
  if (n < 0) return nullptr;
  char* p = exact((size_t)n);
  std::memset(p, 0xCD, (size_t)n);
  g_outs.push_back({p, (size_t)n});
  return reinterpret_cast<T*>(p);
}
void* ws_of(size_t bytes) {
  void* p = std::aligned_alloc(256, (bytes + 255) / 256 * 256);
  std::memset(p, 0xCD, bytes);
  return p;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  FILE* fi = std::fopen(argv[1], "rb");
  if (!fi) return 2;
  char chunk[1 << 16];
  size_t got;
  while ((got = std::fread(chunk, 1, sizeof chunk, fi)) > 0)
    g_in.insert(g_in.end(), chunk, chunk + got);
  std::fclose(fi);
  int64_t h[32];
  for (int64_t& v : h) v = num();
  int32_t status = -1;
  const int32_t zero = 0;
  if (h[0] == 0 || h[0] == 1) {  // balance_loss, balance_bwd
    lrm_balance b{};
    lrm_router& r = b.router;
    r.T = (int32_t)h[1]; r.E = (int32_t)h[2]; r.k = (int32_t)h[3]; r.score = (int32_t)h[4];
    r.flags = (uint32_t)h[5]; r.n_group = r.topk_group = 1; r.scale = 1.f; r.dtype = (int32_t)h[6];
    r.ld = h[7]; b.S = (int32_t)h[8];
    b.coef = (float)real(); b.z_coef = (float)real();
    r.logits = in<char>(); r.expert_mask = in<uint8_t>(); r.token_mask = in<uint8_t>();
    b.expert = in<int32_t>(); b.counts = in<int32_t>(); b.seq = in<int32_t>();
    if (h[0] == 0) {
      float* loss = outp<float>(8);
      float* saved = outp<float>(((int64_t)b.S * r.E + 2) * 4);
      int32_t* counts = outp<int32_t>(b.counts ? -1 : (int64_t)b.S * r.E * 4);
      const size_t n = lrm_balance_workspace_size(&b);
      status = n ? lrm_balance_loss(&b, loss, saved, counts, ws_of(n), n, nullptr) : -1;
    } else {
      const float* saved = in<float>(); const float* dloss = in<float>();
      const float* dw = in<float>();
      status = lrm_balance_bwd(&b, saved, dloss, dw, outp<char>(h[9]), h[10], nullptr);
    }
  } else if (h[0] == 2) {  // the sum of squares, then a step
    lrm_params ps{};
    ps.n = (int32_t)h[1]; ps.p_dtype = (int32_t)h[2]; ps.g_dtype = (int32_t)h[3];
    ps.moments = (int32_t)h[4]; ps.masters = (int32_t)h[5];
    const size_t skip = (size_t)h[6];
    lrm_adamw_step a{};
    a.lr = real(); a.beta1 = real(); a.beta2 = real(); a.eps = real(); a.grad_scale = real();
    a.max_norm = real(); a.step = num(); a.seed = (uint64_t)num();
    std::vector<lrm_param> q((size_t)ps.n);
    for (lrm_param& t : q) {
      t.n = num(); t.lr = (float)real(); t.weight_decay = (float)real();
      t.g = in<char>(false, skip * (ps.g_dtype == LRM_BF16 ? 2 : 4));
      t.p = in<char>(true, skip * (ps.p_dtype == LRM_BF16 ? 2 : 4));
      t.master = in<float>(true, skip * 4);
      t.m = in<char>(true, skip * (ps.moments ? 1 : 4));
      t.v = in<char>(true, skip * (ps.moments ? 1 : 4));
      t.m_exp = in<uint8_t>(true, skip); t.v_exp = in<uint8_t>(true, skip);
    }
    float* lr_dev = in<float>();
    int64_t* steps = in<int64_t>(true);
    ps.param = q.data();
    const size_t nt = lrm_params_table_size(ps.n);
    ps.table = ws_of(nt);
    status = lrm_params_table(&ps, nt, nullptr);
    double* sumsq = outp<double>(8);
    const size_t n = lrm_sumsq_workspace_size(&ps);
    if (status == LRM_OK) status = lrm_grad_sumsq(&ps, sumsq, ws_of(n), n, nullptr);
    a.lr_dev = lr_dev; a.steps = steps;
    if (h[7]) { a.sumsq = sumsq; a.n_sumsq = 1; }
    if (status == LRM_OK) status = lrm_adamw(&ps, &a, nullptr);
  } else {  // the values of moments
    const size_t skip = (size_t)h[4];
    const char* codes = in<char>(false, skip); const uint8_t* exps = in<uint8_t>();
    status = lrm_moment_read(h[1], (int32_t)h[2], codes, exps, (int32_t)h[3], outp<char>(h[5]), nullptr);
  }
  FILE* fo = std::fopen(argv[2], "wb");
  if (!fo) return 2;
  std::fwrite(&status, 4, 1, fo);
  std::fwrite(&zero, 4, 1, fo);
  for (const Out& o : g_outs)
    if (o.n && std::fwrite(o.p, 1, o.n, fo) != o.n) return 4;
  std::fclose(fo);
  return 0;
}
