// Driver of the CPU-emulation build for the router, the experts' forward pass
// and its epilogue's backward pass -- TEST INFRASTRUCTURE ONLY (see
// emu_driver.cpp).
//
//   emu_forward IN OUT
//
// IN: 32 int64 (call, then the call's numbers, see main), then the input
// arrays: each an int64 byte count and the bytes (-1: a NULL pointer).  Every
// array gets an allocation of exactly its bytes, at the alignment asked for,
// so that any access past it is caught.  OUT: int32 status, int32 device
// status, then every output array's bytes.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "lrm.h"

namespace {

std::vector<char> g_in;
size_t g_at = 0;
FILE* g_out = nullptr;

int64_t num() {
  int64_t v;
  std::memcpy(&v, g_in.data() + g_at, 8);
  g_at += 8;
  return v;
}

// 16-byte aligned, with no byte to spare (aligned_alloc rounds sizes up)
void* exact(size_t bytes) {
  char* p = static_cast<char*>(std::malloc(bytes ? bytes : 1));
  if (!p || (reinterpret_cast<uintptr_t>(p) & 15)) std::exit(3);
  return p;
}

template <class T>
T* in() {
  const int64_t n = num();
  if (n < 0) return nullptr;
  void* p = exact((size_t)n);
  std::memcpy(p, g_in.data() + g_at, (size_t)n);
  g_at += (size_t)n;
  return static_cast<T*>(p);
}

struct Out {
  void* p;
  size_t n;
};
std::vector<Out> g_outs;

// an output of n bytes, all 0xCD before the call; n < 0: NULL
template <class T>
T* outp(int64_t n) {
  if (n < 0) return nullptr;
  void* p = exact((size_t)n);
  std::memset(p, 0xCD, (size_t)n);
  g_outs.push_back({p, (size_t)n});
  return static_cast<T*>(p);
}

void* ws_of(size_t bytes) {
  void* p = std::aligned_alloc(256, (bytes + 255) / 256 * 256 + 256);
  std::memset(p, 0xCD, bytes);
  return p;
}

lrm_mat mat(const void* p, int64_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  lrm_mat m{};
  m.ptr = p;
  m.dtype = (int32_t)dtype;
  m.rows = (int32_t)rows;
  m.cols = (int32_t)cols;
  m.ld = ld;
  return m;
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
  int32_t status = -1, dev = 0;
  if (h[0] == 0 || h[0] == 1) {  // route, route_bwd
    lrm_router r{};
    r.T = (int32_t)h[1]; r.E = (int32_t)h[2]; r.k = (int32_t)h[3]; r.score = (int32_t)h[4];
    r.flags = (uint32_t)h[5]; r.n_group = (int32_t)h[6]; r.topk_group = (int32_t)h[7];
    r.group_rule = (int32_t)h[8]; r.scale = (float)h[9] / 1024.f; r.dtype = (int32_t)h[10];
    r.ld = h[11];
    r.logits = in<char>(); r.bias = in<float>(); r.expert_mask = in<uint8_t>();
    r.token_mask = in<uint8_t>();
    if (h[0] == 0) {
      int32_t* e = outp<int32_t>(h[12]); float* w = outp<float>(h[12]);
      int32_t* t = outp<int32_t>(h[13]); int32_t* c = outp<int32_t>(h[14]);
      const size_t n = lrm_route_workspace_size(&r);
      status = lrm_route(&r, e, w, t, c, ws_of(n), n, nullptr);
    } else {
      const int32_t* e = in<int32_t>(); const float* dw = in<float>();
      status = lrm_route_bwd(&r, e, dw, outp<char>(h[12]), h[13], nullptr);
    }
  } else if (h[0] == 2) {  // share
    const int32_t* e = in<int32_t>(); const float* w = in<float>();
    int32_t* ot = outp<int32_t>(h[5]); int32_t* oe = outp<int32_t>(h[5]);
    float* ow = outp<float>(h[5]); int32_t* os = outp<int32_t>(h[5]);
    int32_t* on = outp<int32_t>(4);
    const size_t n = lrm_route_share_workspace_size((int32_t)h[1], (int32_t)h[2]);
    status = lrm_route_share((int32_t)h[1], (int32_t)h[2], e, w, (int32_t)h[3], (int32_t)h[4], ot,
                             oe, ow, os, on, ws_of(n), n, nullptr);
  } else {
    lrm_pairs p{};
    p.T = (int32_t)h[1]; p.N = (int32_t)h[2]; p.E = (int32_t)h[3];
    p.token = in<int32_t>(); p.expert = in<int32_t>(); p.weight = in<float>();
    const int64_t dt = h[5];
    void* ws = nullptr;
    if (h[0] == 3) {  // forward
      lrm_forward f{};
      f.kind = (int32_t)h[4]; f.dtype = (int32_t)dt; f.act = (int32_t)h[6]; f.pairs = p;
      const int64_t d_in = h[7], d = h[8];
      f.X = mat(in<char>(), dt, h[9], d_in, h[10]);
      f.R = mat(in<char>(), dt, 0, f.kind == LRM_LINEAR ? d : d_in, h[11]);
      if (f.kind == LRM_LINEAR) {
        f.W = in<char>(); f.bias = in<char>(); f.w_stride = h[12];
        f.d_in = (int32_t)d_in; f.d_out = (int32_t)d;
      } else {
        f.W_gate = in<char>(); f.W_up = in<char>(); f.W_down = in<char>();
        f.H = (int32_t)d_in; f.I = (int32_t)d;
      }
      lrm_forward_outputs o{};
      o.Y = outp<char>(h[13]); o.Yp = outp<char>(h[14]); o.Z = outp<char>(h[15]);
      o.A = outp<char>(h[16]); o.B = outp<char>(h[17]); o.h_sumsq = outp<double>(h[18]);
      const size_t n = lrm_forward_workspace_size(&f);
      ws = ws_of(n);
      status = n ? lrm_expert_forward(&f, &o, ws, n, nullptr) : -1;
    } else {  // pair_grad
      lrm_pair_grad_problem g{};
      g.act = (int32_t)h[6]; g.dtype = (int32_t)dt; g.pairs = p;
      g.dY = mat(in<char>(), dt, h[9], h[8], h[10]);
      g.Z = mat(in<char>(), dt, 1, h[8], h[11]);
      lrm_pair_grad_outputs o{};
      o.dweight = outp<float>(h[13]); o.G = outp<char>(h[14]); o.dbias = outp<float>(h[15]);
      const size_t n = lrm_pair_grad_workspace_size(&g);
      ws = ws_of(n);
      status = n ? lrm_pair_grad(&g, &o, ws, n, nullptr) : -1;
    }
    dev = status == LRM_OK ? (int32_t)lrm_check_device_errors(ws, nullptr) : -1;
  }
  g_out = std::fopen(argv[2], "wb");
  if (!g_out) return 2;
  std::fwrite(&status, 4, 1, g_out);
  std::fwrite(&dev, 4, 1, g_out);
  for (const Out& o : g_outs)
    if (o.n && std::fwrite(o.p, 1, o.n, g_out) != o.n) return 4;
  std::fclose(g_out);
  return 0;
}
