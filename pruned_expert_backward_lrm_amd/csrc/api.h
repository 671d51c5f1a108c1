// Host-side helpers of the C ABI's entry points: argument checks, the
// workspace carver and the early-return macros.
#pragma once

#include <cstddef>
#include <cstdint>

#include "lrm.h"
#include "platform.h"

namespace lrm {

constexpr int kMaxE = 4096;
// GEMM leading dimensions: a 256-row output tile spans less than 1 GiB, so
// its stores take 32-bit offsets
constexpr int kMaxDim = (1 << 20) - 1;
constexpr size_t kAlign = 256;

// Bump allocator over a caller workspace.  With base == nullptr it only
// measures, so size queries and real calls carve identical layouts.
struct Carve {
  char* base;
  size_t off = 0;
  explicit Carve(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(int64_t n) {
    off = (off + kAlign - 1) / kAlign * kAlign;
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += (size_t)(n > 0 ? n : 0) * sizeof(T);
    return p;
  }
  size_t size() const { return (off + kAlign - 1) / kAlign * kAlign; }
};

inline int esize(int dtype) { return dtype == LRM_BF16 ? 2 : 4; }

inline lrm_status check_pairs(const lrm_pairs* p) {
  if (!p) return LRM_ERR_NULL;
  if (p->T < 0 || p->N < 0 || p->E < 1 || p->E > kMaxE) return LRM_ERR_SHAPE;
  if (p->N > 0 && (!p->token || !p->expert || !p->weight)) return LRM_ERR_NULL;
  return LRM_OK;
}

// A dense input: dtype, layout, shape, 16-byte row alignment.
inline lrm_status check_mat(const lrm_mat* m, const lrm_pairs* p, int dtype, int cols, int need_rows) {
  if (!m) return LRM_ERR_NULL;
  if (m->dtype != LRM_F32 && m->dtype != LRM_BF16) return LRM_ERR_DTYPE;
  if (m->dtype != dtype) return LRM_ERR_DTYPE;
  if (m->rows != LRM_ROWS_TOKEN && m->rows != LRM_ROWS_PAIR) return LRM_ERR_LAYOUT;
  if (need_rows >= 0 && m->rows != need_rows) return LRM_ERR_LAYOUT;
  if (m->cols <= 0 || (cols >= 0 && m->cols != cols)) return LRM_ERR_SHAPE;
  if (m->ld < m->cols) return LRM_ERR_SHAPE;
  if (m->cols % (16 / esize(m->dtype)) != 0) return LRM_ERR_UNSUPPORTED;
  const int64_t nrows = m->rows == LRM_ROWS_TOKEN ? p->T : p->N;
  if (nrows > 0 && !m->ptr) return LRM_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(m->ptr) & 15u) != 0) return LRM_ERR_ALIGN;
  if ((m->ld * esize(m->dtype)) % 16 != 0) return LRM_ERR_ALIGN;
  return LRM_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline lrm_status check_quota(const int32_t* q, int E, int64_t* sum) {
  if (!q) return LRM_ERR_NULL;
  int64_t s = 0;
  for (int e = 0; e < E; ++e) {
    if (q[e] < 0) return LRM_ERR_QUOTA;
    s += q[e];
  }
  if (sum) *sum = s;
  return LRM_OK;
}

#define LRM_TRY_HIP(x)                        \
  do {                                        \
    if ((x) != hipSuccess) return LRM_ERR_HIP; \
  } while (0)
#define LRM_TRY(x)                  \
  do {                              \
    lrm_status st_ = (x);           \
    if (st_ != LRM_OK) return st_;  \
  } while (0)

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace lrm
