// Update of the parameters: the gradients' sum of squares, the AdamW step, and
// the values of 8-bit moments.  (What becomes of the weight gradients that the
// LRMoE backward pass makes; the pages leave the optimizer as it is.)
//
// All are bound by memory: one pass over every array, each element read and
// written once, stored past the caches.  The tensors of a list are cut into chunks of
// 2048 elements, 8 neighbours a thread (16 or 32 bytes of every array); a block takes
// its chunks in turn and finds a chunk's tensor in the table, 64 at a time.  Measured (a
// large copy makes 5.1 TB/s): sum of squares of 151 M fp32 gradients 95 us, 6.3 TB/s, of
// 604 M bf16 ones 202 us, 6.0; the step of 151 M bf16 weights with masters and fp32
// moments 794 us, 5.7 TB/s; with 8-bit moments, bf16 weights and gradients 316 us, 4.9,
// its vector instructions (some 560 for 512 elements) taking as long as the memory; the
// values of 151 M codes in bf16 79 us, 5.8 TB/s.
//
// 8-bit moments (see lrm.h): 4 lanes hold a block of 32, whose largest magnitude
// they find with two quad permutations.  The shared exponent x is the largest's,
// one more where its mantissa is above 7/8, so that rounding up never leaves
// the top octave.  A code is the fp32 bits above bit 20, less the exponent of
// the block's lowest octave; 16 random bits below bit 20 (and a half of what is
// below them) are added first, so an element is rounded up with the probability
// of what is cut off.  With nearest rounding v would stand still: a step of beta2
// = 0.999 changes it by 0.1 %, half a step of three mantissa bits is 3 to 6 %.
#include "common.h"
#include "update.h"

namespace lrm {

namespace {

// The table does not change while a kernel runs: read as constant memory, so that
// the loads stay scalar although the kernel stores to memory as well.
#ifdef LRM_CPU_EMU
#define LRM_CONST
#else
#define LRM_CONST __attribute__((address_space(4)))
#endif

// The tensor that holds chunk c: the last one that starts at or before it.  64 of them
// are looked at at a time.  Returns the chunk behind its last one.
__device__ __forceinline__ int64_t tensor_of(const ParamTable& t, int64_t c, ParamEntry* out) {
  int lo = 0, n = t.n;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave, at = lane_id() * step;
    const bool before = at < n && t.chunk0[lo + (at < n ? at : 0)] <= c;
    const int k = (__popcll(__ballot(before)) - 1) * step;  // (the first one is)
    lo += k;
    n = n - k < step ? n - k : step;
  }
  const LRM_CONST ParamEntry* e = (const LRM_CONST ParamEntry*)t.entry + lo;
  *out = ParamEntry{e->p, e->g, e->master, e->m, e->v, e->m_exp, e->v_exp, e->n,
                    e->chunk0, e->block0, e->lr, e->decay, e->vec, 0};
  return e->chunk0 + (e->n + kChunk - 1) / kChunk;
}

// Eight neighbours from element i (those at or past n: 0).
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t i, int64_t n, bool vec, float (&x)[8]) {
  if (vec && i + 8 <= n) {
    if constexpr (BF16) {
      const u32x4 q = *reinterpret_cast<const u32x4*>((const uint16_t*)base + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(q[j]);
        x[2 * j + 1] = bf16_hi(q[j]);
      }
    } else {
      const f32x4 q = *reinterpret_cast<const f32x4*>((const float*)base + i);
      const f32x4 r = *reinterpret_cast<const f32x4*>((const float*)base + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = q[j];
        x[4 + j] = r[j];
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = 0.f;
    if (i + j < n)
      x[j] = BF16 ? bf16_to_f32(((const uint16_t*)base)[i + j]) : ((const float*)base)[i + j];
  }
}
// Past the caches: the arrays are larger, and lines left to be written back slow the
// kernel that comes next (the sum of squares after the moments were read: 114 us, 76 so).
template <typename V>
__device__ __forceinline__ void store_stream(void* p, V v) {
#ifdef LRM_CPU_EMU
  *reinterpret_cast<V*>(p) = v;
#else
  __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
#endif
}
__device__ __forceinline__ void store8(float* base, int64_t i, int64_t n, bool vec, const float (&x)[8]) {
  if (vec && i + 8 <= n) {
    store_stream(base + i, f32x4{x[0], x[1], x[2], x[3]});
    store_stream(base + i + 4, f32x4{x[4], x[5], x[6], x[7]});
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) base[i + j] = x[j];
}
// bf16 bits in the upper halves of x
__device__ __forceinline__ void store8_hi(uint16_t* base, int64_t i, int64_t n, bool vec,
                                          const uint32_t (&x)[8]) {
  if (vec && i + 8 <= n) {
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = (x[2 * j] >> 16) | (x[2 * j + 1] & 0xffff0000u);
    store_stream(base + i, q);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) base[i + j] = (uint16_t)(x[j] >> 16);
}

// Eight codes, four a word.
__device__ __forceinline__ u32x2 load_codes(const uint8_t* base, int64_t i, int64_t n, bool vec) {
  if (vec && i + 8 <= n) return *reinterpret_cast<const u32x2*>(base + i);
  u32x2 q = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) q[j >> 2] |= (uint32_t)base[i + j] << (8 * (j & 3));
  return q;
}
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, int64_t n, bool vec, u32x2 q) {
  if (vec && i + 8 <= n) {
    store_stream(base + i, q);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (i + j < n) base[i + j] = (uint8_t)(q[j >> 2] >> (8 * (j & 3)));
}

// Octaves below the shared exponent's: 15 (m) or 31 (v).
constexpr int kTopM = 15, kTopV = 31;

// Codes are handled two at a time in 16-bit halves: elements 0 and 2, and 1 and 3,
// of a word (a float's upper half holds sign, exponent and 7 bits of mantissa).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t s16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 halves(uint32_t w) { return __builtin_bit_cast(u16x2, w); }
__device__ __forceinline__ uint32_t word_of(u16x2 v) { return __builtin_bit_cast(uint32_t, v); }
// The upper halves of lo and hi.
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// 1 in the halves of v that are above 0 (v is not below 0), by a minimum with ones that
// the compiler cannot see: it would compare and select every half instead.
template <typename V>
__device__ __forceinline__ V one_if(V v) {
  uint32_t ones = 0x10001u;
#ifndef LRM_CPU_EMU
  asm("" : "+s"(ones));
#endif
  return __builtin_elementwise_min(v, __builtin_bit_cast(V, ones));
}

// The upper words of eight codes' values: of floats, or (F64) of doubles, whose lower
// words are 0.
template <bool SECOND, bool F64>
__device__ __forceinline__ void decode8(u32x2 q, uint32_t e, uint32_t (&x)[8]) {
  constexpr int shift = F64 ? 1 : 4;  // of the mantissa's 3 bits in the upper half
  const uint32_t low = (e - (SECOND ? kTopV : kTopM) + (F64 ? 1023 - 127 : 0)) << (shift + 3);
  const u16x2 base = halves((low & 0xffffu) * 0x10001u);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint32_t b = (p & 1 ? q[p >> 1] >> 8 : q[p >> 1]) & 0x00ff00ffu;
    const u16x2 c = halves(SECOND ? b : b & 0x007f007fu);
    uint32_t t = word_of((c * (uint16_t)(1 << shift) + base) * one_if(c));  // (code 0 stands for 0)
    if (!SECOND) t |= (b << 8) & 0x80008000u;
    x[4 * (p >> 1) + (p & 1)] = t << 16;
    x[4 * (p >> 1) + (p & 1) + 2] = t & 0xffff0000u;
  }
}
__device__ __forceinline__ double upper_word(uint32_t hi) {
  return __builtin_bit_cast(double, (uint64_t)hi << 32);
}

// The bits of x in fp32, rounded towards 0 (beyond its range: the largest numbers; below
// 2^-126: what is left of the mantissa).  A sum with the random bits then
// crosses a border exactly where x itself does.
template <bool SIGNED>
__device__ __forceinline__ uint32_t f32_bits_down(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t hi = (uint32_t)(b >> 32);
  int u = (int)(SIGNED ? hi & 0x7fffffffu : hi) - (896 << 20);
  u = u < 0 ? 0 : (u > (255 << 20) - 1 ? (255 << 20) - 1 : u);
  const uint32_t t = (uint32_t)u << 3 | (uint32_t)b >> 29;
  return SIGNED ? (hi & 0x80000000u) | t : t;
}

// The exponent that a block's four lanes share, from the bits of their largest
// magnitudes.
__device__ __forceinline__ uint32_t quad_max(uint32_t u) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xB1, 0xf, 0xf, false);
  u = o > u ? o : u;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4E, 0xf, 0xf, false);
  return o > u ? o : u;
}
template <bool SECOND>
__device__ __forceinline__ uint32_t block_exponent(const uint32_t (&x)[8]) {
  constexpr uint32_t least = (SECOND ? kTopV : kTopM) + 1;
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t mag = SECOND ? x[j] : x[j] & 0x7fffffffu;
    top = mag > top ? mag : top;
  }
  const uint32_t e = (quad_max(top) + 0xfffffu) >> 23;
  return e > least ? e : least;
}
// x: bits of floats; r: 16 random bits an element at bit SECOND ? 16 : 0 of each.
template <bool SECOND>
__device__ __forceinline__ u32x2 encode8(const uint32_t (&x)[8], uint32_t e, const uint32_t (&r)[8]) {
  constexpr int top = SECOND ? kTopV : kTopM, most = 8 * top + 7;
  const uint32_t low = (e - top) << 23;
  uint32_t t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t mag = SECOND ? x[j] : x[j] & 0x7fffffffu;
    const uint32_t add = SECOND ? (r[j] >> 12 & 0xffff0u) | 8u : ((r[j] & 0xffffu) << 4) | 8u;
    t[j] = mag + add - low;
  }
  u32x2 q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t c[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int j = 4 * w + p;
      s16x2 v = __builtin_bit_cast(s16x2, upper_halves(t[j], t[j + 2])) >> (int16_t)4;
      if (SECOND) {  // (what is not 0 stays so)
        const uint32_t a = x[j], b = x[j + 2];
        const uint32_t some = (a < 1u ? a : 1u) | (b < 1u ? b : 1u) << 16;
        v = __builtin_elementwise_max(v, __builtin_bit_cast(s16x2, some));
      } else {
        v = __builtin_elementwise_max(v, (s16x2)0);
      }
      v = __builtin_elementwise_min(v, (s16x2)(int16_t)most);
      if (!SECOND) {
        const uint32_t sign = upper_halves(x[j], x[j + 2]) >> 8 & 0x00800080u;
        v += one_if(v) * __builtin_bit_cast(s16x2, sign);
      }
      c[p] = __builtin_bit_cast(uint32_t, v);
    }
    q[w] = c[0] | c[1] << 8;
  }
  return q;
}

// ------------------------------------------------------------------ table
__global__ __launch_bounds__(64) void k_params_table(TableBatch b, int first, int count, int n,
                                                     int64_t chunks, ParamEntry* entry,
                                                     int64_t* chunk0) {
  const int i = threadIdx.x;
  if (i < count) {
    entry[first + i] = b.entry[i];
    chunk0[first + i] = b.entry[i].chunk0;
  }
  if (i == 0 && first + count == n) chunk0[n] = chunks;
}

// --------------------------------------------------------- sum of squares
// Squares and sums in fp64: nothing overflows, and what is not finite shows.
template <bool BF16>
__global__ __launch_bounds__(256) void k_grad_sumsq(ParamTable t, double* part) {
  __shared__ double lds[4];
  const int64_t chunks = t.chunk0[t.n];
  double sum = 0.0;
  ParamEntry e;
  int64_t end = 0;  // of e's chunks
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    if (c >= end) end = tensor_of(t, c, &e);
    float x[8];
    load8<BF16>(e.g, (c - e.chunk0) * kChunk + threadIdx.x * 8, e.n, e.vec != 0, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fma((double)x[j], (double)x[j], sum);
  }
  sum = wave_sum(sum);
  if (lane_id() == 0) lds[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(256) void k_sumsq_join(int n, const double* part, double* sumsq) {
  __shared__ double lds[4];
  double v[kSumBlocks / 256];
#pragma unroll
  for (int q = 0; q < kSumBlocks / 256; ++q) {
    const int i = q * 256 + threadIdx.x;
    v[q] = i < n ? part[i] : 0.0;
  }
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < kSumBlocks / 256; ++q) sum += v[q];
  sum = wave_sum(sum);
  if (lane_id() == 0) lds[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) sumsq[0] = (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// ------------------------------------------------------------------ AdamW
__device__ __forceinline__ double total_of(const double* sumsq, int n) {
  const LRM_CONST double* x = (const LRM_CONST double*)sumsq;
  double s = 0.0;
  for (int i = 0; i < n; ++i) s += x[i];
  return s;
}
__device__ __forceinline__ bool finite64(double x) { return x - x == 0.0; }

template <int P, bool GB, bool EIGHT>
__global__ __launch_bounds__(256) void k_adamw(ParamTable t, AdamArgs a) {
  // (Every block starts with this: uniform loads are scalar, and what becomes a
  // factor in fp32 is formed with few fp64 instructions.)
  double f = a.grad_scale;
  if (a.sumsq) {
    const double sum = total_of(a.sumsq, a.n_sumsq);
    if (!finite64(sum)) return;
    // max_norm / norm: 1 / sqrt(sum) from the hardware's estimate (2^-24) and a Newton step
    const double r = __builtin_amdgcn_rsq(sum);
    const double over = a.over * fma(r, fma(-0.5 * sum * r, r, 0.5), r);
    if (sum > 0.0 && over < 1.0) f *= over;  // (over: infinite without clipping)
  }
  float bias = a.bias, root = a.root;
  uint32_t key = a.key;
  if (a.steps) {
    const int64_t step = *(const LRM_CONST int64_t*)a.steps + 1;
    bias = -1.f / expm1f((float)((double)step * a.ln1));
    root = 1.f / __builtin_amdgcn_sqrtf(-expm1f((float)((double)step * a.ln2)));
    key = step_key(a.seed, (uint64_t)step);
  }
  const float lr = a.lr_dev ? *(const LRM_CONST float*)a.lr_dev : a.lr;
  const float size = lr * bias;
  const double f1 = (1.0 - a.beta1) * f, f2 = (1.0 - a.beta2) * f * f;
  const float c = (float)f, b1 = a.b1, d1 = a.d1, b2 = a.b2, d2 = a.d2, eps = a.eps;
  constexpr bool RANDOM_P = P == 1;
  const int64_t chunks = t.chunk0[t.n];
  ParamEntry e;
  int64_t end = 0;  // of e's chunks
  for (int64_t ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    if (ch >= end) end = tensor_of(t, ch, &e);
    const int64_t i = (ch - e.chunk0) * kChunk + threadIdx.x * 8, n = e.n;
    const bool vec = e.vec != 0;
    const float up = size * e.lr, down = lr * e.lr * e.decay;
    float g[8], w[8], m[8], v[8];
    const int64_t blk = i >> 5, blkc = i < n ? blk : 0;
    load8<GB>(e.g, i, n, vec, g);
    load8<P == 1>(P == 2 ? (const void*)e.master : e.p, i, n, vec, w);
    uint32_t um[8], uv[8];  // 8 bits: words of the moments
    if constexpr (EIGHT) {
      const u32x2 qm = load_codes((const uint8_t*)e.m, i, n, vec);
      const u32x2 qv = load_codes((const uint8_t*)e.v, i, n, vec);
      decode8<false, true>(qm, e.m_exp[blkc], um);
      decode8<true, true>(qv, e.v_exp[blkc], uv);
    } else {
      load8<false>(e.m, i, n, vec, m);
      load8<false>(e.v, i, n, vec, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (EIGHT) {
        // in fp64 (as many instructions as in fp32): the codes are the definition's
        const double x = (double)g[j];
        um[j] = f32_bits_down<true>(fma(a.beta1, upper_word(um[j]), f1 * x));
        uv[j] = f32_bits_down<false>(fma(a.beta2, upper_word(uv[j]), f2 * (x * x)));
        m[j] = __uint_as_float(um[j]);
        v[j] = __uint_as_float(uv[j]);
      } else {
        const float x = c * g[j];
        m[j] = fmaf(b1, m[j], d1 * x);
        v[j] = fmaf(b2, v[j], d2 * (x * x));
      }
      const float den = fmaf(__builtin_amdgcn_sqrtf(v[j]), root, eps);
      w[j] = fmaf(-up, m[j] * __builtin_amdgcn_rcpf(den), fmaf(-down, w[j], w[j]));
    }
    uint32_t r[8];
    if constexpr (EIGHT || RANDOM_P) {
      const uint64_t b = (uint64_t)(e.block0 + blk);
      const uint32_t kb = mix32(key + (uint32_t)b * kGold + (uint32_t)(b >> 32) * kRoot3) +
                          (uint32_t)(i & 31) * kGold;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = kb + (uint32_t)j * kGold;
        r[j] ^= r[j] >> 16;
        r[j] *= kRoot2;
        r[j] ^= r[j] >> 15;
      }
    }
    if constexpr (EIGHT) {
      const uint32_t em = block_exponent<false>(um), ev = block_exponent<true>(uv);
      if (i < n) {
        store_codes((uint8_t*)e.m, i, n, vec, encode8<false>(um, em, r));
        store_codes((uint8_t*)e.v, i, n, vec, encode8<true>(uv, ev, r));
        if ((i & 31) == 0) {
          e.m_exp[blk] = (uint8_t)em;
          e.v_exp[blk] = (uint8_t)ev;
        }
      }
    } else {
      store8((float*)e.m, i, n, vec, m);
      store8((float*)e.v, i, n, vec, v);
    }
    if constexpr (P != 1) store8(P == 2 ? e.master : (float*)e.p, i, n, vec, w);
    if constexpr (P != 0) {
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = __float_as_uint(w[j]);
        if constexpr (RANDOM_P) {
          const uint32_t q = r[j] * kRoot3;
          u[j] += (q ^ (q >> 16)) & 0xffffu;
        } else if (j & 1) {
          const uint32_t two = cvt_pk_bf16(w[j - 1], w[j]);
          u[j - 1] = two << 16;
          u[j] = two;
        }
      }
      store8_hi((uint16_t*)e.p, i, n, vec, u);
    }
  }
}

// After the step: one more is made, if it was.
__global__ __launch_bounds__(64) void k_count_step(AdamArgs a, int64_t* steps) {
  if (threadIdx.x != 0) return;
  if (a.sumsq && !finite64(total_of(a.sumsq, a.n_sumsq))) return;
  steps[0] += 1;
}

// ---------------------------------------------------------------- reading
template <bool SECOND, bool BF16>
__global__ __launch_bounds__(256) void k_moment_read(int64_t n, const uint8_t* codes, const uint8_t* exps,
                                                     bool vec, void* out) {
  const int64_t step = (int64_t)gridDim.x * 2048;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += step) {
    uint32_t u[8];
    decode8<SECOND, false>(load_codes(codes, i, n, vec), exps[i >> 5], u);
    if constexpr (BF16) {
      store8_hi((uint16_t*)out, i, n, vec, u);
    } else {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(u[j]);
      store8((float*)out, i, n, vec, x);
    }
  }
}

template <int P, bool GB>
void adamw_launch(const ParamTable& t, int grid, int eight, const AdamArgs& a, hipStream_t s) {
  if (eight)
    LRM_LAUNCH(grid, 256, 0, s, k_adamw<P, GB, true>)(t, a);
  else
    LRM_LAUNCH(grid, 256, 0, s, k_adamw<P, GB, false>)(t, a);
}

int grid_of(int64_t chunks, int most) { return (int)(chunks < most ? chunks : most); }

}  // namespace

hipError_t launch_params_table(const TableBatch& b, int first, int count, int n, int64_t chunks,
                               void* table, hipStream_t s) {
  ParamEntry* entry = static_cast<ParamEntry*>(table);
  LRM_LAUNCH(1, 64, 0, s, k_params_table)(b, first, count, n, chunks, entry,
                                          reinterpret_cast<int64_t*>(entry + n));
  return hipGetLastError();
}

hipError_t launch_grad_sumsq(const ParamTable& t, int64_t chunks, int g_bf16, double* part,
                             double* sumsq, hipStream_t s) {
  const int grid = grid_of(chunks, g_bf16 ? kSumBlocks : kSumBlocks / 2);
  if (grid > 0) {
    if (g_bf16)
      LRM_LAUNCH(grid, 256, 0, s, k_grad_sumsq<true>)(t, part);
    else
      LRM_LAUNCH(grid, 256, 0, s, k_grad_sumsq<false>)(t, part);
  }
  LRM_LAUNCH(1, 256, 0, s, k_sumsq_join)(grid, part, sumsq);
  return hipGetLastError();
}

hipError_t launch_adamw(const ParamTable& t, int64_t chunks, int p, int g_bf16, int eight,
                        const AdamArgs& a, int64_t* steps, hipStream_t s) {
  // Blocks that end after one chunk stream best (151 M bf16 weights with masters and the
  // norm: 945 us, 997 with 16384 blocks, 1046 with 4096).  With 8-bit moments the start of a
  // block weighs more, once there are many: one, two, four and eight chunks a block take
  // 1584, 1509, 1541 and 1590 us with fp32 gradients, 1631, 1419, 1359 and 1322 with bf16
  // ones (604 M bf16 weights, whose step counts itself); 19 M fp32 weights, 9400
  // chunks, 93, 97, 100 and 102 with the norm.
  const int64_t per = eight && chunks > 16384 ? (g_bf16 ? 8 : 2) : 1;
  const int64_t fewer = (chunks + per - 1) / per;
  const int grid = grid_of(per > 1 && fewer < 16384 ? 16384 : fewer, 1 << 20);
  if (grid > 0) {
    if (p == 0 && !g_bf16) adamw_launch<0, false>(t, grid, eight, a, s);
    else if (p == 0) adamw_launch<0, true>(t, grid, eight, a, s);
    else if (p == 1 && !g_bf16) adamw_launch<1, false>(t, grid, eight, a, s);
    else if (p == 1) adamw_launch<1, true>(t, grid, eight, a, s);
    else if (!g_bf16) adamw_launch<2, false>(t, grid, eight, a, s);
    else adamw_launch<2, true>(t, grid, eight, a, s);
  }
  if (steps) LRM_LAUNCH(1, 64, 0, s, k_count_step)(a, steps);
  return hipGetLastError();
}

hipError_t launch_moment_read(int64_t n, int second, const uint8_t* codes, const uint8_t* exps,
                              int bf16, void* out, hipStream_t s) {
  if (n <= 0) return hipSuccess;
  const bool vec = (reinterpret_cast<uintptr_t>(codes) & 7u) == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
  const int64_t blocks = (n + 2047) / 2048;
  const int grid = grid_of(blocks, 1 << 14);
  if (second && bf16)
    LRM_LAUNCH(grid, 256, 0, s, k_moment_read<true, true>)(n, codes, exps, vec, out);
  else if (second)
    LRM_LAUNCH(grid, 256, 0, s, k_moment_read<true, false>)(n, codes, exps, vec, out);
  else if (bf16)
    LRM_LAUNCH(grid, 256, 0, s, k_moment_read<false, true>)(n, codes, exps, vec, out);
  else
    LRM_LAUNCH(grid, 256, 0, s, k_moment_read<false, false>)(n, codes, exps, vec, out);
  return hipGetLastError();
}

}  // namespace lrm
