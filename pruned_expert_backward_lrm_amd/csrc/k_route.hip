// Routing to experts: scores, group limit, top-k choice and weights, the
// gradient of the weights with respect to the logits, and the pairs of one
// GPU's experts.  (The pairs are the input of the LRMoE pass: page 1,
// introduction, "pair"; the pages take the router as given.)
//
// A token is handled by LPT lanes (16, 32 or 64 of a wave, so 4, 2 or 1 tokens
// per wave), each holding the NV experts i*NV .. i*NV + NV - 1 of its lane i:
// lower lanes hold lower experts, so a tie between lanes goes to the lowest.
// Keys are kept as unsigned integers that order like the floats (0: not
// eligible); a round of the choice takes the maximum over the lanes with DPP
// row rotations, then the minimum expert among the lanes that hold it.
//
// Order of the choice: without a bias the scores order like the logits, which
// are exact.  With a bias, and for sums of two scores, the keys are first
// formed in fp32; their error is below kKeyTol (1 + |key|/8), so a token whose
// neighbouring keys are further apart than that is decided.  The others (a few
// per mille) are chosen again from keys formed in fp64.
#include "common.h"
#include "launch.h"

namespace lrm {

namespace {

constexpr int kRouteThreads = 256;

// ---------------------------------------------------------- ordered keys
__device__ __forceinline__ uint32_t ord_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ord_of(double d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, d);
  return u ^ ((u >> 63) ? ~0ull : (1ull << 63));
}
__device__ __forceinline__ float unord(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ double unord(uint64_t k) {
  return __builtin_bit_cast(double, k ^ ((k >> 63) ? (1ull << 63) : ~0ull));
}

template <typename F>
struct KeyOf;
template <>
struct KeyOf<float> { typedef uint32_t type; };
template <>
struct KeyOf<double> { typedef uint64_t type; };

// Largest error of an fp32 key (score + bias, or a sum of two), with room:
// scores are in [0, 1] and good to about 1e-6, a sum is rounded at 2^-24 of
// its size.
constexpr float kKeyTol = 4e-6f;
__device__ __forceinline__ bool too_close(float hi, float lo) {
  return !(hi - lo > kKeyTol * (1.f + 0.125f * fabsf(hi)));
}
__device__ __forceinline__ bool too_close(double, double) { return false; }

// ------------------------------------------------ reductions over LPT lanes
template <int ROT>
__device__ __forceinline__ uint32_t ror32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROT, 0xf, 0xf, false);
}
template <int ROT>
__device__ __forceinline__ uint64_t ror64(uint64_t v) {
  return ((uint64_t)ror32<ROT>((uint32_t)(v >> 32)) << 32) | ror32<ROT>((uint32_t)v);
}
template <int ROT>
__device__ __forceinline__ uint32_t ror(uint32_t v) { return ror32<ROT>(v); }
template <int ROT>
__device__ __forceinline__ uint64_t ror(uint64_t v) { return ror64<ROT>(v); }
template <int ROT>
__device__ __forceinline__ int ror(int v) { return (int)ror32<ROT>((uint32_t)v); }
template <int ROT>
__device__ __forceinline__ float ror(float v) {
  return __uint_as_float(ror32<ROT>(__float_as_uint(v)));
}
template <int ROT>
__device__ __forceinline__ double ror(double v) {
  return __builtin_bit_cast(double, ror64<ROT>(__builtin_bit_cast(uint64_t, v)));
}

// All lanes of the LPT-lane group get op over the group (op commutative; the
// pairs of every step are the same two values in both lanes, so all lanes
// hold the same bits).
template <int LPT, typename V, typename Op>
__device__ __forceinline__ V group_all(V v, Op op) {
  v = op(v, ror<8>(v));
  v = op(v, ror<4>(v));
  v = op(v, ror<2>(v));
  v = op(v, ror<1>(v));
  if constexpr (LPT >= 32) v = op(v, __shfl_xor(v, 16, kWave));
  if constexpr (LPT >= 64) v = op(v, __shfl_xor(v, 32, kWave));
  return v;
}
struct OpMax {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct OpMin {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a < b ? a : b; }
};
struct OpAdd {
  template <typename V>
  __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};

// ------------------------------------------------------------ row loads
// NV values from column c0 of a logits row (columns at or past E: -inf).
// vec: the row starts on a 16-byte boundary.
template <int NV>
__device__ __forceinline__ void load_row(const void* row, int bf16, bool vec, int c0, int E,
                                         float (&z)[NV]) {
  if (NV % 8 == 0 && vec && c0 + NV <= E) {
    if (bf16) {
      const u32x4* src = reinterpret_cast<const u32x4*>((const uint16_t*)row + c0);
#pragma unroll
      for (int q = 0; q < NV / 8; ++q) {
        const u32x4 v = src[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[q * 8 + 2 * j] = bf16_lo(v[j]);
          z[q * 8 + 2 * j + 1] = bf16_hi(v[j]);
        }
      }
    } else {
      const f32x4* src = reinterpret_cast<const f32x4*>((const float*)row + c0);
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        const f32x4 v = src[q];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[q * 4 + j] = v[j];
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    z[j] = -__builtin_inff();
    if (c0 + j < E)
      z[j] = bf16 ? bf16_to_f32(((const uint16_t*)row)[c0 + j]) : ((const float*)row)[c0 + j];
  }
}

__device__ __forceinline__ float load_one(const void* row, int bf16, int c) {
  return bf16 ? bf16_to_f32(((const uint16_t*)row)[c]) : ((const float*)row)[c];
}

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

// A bit per expert of the lane that takes part (NV <= 64).  Bits and selects,
// not branches around single values: hipcc 7.2 drops the assignment of a
// value under a nested branch here.
template <int NV>
__device__ __forceinline__ uint64_t expert_bits(const RouteArgs& a, int c0) {
  uint64_t bits = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + j < a.E ? c0 + j : 0;
    const uint32_t m = a.expert_mask ? a.expert_mask[c] : 1u;
    bits |= (uint64_t)(m != 0 && c0 + j < a.E ? 1u : 0u) << j;
  }
  return bits;
}
// The eligible logits of one lane: masked places become -inf.
template <int NV>
__device__ __forceinline__ void mask_row(uint64_t bits, float (&z)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) z[j] = (bits >> j) & 1 ? z[j] : -__builtin_inff();
}

// k rounds of choice over NV keys per lane; lane j of the group ends with the
// j-th choice in *got (-1: none left).  Returns whether two neighbours in the
// order (the first one left out among them) are too close to tell.
template <int LPT, int NV, typename F>
__device__ __forceinline__ bool choose(typename KeyOf<F>::type (&key)[NV], int i, int k, bool check,
                                       int* got) {
  typedef typename KeyOf<F>::type K;
  bool close = false;
  K prev = 0;
  *got = -1;
  const int rounds = check ? k + 1 : k;
  for (int r = 0; r < rounds; ++r) {
    K best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const K top = group_all<LPT>(best, OpMax());
    const int mine = best == top ? i * NV + at : 0x7fffffff;
    const int win = group_all<LPT>(mine, OpMin());
    if (check && r > 0 && top != 0 && too_close(unord(prev), unord(top))) close = true;
    if (i == r && r < k) *got = top != 0 ? win : -1;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (i * NV + j == win) key[j] = 0;
    prev = top;
  }
  return close;
}

// The groups that stay: a bit per group, from the values val (F; -inf where
// not eligible) of a token's experts, through its row of LDS.
template <int LPT, int NV, typename F>
__device__ __forceinline__ uint64_t keep_groups(const RouteArgs& a, const F (&val)[NV], int i, F* row,
                                                bool check, bool* close) {
  typedef typename KeyOf<F>::type K;
  constexpr int NG = 64 / LPT;  // groups per lane
  const F inf = (F)__builtin_inff();
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (i * NV + j < a.E) row[i * NV + j] = val[j];
  wave_sync();
  const int per = a.E / a.n_group;
  K key[NG];
#pragma unroll
  for (int v = 0; v < NG; ++v) {
    const int g = i * NG + v;
    key[v] = 0;
    if (g >= a.n_group) continue;
    F one = -inf, two = -inf;
    int c = g % per;  // the lanes start at different columns (and LDS banks)
    for (int s = 0; s < per; ++s) {
      const F x = row[g * per + c];
      if (x > one) {
        two = one;
        one = x;
      } else if (x > two) {
        two = x;
      }
      c = c + 1 == per ? 0 : c + 1;
    }
    if (one > -inf) {
      const F sc = a.group_top2 && two > -inf ? one + two : one;
      key[v] = ord_of(sc);
    }
  }
  wave_sync();
  // rounds of choice, as for the experts (one bit per winner)
  uint64_t kept = 0;
  K prev = 0;
  const int rounds = check ? a.topk_group + 1 : a.topk_group;
  for (int r = 0; r < rounds; ++r) {
    K best = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < NG; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const K top = group_all<LPT>(best, OpMax());
    const int mine = best == top ? i * NG + at : 0x7fffffff;
    const int win = group_all<LPT>(mine, OpMin());
    if (check && r > 0 && top != 0 && too_close(unord(prev), unord(top))) *close = true;
    if (r < a.topk_group && top != 0) kept |= 1ull << win;
#pragma unroll
    for (int v = 0; v < NG; ++v)
      if (i * NG + v == win) key[v] = 0;
    prev = top;
  }
  return kept;
}

// Scores of one lane's experts in F: softmax (less its denominator when raw)
// or sigmoid; top: the largest eligible logit of the row (-inf: none).
template <int LPT, int NV, typename F>
__device__ __forceinline__ void scores(const RouteArgs& a, const float (&z)[NV], float top, bool raw,
                                       F (&s)[NV]) {
  if (a.softmax) {
    const F m = top > -__builtin_inff() ? (F)top : (F)0;
    F sum = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s[j] = exp_of((F)z[j] - m);
      sum += s[j];
    }
    if (raw) return;
    sum = group_all<LPT>(sum, OpAdd());
    const F inv = sum > (F)0 ? (F)1 / sum : (F)0;
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] = (F)1 / ((F)1 + exp_of(-(F)z[j]));
  }
}

// The choice of one token with keys in F.  exact: the keys' order is certain.
template <int LPT, int NV, typename F>
__device__ __forceinline__ bool choose_token(const RouteArgs& a, const float (&z)[NV], float top, int i,
                                             F* row, int* got) {
  typedef typename KeyOf<F>::type K;
  const F inf = (F)__builtin_inff();
  const bool by_score = a.bias != nullptr;
  const bool two = a.n_group > 1 && a.group_top2;
  F s[NV];
  bool close = false;
  if (by_score || two) {
    scores<LPT, NV, F>(a, z, top, !by_score, s);
    if (by_score) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (i * NV + j < a.E) s[j] += (F)a.bias[i * NV + j];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (!(z[j] > -__builtin_inff()) && z[j] == z[j]) s[j] = -inf;
  }
  uint64_t kept = ~0ull;
  if (a.n_group > 1) {
    if (by_score || two) {
      kept = keep_groups<LPT, NV, F>(a, s, i, row, true, &close);
    } else {
      F zf[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) zf[j] = (F)z[j];
      kept = keep_groups<LPT, NV, F>(a, zf, i, row, false, &close);
    }
  }
  K key[NV];
  const int per = a.E / a.n_group;
  int g = i * NV / per, c = i * NV - g * per;  // group and place of the lane's first expert
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const F v = by_score ? s[j] : (F)z[j];
    const bool on = i * NV + j < a.E && v != -inf && ((kept >> (g & 63)) & 1);
    key[j] = on ? ord_of(v) : (K)0;
    if (++c == per) {
      c = 0;
      ++g;
    }
  }
  close |= choose<LPT, NV, F>(key, i, a.k, by_score, got);
  return close;
}

// Threads per block: one wave where the rows are long (their fp64 keys are
// staged in LDS for the groups).
template <int NV>
constexpr int route_threads() { return NV > 8 ? kWave : kRouteThreads; }

template <int LPT, int NV>
__global__ __launch_bounds__(route_threads<NV>()) void k_route(RouteArgs a) {
  LRM_DYN_SHARED(double, dyn);  // [tokens of a block][E] rows (groups), then int hist[E] (counts)
  constexpr int NT = route_threads<NV>(), tpb = NT / LPT;
  const int i = threadIdx.x & (LPT - 1);
  const int sub = threadIdx.x / LPT;
  const uint64_t bits = expert_bits<NV>(a, i * NV);
  double* row64 = a.n_group > 1 ? dyn + (int64_t)sub * a.E : nullptr;
  int* hist = reinterpret_cast<int*>(dyn + (a.n_group > 1 ? (int64_t)tpb * a.E : 0));
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += NT) hist[e] = 0;
    __syncthreads();
  }
  const int nrow = (a.T - 1) / tpb + 1;
  for (int rb = blockIdx.x; rb < nrow; rb += gridDim.x) {
    const int64_t t = (int64_t)rb * tpb + sub;
    const bool in = t < a.T;
    const char* lrow = (const char*)a.logits + (in ? t : 0) * a.ld * (a.bf16 ? 2 : 4);
    const bool on = in && (a.token_mask ? a.token_mask[in ? t : 0] != 0 : true);
    float z[NV];
    load_row<NV>(lrow, a.bf16, a.vec != 0, i * NV, a.E, z);
    mask_row<NV>(on ? bits : 0, z);
    float top = -__builtin_inff();
    if (a.softmax && (!a.renorm || a.bias || a.n_group > 1)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) top = z[j] > top ? z[j] : top;
      top = group_all<LPT>(top, OpMax());
    }
    int e;
    const bool close = choose_token<LPT, NV, float>(a, z, top, i, (float*)row64, &e);
    if (__ballot(close)) {  // the whole wave again, in fp64
      int e2;
      choose_token<LPT, NV, double>(a, z, top, i, row64, &e2);
      e = e2;
    }
    // weights: lane j holds choice j
    const bool has = i < a.k && e >= 0 && e < a.E;
    const float ze = has ? load_one(lrow, a.bf16, e) : -__builtin_inff();
    float w = 0.f;
    if (a.renorm) {
      // softmax: exp(z - m) with m the largest chosen logit.  sigmoid: both
      // numerator and sum times e^-m, m = min(largest chosen logit, 0), so
      // that the sum cannot underflow.
      float m = group_all<LPT>(ze, OpMax());
      if (!a.softmax) m = m < 0.f ? m : 0.f;
      float f = 0.f;
      if (has) {
        if (a.softmax)
          f = expf(ze - m);
        else
          f = ze <= 0.f ? expf(ze - m) / (1.f + expf(ze)) : 1.f / (1.f + expf(-ze));
      }
      const float sum = group_all<LPT>(f, OpAdd());
      w = has ? a.scale * (f / sum) : 0.f;
    } else if (a.softmax) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) sum += top > -__builtin_inff() ? expf(z[j] - top) : 0.f;
      sum = group_all<LPT>(sum, OpAdd());
      w = has ? a.scale * (expf(ze - top) / sum) : 0.f;
    } else {
      w = has ? a.scale * (1.f / (1.f + expf(-ze))) : 0.f;
    }
    if (in && i < a.k) {
      const int64_t at = t * a.k + i;
      a.expert[at] = has ? e : -1;
      a.weight[at] = w;
      if (a.token) a.token[at] = (int32_t)t;
      if (a.counts && has) atomicAdd(&hist[e], 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += NT) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
}

// counts[e] = sum over the blocks of part[b][e]
__global__ __launch_bounds__(256) void k_route_counts(int nblk, int E, const int32_t* part,
                                                      int32_t* counts) {
  __shared__ int lds[256];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  int s = 0;
  if (e < E)
    for (int b = r; b < nblk; b += 8) s += part[(int64_t)b * E + e];
  lds[threadIdx.x] = s;
  __syncthreads();
  if (r == 0 && e < E) {
#pragma unroll
    for (int q = 1; q < 8; ++q) s += lds[q * 32 + c];
    counts[e] = s;
  }
}

// ------------------------------------------------------------- backward
template <int LPT, int NV>
__global__ __launch_bounds__(kRouteThreads) void k_route_bwd(RouteArgs a, const int32_t* expert,
                                                             const float* dweight, void* dlogits,
                                                             int64_t ldd, int vec_out) {
  struct Slot {
    int e;
    float d;
  };
  __shared__ Slot slots[kRouteThreads];  // one per lane: lane j of a token, choice j
  const int i = threadIdx.x & (LPT - 1);
  const int base = threadIdx.x & ~(LPT - 1);
  constexpr int tpb = kRouteThreads / LPT;
  const int nrow = (a.T - 1) / tpb + 1;
  const bool dense = a.softmax && !a.renorm;
  const uint64_t bits = dense ? expert_bits<NV>(a, i * NV) : 0;
  for (int rb = blockIdx.x; rb < nrow; rb += gridDim.x) {
    const int64_t t = (int64_t)rb * tpb + threadIdx.x / LPT;
    const bool in = t < a.T;
    const char* lrow = (const char*)a.logits + (in ? t : 0) * a.ld * (a.bf16 ? 2 : 4);
    const bool on = in && (a.token_mask ? a.token_mask[in ? t : 0] != 0 : true);
    const int64_t slot = on && i < a.k ? t * a.k + i : 0;
    const int e0 = expert[slot];
    const bool named = on && i < a.k && e0 >= 0 && e0 < a.E;
    const int ec = named ? e0 : 0;
    const bool open = a.expert_mask ? a.expert_mask[ec] != 0 : true;
    const float zc = load_one(lrow, a.bf16, ec);
    const float dv = dweight[slot];
    const bool has = named && open && zc != -__builtin_inff();
    const int e = has ? e0 : -1;
    const float ze = has ? zc : -__builtin_inff();
    const float v = has ? a.scale * dv : 0.f;
    float p[NV], d = 0.f, dot = 0.f;
    if (a.renorm) {
      float m = group_all<LPT>(ze, OpMax());
      if (!a.softmax) m = m < 0.f ? m : 0.f;
      float f = 0.f, q = 1.f;
      if (has) {
        if (a.softmax) {
          f = expf(ze - m);
        } else {
          q = 1.f / (1.f + expf(ze));  // 1 - sigmoid
          f = ze <= 0.f ? expf(ze - m) * q : 1.f / (1.f + expf(-ze));
        }
      }
      const float sum = group_all<LPT>(f, OpAdd());
      const float n = has ? f / sum : 0.f;
      dot = group_all<LPT>(has ? n * v : 0.f, OpAdd());
      d = n * (v - dot) * q;
    } else if (a.softmax) {
      load_row<NV>(lrow, a.bf16, a.vec != 0, i * NV, a.E, p);
      mask_row<NV>(on ? bits : 0, p);
      float top = -__builtin_inff(), sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) top = p[j] > top ? p[j] : top;
      top = group_all<LPT>(top, OpMax());
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j] = top > -__builtin_inff() ? expf(p[j] - top) : 0.f;
        sum += p[j];
      }
      sum = group_all<LPT>(sum, OpAdd());
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) p[j] *= inv;
      d = has ? expf(ze - top) * inv * v : 0.f;
      dot = group_all<LPT>(d, OpAdd());
    } else if (has) {
      d = v * (1.f / (1.f + expf(-ze))) * (1.f / (1.f + expf(ze)));
    }
    slots[threadIdx.x] = Slot{e, d};
    wave_sync();
    float o[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) o[j] = dense ? -p[j] * dot : 0.f;
    for (int r = 0; r < a.k; ++r) {
      const Slot s = slots[base + r];
      const int c = s.e - i * NV;
#pragma unroll
      for (int j = 0; j < NV; ++j) o[j] += c == j ? s.d : 0.f;
    }
    wave_sync();
    if (!in) continue;
    const int c0 = i * NV;
    if (NV % 8 == 0 && vec_out && c0 + NV <= a.E) {
      if (a.bf16) {
        u32x4* out = reinterpret_cast<u32x4*>((uint16_t*)dlogits + t * ldd + c0);
#pragma unroll
        for (int q = 0; q < NV / 8; ++q)
          out[q] = u32x4{pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                         pack_bf16x2(o[8 * q + 4], o[8 * q + 5]),
                         pack_bf16x2(o[8 * q + 6], o[8 * q + 7])};
      } else {
        f32x4* out = reinterpret_cast<f32x4*>((float*)dlogits + t * ldd + c0);
#pragma unroll
        for (int q = 0; q < NV / 4; ++q)
          out[q] = f32x4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]};
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c0 + j < a.E) {
          if (a.bf16)
            ((uint16_t*)dlogits)[t * ldd + c0 + j] = (uint16_t)f32_to_bf16_bits(o[j]);
          else
            ((float*)dlogits)[t * ldd + c0 + j] = o[j];
        }
    }
  }
}

// --------------------------------------------------------------- the share
// Stable compaction of the slots whose expert is resident: a count per block
// of `chunk` consecutive slots, then every block adds up the counts before it
// (at most kShareBlocks) and writes its own.
__device__ __forceinline__ bool resident(int e, int e0, int E) {
  return e >= e0 && e - e0 < E;
}

__global__ __launch_bounds__(256) void k_share_count(int64_t n, int chunk, const int32_t* expert,
                                                     int e0, int E, int32_t* cnt) {
  __shared__ int lds[4];
  const int64_t p0 = (int64_t)blockIdx.x * chunk, p1 = min<int64_t>(p0 + chunk, n);
  int c = 0;
  for (int64_t p = p0 + threadIdx.x; p < p1; p += 256) c += resident(expert[p], e0, E) ? 1 : 0;
  c = wave_sum(c);
  if (lane_id() == 0) lds[threadIdx.x >> 6] = c;
  __syncthreads();
  if (threadIdx.x == 0) cnt[blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

__global__ __launch_bounds__(256) void k_share_write(int64_t n, int chunk, int k,
                                                     const int32_t* expert, const float* weight,
                                                     int e0, int E, const int32_t* cnt,
                                                     int32_t* out_token, int32_t* out_expert,
                                                     float* out_weight, int32_t* out_slot,
                                                     int32_t* out_n) {
  __shared__ int lds[256 / kWave + 1];
  int before = 0;
  if (cnt)
    for (int b = threadIdx.x; b < (int)blockIdx.x; b += 256) before += cnt[b];
  int run, total;
  block_excl_scan<256>(before, lds, &run);  // run: slots kept by the blocks before
  const int64_t p0 = (int64_t)blockIdx.x * chunk, p1 = min<int64_t>(p0 + chunk, n);
  for (int64_t b0 = p0; b0 < p1; b0 += 256) {
    const int64_t p = b0 + threadIdx.x;
    const int e = p < p1 ? expert[p] : -1;
    const bool in = p < p1 && resident(e, e0, E);
    const int at = run + block_excl_scan<256>(in ? 1 : 0, lds, &total);
    if (in) {
      out_expert[at] = e - e0;
      out_weight[at] = weight[p];
      if (out_token) out_token[at] = (int32_t)(p / k);
      if (out_slot) out_slot[at] = (int32_t)p;
    }
    run += total;
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) out_n[0] = run;
}

template <int LPT, int NV>
hipError_t route_launch(const RouteArgs& a, int32_t* counts, hipStream_t s) {
  constexpr int nt = route_threads<NV>(), tpb = nt / LPT;
  const int64_t nblk = ((int64_t)a.T + tpb - 1) / tpb;
  const int grid = (int)(nblk < kRouteBlocks ? nblk : kRouteBlocks);
  const size_t sh = (a.n_group > 1 ? (size_t)tpb * a.E * 8 : 0) + (counts ? (size_t)a.E * 4 : 0);
  RouteArgs b = a;
  b.counts = counts ? (grid == 1 ? counts : a.counts) : nullptr;
  LRM_LAUNCH(grid, nt, sh, s, k_route<LPT, NV>)(b);
  if (counts && grid > 1)
    LRM_LAUNCH((a.E + 31) / 32, 256, 0, s, k_route_counts)(grid, a.E, a.counts, counts);
  return hipGetLastError();
}

template <int LPT, int NV>
hipError_t route_bwd_launch(const RouteArgs& a, const int32_t* expert, const float* dweight,
                            void* dlogits, int64_t ldd, int vec_out, hipStream_t s) {
  constexpr int tpb = kRouteThreads / LPT;
  const int64_t nblk = ((int64_t)a.T + tpb - 1) / tpb;
  LRM_LAUNCH((unsigned)(nblk < (1 << 20) ? nblk : (1 << 20)), kRouteThreads, 0, s, k_route_bwd<LPT, NV>)(
      a, expert, dweight, dlogits, ldd, vec_out);
  return hipGetLastError();
}

}  // namespace

// Lanes and values per lane: enough lanes for the k choices, enough values for
// the E experts.
#define LRM_ROUTE_DISPATCH(CALL)                          \
  if (a.k <= 16 && a.E <= 128) return CALL(16, 8);        \
  if (a.k <= 32 && a.E <= 256) return CALL(32, 8);        \
  if (a.E <= 512) return CALL(64, 8);                     \
  if (a.E <= 1024) return CALL(64, 16);                   \
  return CALL(64, 64);

hipError_t launch_route(const RouteArgs& a, int32_t* counts, hipStream_t s) {
  if (a.T <= 0) {
    if (counts) return launch_fill_u32(reinterpret_cast<uint32_t*>(counts), 0u, a.E, s);
    return hipSuccess;
  }
#define LRM_CALL(L, V) route_launch<L, V>(a, counts, s)
  LRM_ROUTE_DISPATCH(LRM_CALL)
#undef LRM_CALL
}

hipError_t launch_route_bwd(const RouteArgs& a, const int32_t* expert, const float* dweight,
                            void* dlogits, int64_t ldd, int vec_out, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
#define LRM_CALL(L, V) route_bwd_launch<L, V>(a, expert, dweight, dlogits, ldd, vec_out, s)
  LRM_ROUTE_DISPATCH(LRM_CALL)
#undef LRM_CALL
}

int share_chunk(int64_t n) {
  const int64_t c = (n + kShareBlocks - 1) / kShareBlocks;
  return (int)(c <= 2048 ? 2048 : (c + 255) / 256 * 256);
}

hipError_t launch_route_share(int64_t n, int k, const int32_t* expert, const float* weight, int e0,
                              int E, int32_t* out_token, int32_t* out_expert, float* out_weight,
                              int32_t* out_slot, int32_t* out_n, int32_t* cnt, hipStream_t s) {
  if (n <= 0) return launch_fill_u32(reinterpret_cast<uint32_t*>(out_n), 0u, 1, s);
  const int chunk = share_chunk(n);
  const int nblk = (int)((n + chunk - 1) / chunk);
  if (nblk > 1) LRM_LAUNCH(nblk, 256, 0, s, k_share_count)(n, chunk, expert, e0, E, cnt);
  LRM_LAUNCH(nblk, 256, 0, s, k_share_write)(n, chunk, k, expert, weight, e0, E,
                                             nblk > 1 ? cnt : nullptr, out_token, out_expert,
                                             out_weight, out_slot, out_n);
  return hipGetLastError();
}

}  // namespace lrm
