// Routing to experts: scores, group limit, top-k choice and weights, the
// gradient of the weights with respect to the logits, and the pairs of one
// GPU's experts.  (The pairs are the input of the LRMoE pass: page 1,
// introduction, "pair"; the pages take the router as given.)
//
// A token is handled by LPT lanes (16, 32 or 64 of a wave, so 4, 2 or 1 tokens
// per wave), each holding the NV experts i*NV .. i*NV + NV - 1 of its lane i:
// lower lanes hold lower experts, so a tie between lanes goes to the lowest.
// Keys are kept as unsigned integers that order like the floats (0: not
// eligible).  Up to 512 experts (8 a lane) a key carries its expert's
// complement below it (16 bits of each for bf16 logits, 32 otherwise), so that
// one maximum over the lanes decides key and tie; every lane sorts its 8 once
// and a round only compares the lanes' heads (65536 tokens, 128 experts, top-8:
// 11.8 us, and 3.8 for the counts, instead of 26 with a search of all 8 every
// round; 271 vector instructions for four tokens, 7 us of issue).  Larger rows and
// fp64 keys take the maximum key, then the minimum expert among its holders.
//
// Order of the choice: without a bias the scores order like the logits, which
// are exact.  With a bias, and for sums of two scores, the keys are first
// formed in fp32; their error is below kKeyTol (1 + |key|/8), so a token whose
// neighbouring keys are further apart than that is decided.  The others (a few
// per mille; all, where a bias is -inf: Fixed has no scale then) are chosen again
// from keys formed in fp64.
#include "common.h"
#include "launch.h"

namespace lrm {

namespace {

constexpr int kRouteThreads = 256;

// ---------------------------------------------------------- ordered keys
// (-0 has the key of +0: adding +0 turns it into +0)
__device__ __forceinline__ uint32_t ord_of(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t ord_of(double d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, d + 0.0);
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

// The value in the other 16-lane row of a pair of rows, and in the other half
// of the wave, beside the own one: (even row's, odd row's) and (low, high
// half's), the same in both, so that a commutative op gives both the same bits.
#ifdef LRM_CPU_EMU
template <int DIST>
__device__ __forceinline__ void both_of(uint32_t v, uint32_t& x, uint32_t& y) {
  const uint32_t o = (uint32_t)__shfl_xor((int)v, DIST, kWave);
  x = lane_id() & DIST ? o : v;
  y = lane_id() & DIST ? v : o;
}
#else
template <int DIST>
__device__ __forceinline__ void both_of(uint32_t v, uint32_t& x, uint32_t& y) {
  const auto r = DIST == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                            : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  x = r[0];
  y = r[1];
}
#endif
template <int DIST, typename V, typename Op>
__device__ __forceinline__ V across(V v, Op op) {
  if constexpr (sizeof(V) == 4) {
    uint32_t x, y;
    both_of<DIST>(__builtin_bit_cast(uint32_t, v), x, y);
    return op(__builtin_bit_cast(V, x), __builtin_bit_cast(V, y));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t xl, yl, xh, yh;
    both_of<DIST>((uint32_t)u, xl, yl);
    both_of<DIST>((uint32_t)(u >> 32), xh, yh);
    return op(__builtin_bit_cast(V, (uint64_t)xh << 32 | xl), __builtin_bit_cast(V, (uint64_t)yh << 32 | yl));
  }
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
  if constexpr (LPT >= 32) v = across<16>(v, op);
  if constexpr (LPT >= 64) v = across<32>(v, op);
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

// The same in two steps for 8 values, so that a row is on its way while the one
// before it is worked on: fetched where the whole 8 lie inside an aligned row.
struct RawRow {
  u32x4 q[2];
  __device__ __forceinline__ void fetch(const void* row, int bf16, bool vec, int c0, int E) {
    if (!vec || c0 + 8 > E) return;
    const u32x4* src = reinterpret_cast<const u32x4*>((const char*)row + (int64_t)c0 * (bf16 ? 2 : 4));
    q[0] = src[0];
    if (!bf16) q[1] = src[1];
  }
  __device__ __forceinline__ void values(const void* row, int bf16, bool vec, int c0, int E,
                                         float (&z)[8]) const {
    if (!vec || c0 + 8 > E) {
      load_row<8>(row, bf16, false, c0, E, z);
    } else if (bf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[2 * j] = bf16_lo(q[0][j]);
        z[2 * j + 1] = bf16_hi(q[0][j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[j] = __uint_as_float(q[0][j]);
        z[4 + j] = __uint_as_float(q[1][j]);
      }
    }
  }
};

__device__ __forceinline__ float load_one(const void* row, int bf16, int c) {
  return bf16 ? bf16_to_f32(((const uint16_t*)row)[c]) : ((const float*)row)[c];
}

// e^x in fp32 to about 2 units in the last place, from the hardware's exp2: the
// rounding error of x log2(e) is put back.  x is held to [-150, 88], so that a
// masked logit (-inf) gives 0 and no result is infinite.
__device__ __forceinline__ float exp_of(float x) {
  x = fminf(fmaxf(x, -150.f), 88.f);
  const float t = x * 1.44269502f;  // log2(e) = 1.44269502 + 1.92596299e-8
  const float r = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * 0.693147181f, e);
}
__device__ __forceinline__ double exp_of(double x) { return exp(x); }
// 1 / x for x in [1, 2^127)
__device__ __forceinline__ float inv_of(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return fmaf(r, fmaf(-x, r, 1.f), r);
}
__device__ __forceinline__ double inv_of(double x) { return 1.0 / x; }

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

// Eight keys of a lane in descending order (Batcher's network).
template <typename P>
__device__ __forceinline__ void sort8(P (&s)[8]) {
  auto ce = [&](int x, int y) {
    const P lo = s[x] < s[y] ? s[x] : s[y];
    s[x] = s[x] < s[y] ? s[y] : s[x];
    s[y] = lo;
  };
  ce(0, 1); ce(2, 3); ce(4, 5); ce(6, 7);
  ce(0, 2); ce(1, 3); ce(4, 6); ce(5, 7);
  ce(1, 2); ce(5, 6);
  ce(0, 4); ce(1, 5); ce(2, 6); ce(3, 7);
  ce(2, 4); ce(3, 5);
  ce(1, 2); ce(3, 4); ce(5, 6);
}

// k rounds of choice over packed keys (key above the expert's complement, all
// different, 0: none): lane j of the group ends with the j-th in *got.  check
// as in choose; key(p, q): whether the keys of p and the next one, q, are too
// close to tell.
template <int LPT, typename P, typename CLOSE>
__device__ __forceinline__ bool choose_packed(P (&s)[8], int i, int k, bool check, P* got, CLOSE key) {
  bool close = false;
  P prev = 0;
  *got = 0;
  sort8(s);
  const int rounds = check ? k + 1 : k;
  if (rounds <= 9) {
    // unrolled: after round r only 8 - r keys of a lane can still be asked for
#pragma unroll
    for (int r = 0; r < 9; ++r) {
      if (r < rounds) {
        const P top = group_all<LPT>(s[0], OpMax());
        if (check && r > 0 && top != 0) close |= key(prev, top);
        *got = i == r ? top : *got;
        const bool mine = s[0] == top;
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < 8 - r) s[j] = mine ? s[j + 1] : s[j];
        if (r == 0) s[7] = mine ? 0 : s[7];
        prev = top;
      }
    }
    if (i >= k) *got = 0;
    return close;
  }
  for (int r = 0; r < rounds; ++r) {
    const P top = group_all<LPT>(s[0], OpMax());
    if (check && r > 0 && top != 0) close |= key(prev, top);
    if (i == r && r < k) *got = top;
    const bool mine = s[0] == top;
#pragma unroll
    for (int j = 0; j < 7; ++j) s[j] = mine ? s[j + 1] : s[j];
    s[7] = mine ? 0 : s[7];
    prev = top;
  }
  return close;
}

// fp32 keys (scores, or scores plus bias) as fixed-point numbers above the
// complement of an index below 512, in 32 bits: 23 bits from the least to the
// largest that a key, or half a key or half a sum of two, can be for scores in
// [0, 1] and the biases at hand.  What the fixed point or fp32 cannot tell apart
// is chosen again in fp64.
struct Fixed {
  float base, scale;
  uint32_t tol;
  // least and largest bias
  __device__ __forceinline__ Fixed(float lo, float hi) {
    base = fminf(lo, 0.5f * lo);
    scale = 8388000.f / (1.f + (fmaxf(hi, 0.5f * hi) - base));
    // error of a key: see kKeyTol; two for the two roundings down
    const float big = fmaxf(fabsf(lo), fabsf(hi)) + 1.f;
    const float t = kKeyTol * (1.f + 0.125f * big) * scale + 2.f;
    tol = t < 8388607.f ? (uint32_t)t : 8388607u;  // (a NaN or infinite bias: all too close)
  }
  __device__ __forceinline__ uint32_t pack(float c, int i) const {
    const float q = fminf(fmaxf((c - base) * scale, 0.f), 8388600.f);
    return ((uint32_t)q + 1u) << 9 | (511u - (uint32_t)i);
  }
  __device__ __forceinline__ bool near(uint32_t p, uint32_t q) const { return (p >> 9) - (q >> 9) <= tol; }
  __device__ __forceinline__ static int index(uint32_t p) { return (int)(511u - (p & 511u)); }
};

// Value of v in the lane of the other half of 2 DIST lanes (DIST 1, 2, 4, 8), as
// far as the lanes of a half hold the same value.
template <int DIST>
__device__ __forceinline__ float other_half(float v) {
  constexpr int ctrl = DIST == 1 ? 0xB1 : DIST == 2 ? 0x4E : DIST == 4 ? 0x141 : 0x140;
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, 0xf, 0xf, false));
}

// keep_groups for groups of whole lanes, GL = 1, 2, 4, 8 or 16 of them (8
// experts a lane), without LDS: the two best of a lane, then of the group's
// lanes, then rounds of choice over the groups.
template <int LPT>
__device__ __forceinline__ uint64_t keep_groups8(const RouteArgs& a, const float (&val)[8], int i, int GL,
                                                 const Fixed& fx, bool check, bool* close) {
  const float inf = __builtin_inff();
  float one = -inf, two = -inf;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    two = fmaxf(two, fminf(one, val[j]));
    one = fmaxf(one, val[j]);
  }
  auto merge = [&](float o1, float o2) {
    two = fmaxf(fmaxf(two, o2), fminf(one, o1));
    one = fmaxf(one, o1);
  };
  if (GL > 1) merge(other_half<1>(one), other_half<1>(two));
  if (GL > 2) merge(other_half<2>(one), other_half<2>(two));
  if (GL > 4) merge(other_half<4>(one), other_half<4>(two));
  if (GL > 8) merge(other_half<8>(one), other_half<8>(two));
  const int g = i / GL;
  const bool rep = i % GL == 0 && g < a.n_group && one > -inf;
  const float sc = a.group_top2 && two > -inf ? one + two : one;
  uint64_t kept = 0;
  const int rounds = check ? a.topk_group + 1 : a.topk_group;
  if (check) {
    // (half of a sum, or of the only key; the range reaches down to half keys)
    uint32_t key = rep ? fx.pack(a.group_top2 ? 0.5f * sc : sc, g) : 0u, prev = 0;
    for (int r = 0; r < rounds; ++r) {
      const uint32_t top = group_all<LPT>(key, OpMax());
      if (r > 0 && top != 0 && fx.near(prev, top)) *close = true;
      if (r < a.topk_group && top != 0) kept |= 1ull << (Fixed::index(top) & 63);
      key = key == top ? 0u : key;
      prev = top;
    }
    return kept;
  }
  uint64_t key = rep ? (uint64_t)ord_of(sc) << 32 | (0xffffffffu - (uint32_t)g) : 0ull;
  for (int r = 0; r < rounds; ++r) {
    const uint64_t top = group_all<LPT>(key, OpMax());
    if (top != 0) kept |= 1ull << ((0xffffffffu - (uint32_t)top) & 63u);
    if (key == top) key = 0;
  }
  return kept;
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
    for (int j = 0; j < NV; ++j) s[j] = inv_of((F)1 + exp_of(-(F)z[j]));
  }
}

// The choice of one token with keys in F; true: fp32 keys leave it uncertain.
// SCORED: with a bias or sums of two scores (else the logits are the keys).
template <int LPT, int NV, typename F, bool SCORED>
__device__ __forceinline__ bool choose_token(const RouteArgs& a, const float (&z)[NV],
                                             const float (&bias)[NV], const Fixed& fx, float top,
                                             int i, F* row, int* got, float* zgot) {
  typedef typename KeyOf<F>::type K;
  const F inf = (F)__builtin_inff();
  const bool by_score = SCORED && a.bias != nullptr;
  const bool two = SCORED && a.n_group > 1 && a.group_top2;
  F s[NV];
  bool close = false;
  if (by_score || two) {
    scores<LPT, NV, F>(a, z, top, !by_score, s);
    if (by_score) {
#pragma unroll
      for (int j = 0; j < NV; ++j) s[j] += (F)bias[j];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) s[j] = z[j] == -__builtin_inff() ? -inf : s[j];
  }
  uint64_t kept = ~0ull;
  const int per = a.E / a.n_group;
  if constexpr (NV == 8 && sizeof(F) == 4) {
    // groups of whole lanes
    const int GL = per / 8;
    if (a.n_group > 1 && per % 8 == 0 && GL <= 16 && (GL & (GL - 1)) == 0) {
      const bool sc = by_score || two;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sc ? s[j] : z[j];
      kept = keep_groups8<LPT>(a, v, i, GL, fx, sc, &close);
      kept = (kept >> (i / GL & 63)) & 1 ? ~0ull : 0ull;
    } else if (a.n_group > 1) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = by_score || two ? s[j] : z[j];
      kept = keep_groups<LPT, NV, F>(a, v, i, row, by_score || two, &close);
    }
  } else if (a.n_group > 1) {
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
  if constexpr (NV == 8 && sizeof(F) == 4) {
    const uint32_t below = 0xffffffffu - (uint32_t)(i * 8);
    if (by_score) {
      uint32_t s32[8], w;
#pragma unroll
      for (int j = 0; j < 8; ++j) s32[j] = key[j] ? fx.pack(s[j], i * 8 + j) : 0u;
      close |= choose_packed<LPT>(s32, i, a.k, true, &w,
                                  [&](uint32_t p, uint32_t q) { return fx.near(p, q); });
      *got = w ? Fixed::index(w) : -1;
    } else if (a.bf16) {
      uint32_t s32[8], w;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        s32[j] = key[j] ? (key[j] & 0xffff0000u) | ((below - j) & 0xffffu) : 0u;
      choose_packed<LPT>(s32, i, a.k, false, &w, [](uint32_t, uint32_t) { return false; });
      *got = w ? (int)(0xffffu - (w & 0xffffu)) : -1;
      *zgot = unord(w & 0xffff0000u);  // (the low bits of a bf16 key are zero, or ones under a sign)
      *zgot = __uint_as_float(__float_as_uint(*zgot) & 0xffff0000u);
    } else {
      uint64_t s64[8], w;
#pragma unroll
      for (int j = 0; j < 8; ++j) s64[j] = key[j] ? (uint64_t)key[j] << 32 | (below - j) : 0ull;
      choose_packed<LPT>(s64, i, a.k, false, &w, [](uint64_t, uint64_t) { return false; });
      *got = w ? (int)(0xffffffffu - (uint32_t)w) : -1;
      *zgot = unord((uint32_t)(w >> 32));
    }
  } else {
    close |= choose<LPT, NV, F>(key, i, a.k, by_score, got);
  }
  return close;
}

// Threads per block: one wave where the rows are long (their fp64 keys are
// staged in LDS for the groups).
template <int NV>
constexpr int route_threads() { return NV > 8 ? kWave : kRouteThreads; }

// The weight of a lane's choice from the logits of the token's choices alone
// (zc of the lanes that have one): renormalised, or a sigmoid.
template <int LPT>
__device__ __forceinline__ float chosen_weight(const RouteArgs& a, bool has, float zc) {
  const float ze = has ? zc : -__builtin_inff();
  if (!a.renorm) return has ? a.scale * inv_of(1.f + exp_of(-ze)) : 0.f;
  // softmax: exp(z - m) with m the largest chosen logit.  sigmoid: both
  // numerator and sum times e^-m, m = min(largest chosen logit, 0), so that the
  // sum cannot underflow.
  float m = group_all<LPT>(ze, OpMax());
  if (!a.softmax) m = m < 0.f ? m : 0.f;
  float f = 0.f;
  if (has)
    f = a.softmax ? exp_of(ze - m)
                  : (ze <= 0.f ? exp_of(ze - m) * inv_of(1.f + exp_of(ze)) : inv_of(1.f + exp_of(-ze)));
  const float sum = group_all<LPT>(f, OpAdd());
  return has ? a.scale * (f / sum) : 0.f;
}

// bf16 logits that are the keys as they are (no bias, no groups), in aligned
// rows of whole lanes: keys straight from the words, weights from the keys.
// (A kernel of its own: as a branch of k_route the scalar registers spill, and
// the 65536-token call took 14.2 us when this took 11.3.)
template <int LPT>
__global__ __launch_bounds__(kRouteThreads) void k_route_direct(RouteArgs a) {
  LRM_DYN_SHARED(int, hist);
  constexpr int tpb = kRouteThreads / LPT;
  const int i = threadIdx.x & (LPT - 1), sub = threadIdx.x / LPT;
  const bool lane_on = i * 8 < a.E;
  uint32_t bits = lane_on ? 0xffu : 0u;
  if (a.expert_mask && lane_on) bits = (uint32_t)expert_bits<8>(a, i * 8);
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) hist[e] = 0;
    __syncthreads();
  }
  const uint32_t below = 0xffffu - (uint32_t)(i * 8);
  auto fetch = [&](int64_t t) {
    return *reinterpret_cast<const u32x4*>((const uint16_t*)a.logits + t * a.ld + (lane_on ? i * 8 : 0));
  };
  const int nrow = (a.T - 1) / tpb + 1;
  const int64_t t0 = (int64_t)blockIdx.x * tpb + sub;
  u32x4 raw = fetch(t0 < a.T ? t0 : 0);
  for (int rb = blockIdx.x; rb < nrow; rb += gridDim.x) {
    const int64_t t = (int64_t)rb * tpb + sub, tn = t + (int64_t)gridDim.x * tpb;
    const bool in = t < a.T;
    const u32x4 x = raw;
    if (rb + (int)gridDim.x < nrow) raw = fetch(tn < a.T ? tn : 0);
    const bool on = in && (a.token_mask ? a.token_mask[in ? t : 0] != 0 : true);
    const uint32_t open = on && lane_on ? 0xffffffffu : 0u;
    uint32_t s32[8], w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // both halves: 0x8000 plus the magnitude, or less it (-0 and +0 alike;
      // no half carries into the other)
      const uint32_t neg = (x[j] >> 15) & 0x00010001u;
      const uint32_t y = (x[j] ^ (((neg << 15) - neg) | 0x80008000u)) + neg;
      s32[2 * j] = (y << 16 | (below - 2 * j)) & open;
      s32[2 * j + 1] = ((y & 0xffff0000u) | (below - 2 * j - 1)) & open;
    }
    if (a.expert_mask) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s32[j] = (bits >> j) & 1 ? s32[j] : 0u;
    }
    choose_packed<LPT>(s32, i, a.k, false, &w, [](uint32_t, uint32_t) { return false; });
    // (-inf has key 0x0080: such a choice is none)
    const bool has = i < a.k && w >= 0x00810000u;
    const int e = (int)(0xffffu - (w & 0xffffu));
    const uint32_t hi = w & 0xffff0000u;
    const float zc = __uint_as_float(hi & 0x80000000u ? hi ^ 0x80000000u : 0u - hi);
    const float wt = chosen_weight<LPT>(a, has, zc);
    if (in && i < a.k) {
      const int64_t at = t * a.k + i;
      a.expert[at] = has ? e : -1;
      a.weight[at] = wt;
      if (a.token) a.token[at] = (int32_t)t;
      if (a.counts && has) atomicAdd(&hist[e], 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads)
      a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
  }
}

// (the registers of the fp64 keys would halve the waves of the other tokens:
// at least four a SIMD for rows of up to 512 experts)
template <int LPT, int NV, bool SCORED>
__global__ __launch_bounds__(route_threads<NV>(), NV > 8 ? 1 : 4) void k_route(RouteArgs a) {
  LRM_DYN_SHARED(double, dyn);  // [tokens of a block][E] rows (groups), then int hist[E] (counts)
  constexpr int NT = route_threads<NV>(), tpb = NT / LPT;
  const int i = threadIdx.x & (LPT - 1);
  const int sub = threadIdx.x / LPT;
  const uint64_t bits = expert_bits<NV>(a, i * NV);
  float bias[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = i * NV + j < a.E ? i * NV + j : 0;
    bias[j] = SCORED && a.bias ? a.bias[c] : 0.f;
  }
  // the range of the keys (see Fixed), over the biases of all lanes
  float blo = 0.f, bhi = 0.f;
  if (SCORED && a.bias) {
    blo = bhi = bias[0];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      blo = fminf(blo, bias[j]);
      bhi = fmaxf(bhi, bias[j]);
    }
    blo = group_all<LPT>(blo, OpMin());
    bhi = group_all<LPT>(bhi, OpMax());
  }
  const Fixed fx(blo, bhi);
  double* row64 = a.n_group > 1 ? dyn + (int64_t)sub * a.E : nullptr;
  int* hist = reinterpret_cast<int*>(dyn + (a.n_group > 1 ? (int64_t)tpb * a.E : 0));
  if (a.counts) {
    for (int e = threadIdx.x; e < a.E; e += NT) hist[e] = 0;
    __syncthreads();
  }
  const int nrow = (a.T - 1) / tpb + 1;
  auto row_of = [&](int64_t t) { return (const char*)a.logits + t * a.ld * (a.bf16 ? 2 : 4); };
  RawRow raw;
  if constexpr (NV == 8) {
    const int64_t t0 = (int64_t)blockIdx.x * tpb + sub;
    raw.fetch(row_of(t0 < a.T ? t0 : 0), a.bf16, a.vec != 0, i * 8, a.E);
  }
  for (int rb = blockIdx.x; rb < nrow; rb += gridDim.x) {
    const int64_t t = (int64_t)rb * tpb + sub;
    const bool in = t < a.T;
    const char* lrow = row_of(in ? t : 0);
    const bool on = in && (a.token_mask ? a.token_mask[in ? t : 0] != 0 : true);
    float z[NV], top = -__builtin_inff(), zc = 0.f;  // zc: the choice's logit
    int e = -1;
    if constexpr (NV == 8) {
      raw.values(lrow, a.bf16, a.vec != 0, i * 8, a.E, z);
      const int64_t tn = t + (int64_t)gridDim.x * tpb;
      if (tn < a.T) raw.fetch(row_of(tn), a.bf16, a.vec != 0, i * 8, a.E);
    } else {
      load_row<NV>(lrow, a.bf16, a.vec != 0, i * NV, a.E, z);
    }
    mask_row<NV>(on ? bits : 0, z);
    if (a.softmax && (!a.renorm || a.bias || a.n_group > 1)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) top = z[j] > top ? z[j] : top;
      top = group_all<LPT>(top, OpMax());
    }
    const bool close =
        choose_token<LPT, NV, float, SCORED>(a, z, bias, fx, top, i, (float*)row64, &e, &zc);
    if constexpr (SCORED) {
      if (__ballot(close)) {  // the whole wave again, in fp64
        int e2;
        float z2;
        choose_token<LPT, NV, double, true>(a, z, bias, fx, top, i, row64, &e2, &z2);
        e = e2;
      }
    }
    // weights: lane j holds choice j
    const bool has = i < a.k && e >= 0 && e < a.E;
    if (SCORED || NV > 8) zc = load_one(lrow, a.bf16, has ? e : 0);
    float w;
    if (a.softmax && !a.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) sum += top > -__builtin_inff() ? exp_of(z[j] - top) : 0.f;
      sum = group_all<LPT>(sum, OpAdd());
      w = has ? a.scale * (exp_of(zc - top) / sum) : 0.f;
    } else {
      w = chosen_weight<LPT>(a, has, zc);
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

// counts[e] = sum over the blocks of part[b][e]: 32 experts a block, 32 rows of
// part at a time, eight loads in flight a thread.
__global__ __launch_bounds__(1024) void k_route_counts(int nblk, int E, const int32_t* part,
                                                       int32_t* counts) {
  __shared__ int lds[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c, ec = e < E ? e : 0;
  int s = 0;
  for (int b0 = r; b0 < nblk; b0 += 256) {
    int v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int b = b0 + q * 32;
      v[q] = part[(int64_t)(b < nblk ? b : 0) * E + ec];
      v[q] = b < nblk ? v[q] : 0;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) s += v[q];
  }
  lds[r][c] = s;
  __syncthreads();
  if (r == 0 && e < E) {
#pragma unroll
    for (int q = 1; q < 32; ++q) s += lds[q][c];
    counts[e] = s;
  }
}

// ------------------------------------------------------------- backward
// 65536 tokens, 128 experts, top-8, bf16, renormalised: 12.4 us; 377 vector
// instructions for four tokens, about half of them in the comparisons that spread
// the k slots over a lane's columns, are 10 us of issue.  Where every logit has a
// gradient and the rows are not 16-byte aligned (15001 x 161 fp32: 18.6 us), a
// lane's 8 neighbouring columns take a load and a store each, and the row's lines
// are asked for 8 times: 1.24 M write requests for 9.7 MB.
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
          f = exp_of(ze - m);
        } else {
          q = inv_of(1.f + exp_of(ze));  // 1 - sigmoid
          f = ze <= 0.f ? exp_of(ze - m) * q : inv_of(1.f + exp_of(-ze));
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
        p[j] = top > -__builtin_inff() ? exp_of(p[j] - top) : 0.f;
        sum += p[j];
      }
      sum = group_all<LPT>(sum, OpAdd());
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) p[j] *= inv;
      d = has ? exp_of(ze - top) * inv * v : 0.f;
      dot = group_all<LPT>(d, OpAdd());
    } else if (has) {
      d = v * inv_of(1.f + exp_of(-ze)) * inv_of(1.f + exp_of(ze));
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
  const bool direct = NV == 8 && a.bf16 && a.vec && a.E % 8 == 0 && !a.bias && a.n_group == 1 &&
                      (a.renorm || !a.softmax);
  if (direct)
    LRM_LAUNCH(grid, kRouteThreads, sh, s, k_route_direct<LPT>)(b);
  else if (a.bias || (a.n_group > 1 && a.group_top2))
    LRM_LAUNCH(grid, nt, sh, s, k_route<LPT, NV, true>)(b);
  else
    LRM_LAUNCH(grid, nt, sh, s, k_route<LPT, NV, false>)(b);
  if (counts && grid > 1)
    LRM_LAUNCH((a.E + 31) / 32, 1024, 0, s, k_route_counts)(grid, a.E, a.counts, counts);
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
