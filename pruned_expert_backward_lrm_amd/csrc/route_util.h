// Device-side helpers of the kernels that take a token's row of logits in LPT
// lanes (16, 32 or 64 of a wave), NV consecutive experts a lane.
#pragma once

#include "common.h"
#include "launch.h"

namespace lrm {

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

// Lanes and values per lane: enough lanes for the k choices, enough values for
// the E experts.
#define LRM_ROUTE_DISPATCH(CALL)                          \
  if (a.k <= 16 && a.E <= 128) return CALL(16, 8);        \
  if (a.k <= 32 && a.E <= 256) return CALL(32, 8);        \
  if (a.E <= 512) return CALL(64, 8);                     \
  if (a.E <= 1024) return CALL(64, 16);                   \
  return CALL(64, 64);

}  // namespace lrm
