// The experts' forward pass for few pairs (decoding: at most kFewPairs, one a
// lane): no bucketing, no row tiles.  The time is the weights' bytes of the
// experts that the pairs name, and for one token the chain of dependent loads,
// so the kernels keep that chain short (the pairs' experts and tokens in one
// step, then weights and rows together), keep many weight loads in flight and
// spread an expert's weight rows over many blocks.
//
// k_fwd_few: a block takes one expert and 16 NF weight rows (GLU: 8 NF of each
// product, gate and up halves of one fragment) and multiplies 16 of its pairs
// at a time: its four waves split K, 128 bytes of a weight row at a time, from
// memory straight into MFMA fragments (no weight is used by two waves, so LDS
// would only add a copy), and join their sums in LDS.
// k_fwd_few_join: a block takes one token and 8 output columns; a wave takes a
// pair of the token, and the weighted sum over them and the residual happen on
// the way out, so that one decoded token needs two launches.  Every token
// reads its experts' weights on its own.  It multiplies in fp32, so silu(a) b
// comes to it in fp32 too (h32; 24 KB for a token of 8 pairs, from the L2); the
// MFMA products take it in the inputs' type.
//
// Sums are made in a fixed order.
//
// One token of a Qwen3-shaped layer (8 experts, 75.5 MB of weights): 12.5 us for
// gate and up, 7.4 us for the down product and the join; a copy of those bytes
// takes 16 us.
#include "common.h"
#include "gemm_util.h"
#include "launch.h"

namespace lrm {

namespace {

constexpr int kWaves = 4;      // of k_fwd_few: they split K
constexpr int kJoinWaves = 8;  // of k_fwd_few_join: a pair each

// The pairs, one a lane (every wave on its own).
struct FewPairs {
  int e, t;   // of pair `lane`; -1 past N
  bool here;  // inside the ranges
  __device__ __forceinline__ explicit FewPairs(const FwdFewArgs& g) {
    const int p = lane_id();
    e = t = -1;
    if (g.N > 0) {  // (the arrays may be null without pairs)
      const int at = p < g.N ? p : 0, ev = g.expert[at], tv = g.token[at];
      e = p < g.N ? ev : -1;
      t = p < g.N ? tv : -1;
    }
    here = p < g.N && (unsigned)e < (unsigned)g.E && (unsigned)t < (unsigned)g.T;
  }
  // the bits that the bucketing reports
  __device__ __forceinline__ uint32_t errors(const FwdFewArgs& g) const {
    const int p = lane_id(), before = __shfl_up(t, 1, kWave);
    uint32_t b = 0;
    if (__ballot(p < g.N && (unsigned)e >= (unsigned)g.E)) b |= kErrExpertRange;
    if (__ballot(p < g.N && (unsigned)t >= (unsigned)g.T)) b |= kErrTokenRange;
    if (__ballot(p > 0 && p < g.N && before > t)) b |= kErrTokenOrder;
    return b;
  }
};

// list[i] = the i-th set bit of m (a wave's own piece of LDS)
__device__ __forceinline__ void list_bits(uint64_t m, int* list) {
  const int l = lane_id();
  if ((m >> l) & 1) list[__popcll(m & ((1ull << l) - 1))] = l;
  wave_sync();
}

template <bool BF16>
__device__ __forceinline__ f32x4 few_mma(u32x4 b, u32x4 a, f32x4 c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b),
                                                   __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[s]), __uint_as_float(a[s]), c, 0, 0, 0);
    return c;
  }
}

// acc[f] += the product of 16-byte granules over the units u = u0, u0 + step, ..
// of 128 bytes of a row of kb bytes; brow[f], arow: this lane's rows.  Granules
// past K read the row's last ones, times zero (weights are finite).  UB units
// are loaded before the first is multiplied.
template <bool BF16, int NF, int UB>
__device__ __forceinline__ void sweep(const char* const (&brow)[NF], const char* arow, int kb, int u0,
                                      int step, f32x4 (&acc)[NF]) {
  const int lane = (lane_id() >> 4) * 16, last = kb - 16, units = (kb + 127) / 128;
  for (int u = u0; u < units; u += UB * step) {
    u32x4 b[UB][2][NF], a[UB][2];
#pragma unroll
    for (int q = 0; q < UB; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (u + q * step) * 128 + h * 64 + lane, kc = k < last ? k : last;
#pragma unroll
        for (int f = 0; f < NF; ++f) b[q][h][f] = *reinterpret_cast<const u32x4*>(brow[f] + kc);
        a[q][h] = *reinterpret_cast<const u32x4*>(arow + kc);
      }
#pragma unroll
    for (int q = 0; q < UB; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (u + q * step) * 128 + h * 64 + lane;
        const u32x4 av = k <= last ? a[q][h] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = few_mma<BF16>(b[q][h][f], av, acc[f]);
      }
  }
}

template <bool BF16>
__device__ __forceinline__ void put4(void* base, int64_t at, f32x4 v) {
  if constexpr (BF16)
    *reinterpret_cast<u32x2*>((uint16_t*)base + at) =
        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  else
    *reinterpret_cast<f32x4*>((float*)base + at) = v;
}
template <bool BF16>
__device__ __forceinline__ float get1(const void* base, int64_t at) {
  return BF16 ? bf16_to_f32(((const uint16_t*)base)[at]) : ((const float*)base)[at];
}

__device__ __forceinline__ f32x4 act4(int act, f32x4 z) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    z[q] = act == kActRelu   ? act_of<kActRelu, false>(z[q])
           : act == kActGelu ? act_of<kActGelu, false>(z[q])
           : act == kActSilu ? act_of<kActSilu, false>(z[q])
                             : z[q];
  return z;
}

template <bool BF16>
__device__ __forceinline__ float dot16(u32x4 x, u32x4 y) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      s = fmaf(bf16_lo(x[k]), bf16_lo(y[k]), s);
      s = fmaf(bf16_hi(x[k]), bf16_hi(y[k]), s);
    } else {
      s = fmaf(__uint_as_float(x[k]), __uint_as_float(y[k]), s);
    }
  }
  return s;
}

// x: the same values' partners in fp32 (V / 4 vectors of four)
template <bool BF16>
__device__ __forceinline__ float dot16(u32x4 w, const f32x4* x, float s) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      s = fmaf(bf16_lo(w[k]), x[k >> 1][2 * (k & 1)], s);
      s = fmaf(bf16_hi(w[k]), x[k >> 1][2 * (k & 1) + 1], s);
    } else {
      s = fmaf(__uint_as_float(w[k]), x[0][k], s);
    }
  }
  return s;
}

// What becomes of four consecutive columns c .. of pair p: u = W0 x, v = W1 x.
template <bool BF16, bool GLU>
__device__ __forceinline__ void few_emit(const FwdFewArgs& g, int e, int p, int c, f32x4 u, f32x4 v) {
  const int64_t at = (int64_t)p * g.n + c;
  if constexpr (GLU) {
    if (g.A) put4<BF16>(g.A, at, u);
    if (g.B) put4<BF16>(g.B, at, v);
    f32x4 h;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = u[k] * sigmoidf_acc(u[k]) * v[k];
    if (g.h32)
      put4<false>(g.H, at, h);
    else
      put4<BF16>(g.H, at, h);
  } else {
    if (g.bias) {
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] += get1<BF16>(g.bias, (int64_t)e * g.n + c + k);
    }
    if (g.Z) put4<BF16>(g.Z, at, u);
    if (g.act != kActNone) u = act4(g.act, u);
    if (g.Y) put4<BF16>(g.Y, at, u);
    if (g.Yf) *reinterpret_cast<f32x4*>(g.Yf + at) = u;
  }
}

template <bool BF16, bool GLU, int NF>
__global__ __launch_bounds__(256, 2) void k_fwd_few(FwdFewArgs g) {
  constexpr int ES = BF16 ? 2 : 4, COLS = GLU ? 8 * NF : 16 * NF;
  __shared__ int lists[kWaves][kWave];
  __shared__ f32x4 red[kWaves][NF][kWave];
  const int w = threadIdx.x >> 6, l = lane_id();
  const int n0 = blockIdx.x * COLS;
  const FewPairs pairs(g);
  if (g.err && blockIdx.x == 0 && blockIdx.y == 0) {
    const uint32_t b = pairs.errors(g);
    if (threadIdx.x == 0) g.err[0] = b;
  }
  // the block's expert: blockIdx.y itself, or (fewer pairs than experts) that
  // of pair blockIdx.y, if no earlier pair has it
  const int e = g.by_pair ? __shfl(pairs.e, (int)blockIdx.y, kWave) : (int)blockIdx.y;
  const uint64_t m = __ballot(pairs.here && pairs.e == e);
  if (m == 0 || (g.by_pair && __builtin_ctzll(m) != (int)blockIdx.y)) return;
  const int M = __popcll(m);
  int* list = lists[w];
  list_bits(m, list);
  const int kb = g.K * ES;
  const char* brow[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int r = l & 15;
    const int c = n0 + (GLU ? f * 8 + (r & 7) : f * 16 + r);
    const char* W = (const char*)(GLU && r >= 8 ? g.W1 : g.W0);
    brow[f] = W + ((int64_t)e * g.w_stride + (int64_t)(c < g.n ? c : g.n - 1) * g.K) * ES;
  }
  if (NF == 1 && M == 1) {
    // one pair: a wave takes four of the 16 weight rows, 1 KB of a row a load
    // (16 rows x 64 bytes a load, as the fragments have it: two tokens of the
    // Qwen3-shaped layer 38 us instead of 32), 16 KB of weights in flight
    constexpr int UB = 4;
    const int p = list[0], t = __shfl(pairs.t, p, kWave), G = kb / 16;
    const u32x4* x = reinterpret_cast<const u32x4*>((const char*)g.X +
                                                    (int64_t)(g.x_pair ? p : t) * g.ldx * ES);
    const u32x4* row[4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
      row[r] = reinterpret_cast<const u32x4*>(
          __builtin_bit_cast(const char*, __shfl((uint64_t)(uintptr_t)brow[0], w * 4 + r, kWave)));
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < G; i0 += UB * kWave) {
      u32x4 a[UB], b[4][UB];
#pragma unroll
      for (int q = 0; q < UB; ++q) {
        const int i = i0 + q * kWave + l, ic = i < G ? i : G - 1;
#pragma unroll
        for (int r = 0; r < 4; ++r) b[r][q] = row[r][ic];
        a[q] = x[ic];
        if (i >= G) a[q] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int q = 0; q < UB; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] += dot16<BF16>(a[q], b[r][q]);
    }
    f32x4 s;
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = wave_sum(sum[r]);
    if (l == 0) red[w][0][0] = s;
    __syncthreads();
    // rows 4 v .. of wave v: columns, or (GLU) waves 0, 1 gate and 2, 3 up
    const int v = threadIdx.x, c = n0 + v * 4;
    if (v < (GLU ? 2 : 4) && c < g.n) {
      const f32x4 u = red[v][0][0];
      few_emit<BF16, GLU>(g, e, p, c, u, GLU ? red[v + (GLU ? 2 : 0)][0][0] : u);
    }
    return;
  }
  for (int m0 = 0; m0 < M; m0 += 16) {
    const int p = list[min(m0 + (l & 15), M - 1)];
    const int t = __shfl(pairs.t, p, kWave);
    const char* arow = (const char*)g.X + (int64_t)(g.x_pair ? p : t) * g.ldx * ES;
    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    sweep<BF16, NF, NF == 1 ? 8 : 2>(brow, arow, kb, w, kWaves, acc);
#pragma unroll
    for (int f = 0; f < NF; ++f) red[w][f][l] = acc[f];
    __syncthreads();
    // lane x of fragment f: pair x & 15, weight rows 4 (x >> 4) .. + 3
    if ((int)threadIdx.x < NF * kWave) {
      const int f = threadIdx.x >> 6, x = l, i = m0 + (x & 15);
      const int c = n0 + f * (GLU ? 8 : 16) + (x >> 4) * 4;
      auto sum = [&](int y) {
        f32x4 s = red[0][f][y];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) s += red[v][f][y];
        return s;
      };
      if (i < M && c < g.n && (!GLU || x < 32)) {
        const f32x4 u = sum(x);
        few_emit<BF16, GLU>(g, e, list[i], c, u, GLU ? sum(x + 32) : u);
      }
    }
    __syncthreads();
  }
}

// acc[r] += the granules i0 .. i0 + UB * kWave - 1 (those below G) of weight row
// r times x, one a lane and step.  All loads are on their way before the first
// product.
template <bool BF16, int UB, int ROWS>
__device__ __forceinline__ void join_step(const u32x4* const (&row)[ROWS], const f32x4* x, int i0,
                                          int G, float (&acc)[ROWS]) {
  constexpr int XV = BF16 ? 2 : 1;
  u32x4 b[UB][ROWS];
  f32x4 a[UB][XV];
#pragma unroll
  for (int q = 0; q < UB; ++q) {
    const int i = i0 + q * kWave + lane_id(), ic = i < G ? i : G - 1;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) b[q][r] = row[r][ic];
#pragma unroll
    for (int v = 0; v < XV; ++v) {
      a[q][v] = x[ic * XV + v];
      if (i >= G) a[q][v] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
#pragma unroll
  for (int q = 0; q < UB; ++q)
#pragma unroll
    for (int r = 0; r < ROWS; ++r) acc[r] = dot16<BF16>(b[q][r], a[q], acc[r]);
}

// The products of one token's pairs and their weighted sum: out[t] = R[t] +
// sum of w_p W0 x_p, with x_p row p of X (silu(a) b in fp32), and Y.  The
// block's 8 weight rows lie one after the other in memory; a wave reads 1 KB of
// each at a time, 16 KB in flight as in k_fwd_few (half of that for the last
// granules, or rows of one KB at most), and holds x over the eight rows.
template <bool BF16>
__global__ __launch_bounds__(512, 2) void k_fwd_few_join(FwdFewArgs g) {
  constexpr int ES = BF16 ? 2 : 4, COLS = 8;
  __shared__ int lists[kJoinWaves][kWave];
  __shared__ float ys[kFewPairs][COLS];
  const int w = threadIdx.x >> 6, l = lane_id();
  const int n0 = blockIdx.x * COLS, t = blockIdx.y;
  const FewPairs pairs(g);
  const int c = n0 + (int)threadIdx.x;  // threads 0 .. 7: a column each
  const bool out = (int)threadIdx.x < COLS && c < g.n;
  float sum = 0.f;
  if (out && g.R) sum = get1<BF16>(g.R, (int64_t)t * g.ldr + c);
  const uint64_t m = __ballot(pairs.here && pairs.t == t);
  const int M = __popcll(m);
  int* list = lists[w];
  list_bits(m, list);
  const int G = g.K * ES / 16;  // granules of a row
  for (int j = w; j < M; j += kJoinWaves) {
    const int p = list[j], e = __shfl(pairs.e, p, kWave);
    const f32x4* x = reinterpret_cast<const f32x4*>((const float*)g.X + (int64_t)p * g.ldx);
    const u32x4* row[COLS];
#pragma unroll
    for (int r = 0; r < COLS; ++r)
      row[r] = reinterpret_cast<const u32x4*>(
          (const char*)g.W0 +
          ((int64_t)e * g.w_stride + (int64_t)(n0 + r < g.n ? n0 + r : g.n - 1) * g.K) * ES);
    float acc[COLS];
#pragma unroll
    for (int r = 0; r < COLS; ++r) acc[r] = 0.f;
    int i0 = 0;
    for (; i0 + kWave < G; i0 += 2 * kWave) join_step<BF16, 2, COLS>(row, x, i0, G, acc);
    if (i0 < G) join_step<BF16, 1, COLS>(row, x, i0, G, acc);
#pragma unroll
    for (int r = 0; r < COLS; ++r) acc[r] = wave_sum(acc[r]);
    if (l == 0) {
#pragma unroll
      for (int r = 0; r < COLS; ++r) ys[j][r] = acc[r];
    }
  }
  __syncthreads();
  if (!out) return;
  for (int j = 0; j < M; ++j) {
    const float y = ys[j][threadIdx.x];
    sum = fmaf(g.weight[list[j]], y, sum);
    if (g.Y) {
      if constexpr (BF16)
        ((uint16_t*)g.Y)[(int64_t)list[j] * g.n + c] = (uint16_t)f32_to_bf16_bits(y);
      else
        ((float*)g.Y)[(int64_t)list[j] * g.n + c] = y;
    }
  }
  if constexpr (BF16)
    ((uint16_t*)g.out)[(int64_t)t * g.n + c] = (uint16_t)f32_to_bf16_bits(sum);
  else
    ((float*)g.out)[(int64_t)t * g.n + c] = sum;
}

// out[t] = R[t] + sum of w_p Yf[p] over the token's pairs: one block per token
// and 1024 columns (the pairs' rows in fp32, not stored in between as bf16).
template <bool BF16>
__global__ __launch_bounds__(256) void k_fwd_few_sum(FwdFewArgs g) {
  __shared__ int lists[256 / kWave][kWave];
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
  const FewPairs pairs(g);
  const uint64_t m = __ballot(pairs.here && pairs.t == t);
  const int M = __popcll(m);
  int* list = lists[threadIdx.x >> 6];
  list_bits(m, list);
  if (c >= g.n) return;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  if (g.R) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = get1<BF16>(g.R, (int64_t)t * g.ldr + c + k);
  }
  constexpr int UB = 8;
  for (int j = 0; j < M; j += UB) {
    f32x4 y[UB];
    float wt[UB];
#pragma unroll
    for (int q = 0; q < UB; ++q) {
      const int p = list[j + q < M ? j + q : M - 1];
      y[q] = *reinterpret_cast<const f32x4*>(g.Yf + (int64_t)p * g.n + c);
      wt[q] = g.weight[p];
    }
#pragma unroll
    for (int q = 0; q < UB; ++q)
      if (j + q < M) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = fmaf(wt[q], y[q][k], sum[k]);
      }
  }
  put4<BF16>(g.out, (int64_t)t * g.n + c, sum);
}

// |H[p]|^2 of every present pair: one wave each (BF16: H is of that type)
template <bool BF16>
__global__ __launch_bounds__(256) void k_fwd_few_sumsq(FwdFewArgs g, double* out) {
  const int p = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (p >= g.N || (unsigned)g.expert[p] >= (unsigned)g.E || (unsigned)g.token[p] >= (unsigned)g.T)
    return;
  double s = 0.0;
  for (int c = lane_id(); c < g.n; c += kWave) {
    const double h = get1<BF16>(g.H, (int64_t)p * g.n + c);
    s = fma(h, h, s);
  }
  s = wave_sum(s);
  if (lane_id() == 0) out[p] = s;
}

template <bool BF16, bool GLU>
hipError_t few_launch(const FwdFewArgs& g, hipStream_t s) {
  const int slots = g.by_pair ? g.N : g.E;
  // 8 (GLU) or 16 weight rows of a product a block while that gives fewer than
  // kFewBlocks blocks; four times as many otherwise
  const int narrow = GLU ? 8 : 16;
  const int64_t blocks = (int64_t)slots * ((g.n + narrow - 1) / narrow);
  if (blocks <= kFewBlocks)
    LRM_LAUNCH(dim3((g.n + narrow - 1) / narrow, slots), 256, 0, s, k_fwd_few<BF16, GLU, 1>)(g);
  else
    LRM_LAUNCH(dim3((g.n + 4 * narrow - 1) / (4 * narrow), slots), 256, 0, s,
               k_fwd_few<BF16, GLU, 4>)(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fwd_few(const FwdFewArgs& g, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  if (g.N > kFewPairs) return hipErrorInvalidValue;
  if (g.bf16) return g.glu ? few_launch<true, true>(g, s) : few_launch<true, false>(g, s);
  return g.glu ? few_launch<false, true>(g, s) : few_launch<false, false>(g, s);
}

hipError_t launch_fwd_few_sumsq(const FwdFewArgs& g, double* out, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  if (g.bf16 && !g.h32)
    LRM_LAUNCH((g.N + 3) / 4, 256, 0, s, k_fwd_few_sumsq<true>)(g, out);
  else
    LRM_LAUNCH((g.N + 3) / 4, 256, 0, s, k_fwd_few_sumsq<false>)(g, out);
  return hipGetLastError();
}

hipError_t launch_fwd_few_join(const FwdFewArgs& g, hipStream_t s) {
  if (g.T <= 0) return hipSuccess;
  if (g.N > kFewPairs || g.T > 65535) return hipErrorInvalidValue;
  const dim3 grid((g.n + 7) / 8, g.T);
  if (g.bf16)
    LRM_LAUNCH(grid, 64 * kJoinWaves, 0, s, k_fwd_few_join<true>)(g);
  else
    LRM_LAUNCH(grid, 64 * kJoinWaves, 0, s, k_fwd_few_join<false>)(g);
  return hipGetLastError();
}

hipError_t launch_fwd_few_sum(const FwdFewArgs& g, hipStream_t s) {
  if (g.T <= 0) return hipSuccess;
  if (g.N > kFewPairs || g.T > 65535) return hipErrorInvalidValue;
  const dim3 grid((g.n + 1023) / 1024, g.T);
  if (g.bf16)
    LRM_LAUNCH(grid, 256, 0, s, k_fwd_few_sum<true>)(g);
  else
    LRM_LAUNCH(grid, 256, 0, s, k_fwd_few_sum<false>)(g);
  return hipGetLastError();
}

}  // namespace lrm
