// Backward pass of the expert forward's epilogue: for pair p with output
// y_p = act(z_p) and incoming gradient dy_p (its dY row)
//   dweight[p] = <dy_p, act(z_p)>,  G[p] = dy_p act'(z_p),
//   dbias[e] = sum over the pairs of e of w_p dy_p act'(z_p).
// (G is what the LRMoE score and weight gradient take: page 1, bullet "Отбор по
// метрике LRM"; the routing weight stays a factor of its own.)
//
// HBM-bound: dY (read once per pair, its token's pairs are neighbours and hit
// in L2) and Z in, G out.  Without dbias one wave takes one pair.  With dbias
// the pairs are taken in expert order: a block holds a run of one expert's
// pairs, a wave a row at a time with its columns in registers, so that one
// pass over the data makes all three outputs; the column sums of the blocks
// are joined by a second launch in a fixed order.  Measured: dweight alone
// (131072 pairs, 2048 columns, bf16) 99 us for 606 MB, 6.1 TB/s of reads; with
// G and dbias and GELU (32768 pairs, 1408 columns) 64 us for 197 MB, of which the
// arithmetic is 45 (33 vector instructions an element, two of them at a quarter
// of the rate), and 6 us for the join.  With bf16 data the activations are good
// to 16 2^-24 (1 + |z|) (see act_both), also in the sums that leave in fp32: the
// data's own rounding is 2^-8 |z|.
#include "common.h"
#include "launch.h"

namespace lrm {

namespace {

// Eight consecutive values of a row (columns at or past d: zeros).
template <bool BF16>
__device__ __forceinline__ void load8(const void* row, int c, int d, float (&v)[8]) {
  if constexpr (BF16) {  // d is a multiple of 8
    u32x4 x = {0u, 0u, 0u, 0u};
    if (c < d) x = *reinterpret_cast<const u32x4*>((const uint16_t*)row + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(x[j]);
      v[2 * j + 1] = bf16_hi(x[j]);
    }
  } else {  // d is a multiple of 4
    f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
    if (c < d) x = *reinterpret_cast<const f32x4*>((const float*)row + c);
    if (c + 4 < d) y = *reinterpret_cast<const f32x4*>((const float*)row + c + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = x[j];
      v[4 + j] = y[j];
    }
  }
}
template <bool BF16>
__device__ __forceinline__ void store8(void* row, int c, int d, const float (&v)[8]) {
  if constexpr (BF16) {
    if (c < d)
      *reinterpret_cast<u32x4*>((uint16_t*)row + c) =
          u32x4{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[4], v[5]),
                cvt_pk_bf16(v[6], v[7])};
  } else {
    if (c < d) *reinterpret_cast<f32x4*>((float*)row + c) = f32x4{v[0], v[1], v[2], v[3]};
    if (c + 4 < d) *reinterpret_cast<f32x4*>((float*)row + c + 4) = f32x4{v[4], v[5], v[6], v[7]};
  }
}

__device__ __forceinline__ const void* row_at(const void* m, int64_t r, int64_t ld, bool bf16) {
  return (const char*)m + r * ld * (bf16 ? 2 : 4);
}

// One wave per pair, in pair order: dweight and G.
template <bool BF16, int ACT>
__global__ __launch_bounds__(256) void k_pair_grad(PairGradArgs a) {
  const int p = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (a.err && blockIdx.x == 0 && threadIdx.x == 0) a.err[0] = 0u;
  if (p >= a.N) return;
  const int e = a.expert[p], t = a.token[p];
  const bool there = e >= 0 && e < a.E && t >= 0 && t < a.T;
  const void* dy = row_at(a.dY, a.dy_pair ? p : (there ? t : 0), a.ldy, BF16);
  const void* z = row_at(a.Z, p, a.ldz, BF16);
  void* g = a.G ? (char*)a.G + (int64_t)p * a.d * (BF16 ? 2 : 4) : nullptr;
  float sum = 0.f;
  for (int c = lane_id() * 8; c < a.d; c += kWave * 8) {
    float y8[8], z8[8], g8[8];
    if (there) {
      load8<BF16>(dy, c, a.d, y8);
      load8<BF16>(z, c, a.d, z8);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g8[j] = 0.f;
      if (there) {
        float act, der;
        act_both<ACT, BF16>(z8[j], act, der);
        sum = fmaf(y8[j], act, sum);
        g8[j] = y8[j] * der;
      }
    }
    if (g) store8<BF16>(g, c, a.d, g8);
  }
  if (a.dweight) {
    sum = wave_sum(sum);
    if (lane_id() == 0) a.dweight[p] = sum;
  }
}

// Expert order: block (s, e, column block) takes rows [M s / S, M (s + 1) / S)
// of expert e's M pairs and the columns [cb, cb + NC * 512).
template <bool BF16, int ACT, int NC>
__global__ __launch_bounds__(256) void k_pair_grad_bias(PairGradArgs a) {
  __shared__ float lds[4][NC * 512];
  const int e = blockIdx.y, s = blockIdx.x, S = gridDim.x;
  const int cb = blockIdx.z * NC * 512;
  const int o = a.offsets[e], M = a.offsets[e + 1] - o;
  const int r0 = (int)((int64_t)M * s / S), r1 = (int)((int64_t)M * (s + 1) / S);
  const int w = threadIdx.x >> 6, l = lane_id();
  float acc[NC][8];
#pragma unroll
  for (int q = 0; q < NC; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[q][j] = 0.f;
  for (int r = r0 + w; r < r1; r += 4) {
    const int p = a.kept[o + r];
    const float wt = a.weight[p];
    const void* dy = row_at(a.dY, a.dy_pair ? p : a.token[p], a.ldy, BF16);
    const void* z = row_at(a.Z, p, a.ldz, BF16);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < NC; ++q) {
      const int c = cb + q * 512 + l * 8;
      float y8[8], z8[8], g8[8];
      load8<BF16>(dy, c, a.d, y8);
      load8<BF16>(z, c, a.d, z8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float act, der;
        act_both<ACT, BF16>(z8[j], act, der);
        sum = fmaf(y8[j], act, sum);
        g8[j] = y8[j] * der;
        acc[q][j] = fmaf(wt, g8[j], acc[q][j]);
      }
      if (a.G) store8<BF16>((char*)a.G + (int64_t)p * a.d * (BF16 ? 2 : 4), c, a.d, g8);
    }
    if (a.dweight) {
      sum = wave_sum(sum);
      if (l == 0) a.dweight[p] = sum;
    }
  }
#pragma unroll
  for (int q = 0; q < NC; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[w][q * 512 + l * 8 + j] = acc[q][j];
  __syncthreads();
  float* out = a.part + ((int64_t)s * a.E + e) * a.d;
  for (int c = threadIdx.x; c < NC * 512 && cb + c < a.d; c += 256)
    out[cb + c] = (lds[0][c] + lds[1][c]) + (lds[2][c] + lds[3][c]);
}

// dbias = sum of the S partial sums, in order; and the outputs of absent pairs.
template <bool BF16>
__global__ __launch_bounds__(256) void k_pair_grad_join(PairGradArgs a, int S) {
  const int64_t n = (int64_t)a.E * a.d;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    float v = 0.f;
    for (int s0 = 0; s0 < S; s0 += 8) {
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = a.part[(s0 + q < S ? s0 + q : 0) * n + i];
#pragma unroll
      for (int q = 0; q < 8; ++q) v += s0 + q < S ? x[q] : 0.f;
    }
    a.dbias[i] = v;
  }
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < a.N; p += step) {
    if (a.pos[p] >= 0) continue;
    if (a.dweight) a.dweight[p] = 0.f;
    if (a.G) {
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < a.d; c += 8)
        store8<BF16>((char*)a.G + p * a.d * (BF16 ? 2 : 4), c, a.d, zero);
    }
  }
}

template <bool BF16, int ACT>
hipError_t launch_act(const PairGradArgs& a, hipStream_t s) {
  const bool one_pass = a.dbias && a.d <= kPairGradCols;
  if (!one_pass && (a.dweight || a.G || !a.dbias)) {
    PairGradArgs b = a;
    if (a.dbias) b.err = nullptr;
    LRM_LAUNCH(a.N > 0 ? (a.N + 3) / 4 : 1, 256, 0, s, k_pair_grad<BF16, ACT>)(b);
  }
  if (a.dbias) {
    PairGradArgs b = a;
    if (!one_pass) {
      b.dweight = nullptr;
      b.G = nullptr;
    }
    const int S = pair_grad_splits(a.N, a.E);
    const int nc = (a.d + 511) / 512;
    if (nc <= 1)
      LRM_LAUNCH(dim3(S, a.E, 1), 256, 0, s, k_pair_grad_bias<BF16, ACT, 1>)(b);
    else if (nc <= 2)
      LRM_LAUNCH(dim3(S, a.E, 1), 256, 0, s, k_pair_grad_bias<BF16, ACT, 2>)(b);
    else if (nc <= 3)
      LRM_LAUNCH(dim3(S, a.E, 1), 256, 0, s, k_pair_grad_bias<BF16, ACT, 3>)(b);
    else
      LRM_LAUNCH(dim3(S, a.E, (nc + 3) / 4), 256, 0, s, k_pair_grad_bias<BF16, ACT, 4>)(b);
    const int64_t n = (int64_t)a.E * a.d;
    const int64_t blocks = ((n > a.N ? n : a.N) + 255) / 256;
    const int grid = (int)(blocks < 2048 ? blocks : 2048);
    LRM_LAUNCH(grid, 256, 0, s, k_pair_grad_join<BF16>)(a, S);
  }
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_type(const PairGradArgs& a, hipStream_t s) {
  switch (a.act) {
    case kActRelu: return launch_act<BF16, kActRelu>(a, s);
    case kActGelu: return launch_act<BF16, kActGelu>(a, s);
    case kActSilu: return launch_act<BF16, kActSilu>(a, s);
    default: return launch_act<BF16, kActNone>(a, s);
  }
}

}  // namespace

// Splits of an expert's pairs: about 2048 blocks in all, none for fewer than
// 16 pairs of an average expert.
int pair_grad_splits(int N, int E) {
  const int by_rows = (int)(((int64_t)N + (int64_t)E * 16 - 1) / ((int64_t)E * 16));
  const int by_blocks = (2048 + E - 1) / E;
  const int s = by_rows < by_blocks ? by_rows : by_blocks;
  return s < 1 ? 1 : s;
}

hipError_t launch_pair_grad(const PairGradArgs& a, hipStream_t s) {
  if (a.dbias && (!a.offsets || !a.kept || !a.pos || !a.part)) return hipErrorInvalidValue;
  return a.bf16 ? launch_type<true>(a, s) : launch_type<false>(a, s);
}

}  // namespace lrm
