// The experts' forward pass: grouped products over the packed pairs of each
// expert with their epilogues, and the join of the pairs' rows per token.
// (LRMoE keeps the forward complete: page 1, section "Что делает LRMoE: полный
// прямой проход, обрезанный обратный".)  For packed row m (pair p = kept[m],
// expert e):
//   GLU:  a = W0_e x, b = W1_e x  -> A[p], B[p] (wanted or not), H[m] = silu(a) b
//   else: z = W0_e x + bias_e     -> Z[p], y = act(z) -> Y[p]
//   join: out[t] = R[t] + sum over the pairs p of t of w_p y_p
// x is row token[p] or p of X, or row m of the packed H.
#include "common.h"
#include "launch.h"

namespace lrm {

namespace {

// Largest e with tile[e] <= i (i < tile[E]).
__device__ __forceinline__ int find_tile(const int32_t* tile, int E, int i) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tile[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float act_rt(int act, float z) {
  switch (act) {
    case kActRelu: return act_of<kActRelu>(z);
    case kActGelu: return act_of<kActGelu>(z);
    case kActSilu: return act_of<kActSilu>(z);
  }
  return z;
}

// y between the down product and the join takes 24 bits: its bf16 rounding
// (which is Yp where the caller wants it) and the next 8 bits of the
// difference, as a signed byte of the bit pattern.  With bf16 alone Y would
// carry two roundings of half the terms' size on top of its own.
__device__ __forceinline__ uint32_t split_lo(float y, uint32_t hi) {
  const int d = ((int)__float_as_uint(y) - (int)(hi << 16) + 128) >> 8;
  return (uint32_t)(d > 127 ? 127 : d) & 0xffu;
}
__device__ __forceinline__ float join_bits(uint32_t hi16, int lo8) {
  return __uint_as_float((hi16 << 16) + (uint32_t)(lo8 << 8));
}

// Four consecutive columns c .. c+3 (c < n, n a multiple of 4) of packed row m,
// pair p: the accumulators of W0 (u) and of W1 (v; GLU).
template <bool BF16, bool GLU>
__device__ __forceinline__ void emit4(const FwdGemmArgs& g, int e, int m, int p, int c, f32x4 u, f32x4 v) {
  const int64_t pr = (int64_t)p * g.n + c, mr = (int64_t)m * g.n + c;
  auto put = [](void* dst, int64_t at, f32x4 x) {
    if constexpr (BF16)
      *reinterpret_cast<u32x2*>((uint16_t*)dst + at) =
          u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    else
      *reinterpret_cast<f32x4*>((float*)dst + at) = x;
  };
  if constexpr (GLU) {
    if (g.A) put(g.A, pr, u);
    if (g.B) put(g.B, pr, v);
    f32x4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = u[j] * sigmoidf_acc(u[j]) * v[j];
    put(g.H, mr, h);
  } else {
    if (g.bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = (int64_t)e * g.n + c + j;
        u[j] += BF16 ? bf16_to_f32(((const uint16_t*)g.bias)[at]) : ((const float*)g.bias)[at];
      }
    }
    if (g.Z) put(g.Z, pr, u);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = act_rt(g.act, u[j]);
    if (g.Y) put(g.Y, pr, u);
    if (BF16 && g.Ylo) {
      uint32_t lo = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) lo |= split_lo(u[j], f32_to_bf16_bits(u[j])) << (8 * j);
      *reinterpret_cast<uint32_t*>(g.Ylo + pr) = lo;
    }
  }
}

// Row of the A operand of packed row m.
__device__ __forceinline__ int64_t src_row(const FwdGemmArgs& g, int m) {
  if (!g.gather) return m;
  const int p = g.kept[m];
  return g.x_pair ? p : g.token[p];
}

// 64 x 64 tile of fp32 multiply-adds, 16 k at a time through LDS.
template <bool BF16, bool GLU>
__global__ __launch_bounds__(256) void k_fwd_simple(FwdGemmArgs g) {
  __shared__ float As[16][68], Bs[16][68], Cs[GLU ? 16 : 1][68];
  const int nt = (g.n + 63) / 64;
  const int mt = blockIdx.x / nt, n0 = (int)(blockIdx.x % nt) * 64;
  if (mt >= g.mt_off[g.E]) return;
  const int e = find_tile(g.mt_off, g.E, mt);
  const int m0 = g.offsets[e] + (mt - g.mt_off[e]) * 64;
  const int mend = g.offsets[e + 1];
  const int tr = threadIdx.x >> 4, tc = threadIdx.x & 15;
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 4;  // loads: row, 4 k
  constexpr int ES = BF16 ? 2 : 4;
  const char* arow = nullptr;
  if (m0 + lr < mend) arow = (const char*)g.X + src_row(g, m0 + lr) * g.ldx * ES;
  const char* brow = nullptr;
  const char* crow = nullptr;
  if (n0 + lr < g.n) {
    const int64_t at = (int64_t)e * g.w_stride + (int64_t)(n0 + lr) * g.K;
    brow = (const char*)g.W0 + at * ES;
    if (GLU) crow = (const char*)g.W1 + at * ES;
  }
  auto ld = [&](const char* row, int k, float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 0.f;
    if (!row || k >= g.K) return;
    if constexpr (BF16) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(row + (int64_t)k * 2);
      v[0] = bf16_lo(x[0]); v[1] = bf16_hi(x[0]);
      v[2] = bf16_lo(x[1]); v[3] = bf16_hi(x[1]);
    } else {
      const f32x4 x = *reinterpret_cast<const f32x4*>(row + (int64_t)k * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = x[j];
    }
  };
  f32x4 u[4], v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < g.K; k0 += 16) {
    float x[4], y[4], w[4];
    ld(arow, k0 + lk, x);
    ld(brow, k0 + lk, y);
    if (GLU) ld(crow, k0 + lk, w);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      As[lk + j][lr] = x[j];
      Bs[lk + j][lr] = y[j];
      if (GLU) Cs[lk + j][lr] = w[j];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(&As[k][tr * 4]);
      const f32x4 b = *reinterpret_cast<const f32x4*>(&Bs[k][tc * 4]);
      f32x4 c = b;
      if (GLU) c = *reinterpret_cast<const f32x4*>(&Cs[k][tc * 4]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u[i][j] = fmaf(a[i], b[j], u[i][j]);
          if (GLU) v[i][j] = fmaf(a[i], c[j], v[i][j]);
        }
    }
  }
  const int c = n0 + tc * 4;
  if (c >= g.n) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + tr * 4 + i;
    if (m < mend) emit4<BF16, GLU>(g, e, m, g.kept[m], c, u[i], v[i]);
  }
}

// |H[m]|^2 of every packed row, to the row of its pair.
template <bool BF16>
__global__ __launch_bounds__(256) void k_fwd_sumsq(FwdGemmArgs g, double* out) {
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= g.offsets[g.E]) return;
  double s = 0.0;
  for (int c = lane_id() * 4; c < g.n; c += kWave * 4) {
    f32x4 h;
    if constexpr (BF16) {
      const u32x2 x = *reinterpret_cast<const u32x2*>((const uint16_t*)g.H + (int64_t)m * g.n + c);
      h = f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])};
    } else {
      h = *reinterpret_cast<const f32x4*>((const float*)g.H + (int64_t)m * g.n + c);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s = fma((double)h[j], (double)h[j], s);
  }
  s = wave_sum(s);
  if (lane_id() == 0) out[g.kept[m]] = s;
}

// One wave per token and 512 (bf16) or 256 (fp32) columns.
template <bool BF16>
__global__ __launch_bounds__(256) void k_fwd_join(FwdJoinArgs a) {
  constexpr int V = BF16 ? 8 : 4, COLS = V * kWave;
  const int nblk = (a.d + COLS - 1) / COLS;
  const int64_t gw = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (gw >= (int64_t)a.T * nblk) return;
  const int t = (int)(gw / nblk), c = (int)(gw % nblk) * COLS + lane_id() * V;
  const int p0 = min(max(a.tok_off[t], 0), a.N);
  const int p1 = min(max(a.tok_off[t + 1], p0), a.N);
  if (c >= a.d) return;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  if (a.R) {
    if constexpr (BF16) {
      const u32x4 x = *reinterpret_cast<const u32x4*>((const uint16_t*)a.R + (int64_t)t * a.ldr + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[2 * j] = bf16_lo(x[j]);
        acc[2 * j + 1] = bf16_hi(x[j]);
      }
    } else {
      const f32x4 x = *reinterpret_cast<const f32x4*>((const float*)a.R + (int64_t)t * a.ldr + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = x[j];
    }
  }
  for (int p = p0; p < p1; ++p) {
    if (a.pos[p] < 0) continue;
    const float w = a.weight[p];
    const int64_t at = (int64_t)p * a.d + c;
    if constexpr (BF16) {
      const u32x4 x = *reinterpret_cast<const u32x4*>((const uint16_t*)a.Y + at);
      const u32x2 lo = *reinterpret_cast<const u32x2*>(a.Ylo + at);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t hi = (x[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        const int l8 = (int)(int8_t)(lo[j >> 2] >> (8 * (j & 3)));
        acc[j] = fmaf(w, join_bits(hi, l8), acc[j]);
      }
    } else {
      const f32x4 x = *reinterpret_cast<const f32x4*>((const float*)a.Y + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, x[j], acc[j]);
    }
  }
  const int64_t o = (int64_t)t * a.d + c;
  if constexpr (BF16)
    *reinterpret_cast<u32x4*>((uint16_t*)a.out + o) =
        u32x4{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
              pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7])};
  else
    *reinterpret_cast<f32x4*>((float*)a.out + o) = f32x4{acc[0], acc[1], acc[2], acc[3]};
}

}  // namespace

int fwd_tile_rows(const FwdGemmArgs&) { return 64; }

hipError_t launch_fwd_gemm(const FwdGemmArgs& g, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  const int64_t tiles = ((int64_t)g.N / 64 + g.E) * ((g.n + 63) / 64);
  if (tiles > 0x7fffffffll) return hipErrorInvalidValue;
  if (g.bf16) {
    if (g.glu)
      LRM_LAUNCH((unsigned)tiles, 256, 0, s, k_fwd_simple<true, true>)(g);
    else
      LRM_LAUNCH((unsigned)tiles, 256, 0, s, k_fwd_simple<true, false>)(g);
  } else {
    if (g.glu)
      LRM_LAUNCH((unsigned)tiles, 256, 0, s, k_fwd_simple<false, true>)(g);
    else
      LRM_LAUNCH((unsigned)tiles, 256, 0, s, k_fwd_simple<false, false>)(g);
  }
  return hipGetLastError();
}

hipError_t launch_fwd_sumsq(const FwdGemmArgs& g, double* out, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  if (g.bf16)
    LRM_LAUNCH((g.N + 3) / 4, 256, 0, s, k_fwd_sumsq<true>)(g, out);
  else
    LRM_LAUNCH((g.N + 3) / 4, 256, 0, s, k_fwd_sumsq<false>)(g, out);
  return hipGetLastError();
}

hipError_t launch_fwd_join(const FwdJoinArgs& a, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
  const int cols = a.bf16 ? 8 * kWave : 4 * kWave;
  const int64_t blocks = ((int64_t)a.T * ((a.d + cols - 1) / cols) + 3) / 4;
  if (blocks > 0x7fffffffll) return hipErrorInvalidValue;
  if (a.bf16)
    LRM_LAUNCH((unsigned)blocks, 256, 0, s, k_fwd_join<true>)(a);
  else
    LRM_LAUNCH((unsigned)blocks, 256, 0, s, k_fwd_join<false>)(a);
  return hipGetLastError();
}

}  // namespace lrm
