// Balance of the experts' load: with p_te the experts' shares of token t
//   balance = coef / S' sum over sequences s, experts e of a_se sum over t of p_te,
//   z = z_coef / n sum over t of (log sum_e exp z_te)^2
// (a_se = M f_se / n_s: see lrm.h) and their gradient
//   d balance / d z_tj = coef / S' p_tj (a_sj - sum_e p_te a_se) [(1 - sigma_j)],
//   d z / d z_tj = 2 z_coef / n log(sum) p_tj
// joined with that of the routing weights.  (The pages take a balanced router as
// given; its counts are those of the controller: page 1, bullet "Квоты до вычислений".)
//
// The loss reads the logits once: a block takes a run of tokens (a chunk) and, for
// every sequence that reaches into it, leaves one row of column sums, counts and
// three numbers.  Chunk c and sequence s meet in row c + s: along the tokens one of
// the two grows at a time, so no two pairs share a row and chunks + S rows are
// enough, whatever the offsets (which only the GPU knows).  A second launch adds a
// sequence's rows in fp64, a third one the sequences (not for a single one of up to
// 256 experts).
#include "common.h"
#include "launch.h"
#include "route_util.h"

namespace lrm {

namespace {

template <int NV>
constexpr int balance_threads() { return NV > 8 ? 256 : 512; }

// e^x for x <= 0.  bf16 logits, good to 2^-9 of themselves, take the hardware's
// exp2 of the rounded product (error 2^-24 |x|); fp32 ones put its error back.
template <bool BF16>
__device__ __forceinline__ float exp_row(float x) {
  return BF16 ? __builtin_amdgcn_exp2f(x * 1.44269504f) : exp_of(x);
}

// Shares p of a lane's experts from their eligible logits z (masked: -inf), in
// place; inv_sum their factor; rest (sigmoid): 1 - sigma.  Returns whether the
// token has an eligible expert; lse: log of the exps' sum (softmax).
template <int LPT, int NV, bool BF16, bool SIG, bool GRAD>
__device__ __forceinline__ bool shares(float (&z)[NV], float (&rest)[GRAD && SIG ? NV : 1], float* lse) {
  float top = -__builtin_inff(), sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) top = z[j] > top ? z[j] : top;
  top = group_all<LPT>(top, OpMax());
  const bool live = top > -__builtin_inff();
  if constexpr (SIG) {
    // sigma times e^-m, m = top where every score would be tiny, so that the
    // sum does not underflow
    const float m = live && top < -60.f ? top : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float q = exp_row<BF16>(-fabsf(z[j])), r = inv_of(1.f + q);
      const float up = m < 0.f ? exp_row<BF16>(z[j] - m) : q;
      if constexpr (GRAD) rest[j] = z[j] > 0.f ? q * r : r;
      z[j] = z[j] > 0.f ? r : up * r;  // (0 for -inf)
      sum += z[j];
    }
  } else {
    const float m = live ? top : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = exp_row<BF16>(z[j] - m);
      sum += z[j];
    }
  }
  sum = group_all<LPT>(sum, OpAdd());
  const float inv = live ? 1.f / sum : 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) z[j] *= inv;
  *lse = SIG || !live ? 0.f : top + logf(sum);
  return live;
}

// Largest s in [0, S) with seq[s] <= t, or 0.
__device__ __forceinline__ int sequence_at(const int32_t* seq, int S, int64_t t) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// NV values from column c0 of row t of the output (columns at or past E: none).
template <int NV>
__device__ __forceinline__ void store_row(void* out, bool bf16, bool vec, int64_t at, int c0, int E,
                                          const float (&o)[NV]) {
  if (vec && c0 + NV <= E) {
    if (bf16) {
      u32x4* dst = reinterpret_cast<u32x4*>((uint16_t*)out + at + c0);
#pragma unroll
      for (int q = 0; q < NV / 8; ++q)
        dst[q] = u32x4{cvt_pk_bf16(o[8 * q], o[8 * q + 1]), cvt_pk_bf16(o[8 * q + 2], o[8 * q + 3]),
                       cvt_pk_bf16(o[8 * q + 4], o[8 * q + 5]), cvt_pk_bf16(o[8 * q + 6], o[8 * q + 7])};
    } else {
      f32x4* dst = reinterpret_cast<f32x4*>((float*)out + at + c0);
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) dst[q] = f32x4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + j < E) {
      if (bf16) ((uint16_t*)out)[at + c0 + j] = (uint16_t)f32_to_bf16_bits(o[j]);
      else ((float*)out)[at + c0 + j] = o[j];
    }
}

// ------------------------------------------------------------------- loss
template <int LPT, int NV, bool BF16, bool SIG>
__global__ __launch_bounds__(balance_threads<NV>()) void k_balance(RouteArgs a, BalanceArgs b) {
  LRM_DYN_SHARED(float, dyn);  // [rows][E] column sums, int hist[E]
  constexpr int NT = balance_threads<NV>(), tpb = NT / LPT, NW = NT / kWave;
  constexpr int NR = NV == 8 ? NW : 1;  // rows of column sums: a wave's each, or one in turn
  __shared__ BalanceRow part[NW];
  int* hist = reinterpret_cast<int*>(dyn + NR * a.E);
  const int i = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
  const int w = threadIdx.x >> 6;
  const uint64_t bits = expert_bits<NV>(a, i * NV);
  const int64_t c0 = (int64_t)blockIdx.x * b.chunk;
  const int64_t c1 = min<int64_t>(c0 + b.chunk, a.T);
  if (b.cnt)
    for (int e = threadIdx.x; e < a.E; e += NT) hist[e] = 0;
  for (int s = b.seq ? sequence_at(b.seq, b.S, c0) : 0; s < b.S; ++s) {
    int64_t t0 = c0, t1 = c1;
    if (b.seq) {
      t0 = max<int64_t>(c0, b.seq[s]);
      t1 = min<int64_t>(c1, b.seq[s + 1]);
      if (b.seq[s] >= c1) break;
      if (t0 >= t1) continue;
    }
    float acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.f;
    int live = 0, filled = 0;
    double lse2 = 0.0;
    __syncthreads();  // hist is clear, the row before has been read
    for (int64_t r = t0; r < t1; r += tpb) {
      const int64_t t = r + slot;
      const bool in = t < t1;
      const bool on = in && (a.token_mask ? a.token_mask[in ? t : 0] != 0 : true);
      float z[NV], rest[1], lse;
      load_row<NV>((const char*)a.logits + (in ? t : t0) * a.ld * (BF16 ? 2 : 4), BF16, a.vec != 0, i * NV,
                   a.E, z);
      mask_row<NV>(on ? bits : 0, z);
      const bool has = shares<LPT, NV, BF16, SIG, false>(z, rest, &lse);
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[j] += z[j];
      if (i == 0 && has) {
        ++live;
        lse2 += (double)lse * (double)lse;
      }
      if (b.cnt && on && i < a.k) {
        const int e = b.expert[t * a.k + i];
        const bool named = e >= 0 && e < a.E;
        if (named && (a.expert_mask ? a.expert_mask[named ? e : 0] != 0 : true)) {
          ++filled;
          atomicAdd(&hist[e], 1);
        }
      }
    }
    // the tokens of a wave, then the waves, in order
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (LPT == 16) acc[j] = across<16>(acc[j], OpAdd());
      if constexpr (LPT <= 32) acc[j] = across<32>(acc[j], OpAdd());
    }
    live = wave_sum(live);
    filled = wave_sum(filled);
    lse2 = wave_sum(lse2);
    if (lane_id() == 0) part[w] = BalanceRow{lse2, live, filled};
    for (int q = 0; q < (NR == 1 ? NW : 1); ++q) {
      if ((NR > 1 || q == w) && lane_id() < LPT) {
        float* row = dyn + (NR > 1 ? w : 0) * a.E;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int e = i * NV + j;
          if (e < a.E) row[e] = NR > 1 || q == 0 ? acc[j] : row[e] + acc[j];
        }
      }
      __syncthreads();
    }
    const int64_t at = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < a.E; e += NT) {
      float v = dyn[e];
      for (int q = 1; q < NR; ++q) v += dyn[q * a.E + e];
      b.sums[at * a.E + e] = v;
      if (b.cnt) {
        b.cnt[at * a.E + e] = hist[e];
        hist[e] = 0;
      }
    }
    if (threadIdx.x == 0) {
      BalanceRow v = part[0];
      for (int q = 1; q < NW; ++q) {
        v.lse2 += part[q].lse2;
        v.live += part[q].live;
        v.filled += part[q].filled;
      }
      b.rows[at] = v;
    }
  }
}

// Sum over a block of 1024 threads, in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  __syncthreads();
  if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = lds[0];
  for (int q = 1; q < 16; ++q) s += lds[q];
  return s;
}

// The losses and the batch's factors from the sums over all sequences.
__device__ __forceinline__ void balance_end(const BalanceArgs& b, int E, double bal, double lse2,
                                            double n, double full) {
  const double fb = full > 0.0 ? (double)b.coef / full : 0.0;
  const double fz = n > 0.0 ? (double)b.z_coef / n : 0.0;
  b.loss[0] = (float)(fb * bal);
  b.loss[1] = (float)(fz * lse2);
  b.saved[(int64_t)b.S * E] = (float)((double)b.coef / (full > 0.0 ? full : 1.0));
  b.saved[(int64_t)b.S * E + 1] = (float)(2.0 * (double)b.z_coef / (n > 0.0 ? n : 1.0));
}

// One block for CW columns of one sequence: 1024 / CW threads a column, each
// sixteen rows at a time.
template <int CW>
__global__ __launch_bounds__(1024) void k_balance_join(RouteArgs a, BalanceArgs b) {
  constexpr int RG = 1024 / CW;
  __shared__ double part[RG][CW];
  __shared__ int ipart[RG][CW];
  __shared__ double lds[16];
  const int col = threadIdx.x % CW, rg = threadIdx.x / CW;
  const int e = blockIdx.x * CW + col, ec = e < a.E ? e : 0;
  for (int s = blockIdx.y; s < b.S; s += gridDim.y) {
    // the rows of this sequence (offsets held to the tokens)
    int64_t t0 = 0, t1 = a.T;
    if (b.seq) {
      t0 = max<int64_t>(b.seq[s], 0);
      t1 = min<int64_t>(b.seq[s + 1], a.T);
    }
    const int64_t r0 = t0 < t1 ? t0 / b.chunk + s : 0;
    const int64_t r1 = t0 < t1 ? (t1 - 1) / b.chunk + s + 1 : 0;
    double live = 0.0, filled = 0.0, experts = 0.0, lse2 = 0.0;  // (whole numbers below 2^53)
    for (int64_t r = r0 + threadIdx.x; r < r1; r += 1024) {
      const BalanceRow v = b.rows[r];
      live += (double)v.live;
      filled += (double)v.filled;
      lse2 += v.lse2;
    }
    for (int c = threadIdx.x; c < a.E; c += 1024) {
      experts += !a.expert_mask || a.expert_mask[c] ? 1.0 : 0.0;
      if (b.counts) filled += (double)b.counts[(int64_t)s * a.E + c];
    }
    double P = 0.0;
    int n = 0;
    for (int64_t rr = r0 + rg; rr < r1; rr += 16 * RG) {
      float x[16];
      int y[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t r = rr + q * RG < r1 ? rr + q * RG : rr;
        x[q] = b.sums[r * a.E + ec];
        y[q] = b.cnt ? b.cnt[r * a.E + ec] : 0;
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const bool ok = rr + q * RG < r1;
        P += ok ? (double)x[q] : 0.0;
        n += ok ? y[q] : 0;
      }
    }
    live = block_sum(live, lds);
    filled = block_sum(filled, lds);
    experts = block_sum(experts, lds);
    lse2 = block_sum(lse2, lds);
    part[rg][col] = P;
    ipart[rg][col] = n;
    __syncthreads();
    double bal = 0.0;
    if (rg == 0 && e < a.E) {
      for (int q = 1; q < RG; ++q) {
        P += part[q][col];
        n += ipart[q][col];
      }
      if (b.counts) n = b.counts[(int64_t)s * a.E + e];
      const double f = filled > 0.0 ? (double)n / filled : 0.0;
      const double v = live > 0.0 ? experts * f / live : 0.0;
      b.saved[(int64_t)s * a.E + e] = (float)v;
      if (b.counts_out) b.counts_out[(int64_t)s * a.E + e] = n;
      bal = v * P;
    }
    bal = block_sum(bal, lds);
    if (threadIdx.x == 0) {
      if (b.S == 1 && gridDim.x == 1) {
        balance_end(b, a.E, bal, lse2, live, live > 0.0 ? 1.0 : 0.0);
      } else {
        b.seq_bal[(int64_t)s * gridDim.x + blockIdx.x] = bal;
        if (blockIdx.x == 0) b.seq_rows[s] = BalanceSeq{lse2, live};
      }
    }
  }
}

// The sequences: n of their columns' sums and their numbers, in a fixed order.
__global__ __launch_bounds__(1024) void k_balance_end(int64_t n, int E, BalanceArgs b) {
  __shared__ double lds[16];
  double bal = 0.0, lse2 = 0.0, live = 0.0, full = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) bal += b.seq_bal[i];
  for (int s = threadIdx.x; s < b.S; s += 1024) {
    const BalanceSeq v = b.seq_rows[s];
    lse2 += v.lse2;
    live += v.live;
    full += v.live > 0.0 ? 1.0 : 0.0;
  }
  bal = block_sum(bal, lds);
  lse2 = block_sum(lse2, lds);
  live = block_sum(live, lds);
  full = block_sum(full, lds);
  if (threadIdx.x == 0) balance_end(b, E, bal, lse2, live, full);
}

// --------------------------------------------------------------- gradient
// A block takes a run of tokens; the lanes of a token hold a whole row of p and
// of a.  The chosen slots' part is added in LDS, all slots of a token at once; slot
// after slot where a choice names an expert twice.
template <int LPT, int NV, bool BF16, bool SIG>
__global__ __launch_bounds__(NV > 8 ? kWave : 256) void k_balance_bwd(RouteArgs a, BalanceBwdArgs b) {
  constexpr int NT = NV > 8 ? kWave : 256, tpb = NT / LPT;
  alignas(16) __shared__ float lds[NT * NV];
  const int i = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
  const int c0 = i * NV;
  const uint64_t bits = expert_bits<NV>(a, c0);
  float* row = lds + slot * LPT * NV;
  const float db = (b.dloss ? b.dloss[0] : 1.f) * b.saved[(int64_t)b.S * a.E];
  const float dz = (b.dloss ? b.dloss[1] : 1.f) * b.saved[(int64_t)b.S * a.E + 1];
  float w[NV];
  int s = -1;        // the sequence whose row is in w
  bool inside = false;
  const int64_t r0 = (int64_t)blockIdx.x * b.chunk;
  const int64_t r1 = min<int64_t>(r0 + b.chunk, a.T);
  int at = 0;        // the sequence of the token, or of the last one before it
  if (b.seq) at = sequence_at(b.seq, b.S, r0 + slot);
  for (int64_t r = r0; r < r1; r += tpb) {
    const int64_t t = r + slot;
    const bool in = t < r1;
    const int64_t tc = in ? t : r0;
    const bool on = in && (a.token_mask ? a.token_mask[tc] != 0 : true);
    const char* lrow = (const char*)a.logits + tc * a.ld * (BF16 ? 2 : 4);
    float z[NV], o[NV], rest[SIG ? NV : 1], lse;
    load_row<NV>(lrow, BF16, a.vec != 0, c0, a.E, z);
    int e = -1;
    float zc = -__builtin_inff(), v = 0.f;
    if (b.dweight && on && i < a.k) {
      const int e0 = b.expert[t * a.k + i];
      const bool named = e0 >= 0 && e0 < a.E;
      const int ec = named ? e0 : 0;
      const float x = load_one(lrow, BF16, ec);
      const bool has = named && (a.expert_mask ? a.expert_mask[ec] != 0 : true) && x != -__builtin_inff();
      e = has ? e0 : -1;
      zc = has ? x : -__builtin_inff();
      v = has ? a.scale * b.dweight[t * a.k + i] : 0.f;
    }
    if (b.seq) {
      while (at + 1 < b.S && b.seq[at + 1] <= t) ++at;
      inside = b.seq[at] <= t && t < b.seq[at + 1];
    } else {
      inside = true;
    }
    if (at != s) {
      s = at;
#pragma unroll
      for (int j = 0; j < NV; ++j) w[j] = c0 + j < a.E ? b.saved[(int64_t)s * a.E + c0 + j] : 0.f;
    }
    mask_row<NV>(on ? bits : 0, z);
    shares<LPT, NV, BF16, SIG, true>(z, rest, &lse);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) dot = fmaf(z[j], w[j], dot);
    dot = group_all<LPT>(dot, OpAdd());
    const float gb = inside ? db : 0.f, gz = inside && !SIG ? dz * lse : 0.f;
    // the chosen slots' part: d on the slot, and (softmax of all) dw p_j on every expert
    float d = 0.f, dw = 0.f;
    if (b.dweight) {
      const bool has = e >= 0;
      if (a.renorm) {
        float m = group_all<LPT>(zc, OpMax());
        if (SIG) m = m < 0.f ? m : 0.f;
        float f = 0.f, q = 1.f;
        if (has) {
          if (!SIG) {
            f = exp_of(zc - m);
          } else {
            q = inv_of(1.f + exp_of(zc));  // 1 - sigmoid
            f = zc <= 0.f ? exp_of(zc - m) * q : inv_of(1.f + exp_of(-zc));
          }
        }
        const float sum = group_all<LPT>(f, OpAdd());
        const float n = has ? f / sum : 0.f;
        const float nv = group_all<LPT>(has ? n * v : 0.f, OpAdd());
        d = n * (v - nv) * q;
      } else if (SIG) {
        d = has ? v * inv_of(1.f + exp_of(-zc)) * inv_of(1.f + exp_of(zc)) : 0.f;
      } else {
        // (p of the chosen: log p = z - lse)
        d = has ? exp_of(zc - lse) * v : 0.f;
        dw = group_all<LPT>(d, OpAdd());
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g = gb * (w[j] - dot);
      if constexpr (SIG) g *= rest[j];
      o[j] = z[j] * (g + (gz - dw));
    }
    if (b.dweight) {
      // does a choice name an expert twice?
      if (e >= 0) row[e] = (float)i;
      wave_sync();
      const bool twice = e >= 0 && row[e] != (float)i;
      wave_sync();
#pragma unroll
      for (int j = 0; j < NV; ++j) row[c0 + j] = o[j];
      wave_sync();
      if (__ballot(twice)) {
        for (int q = 0; q < a.k; ++q) {
          if (i == q && e >= 0) row[e] += d;
          wave_sync();
        }
      } else {
        if (e >= 0) row[e] += d;
        wave_sync();
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) o[j] = row[c0 + j];
      wave_sync();
    }
    if (in) store_row<NV>(b.dlogits, BF16, b.vec_out != 0, t * b.ldd, c0, a.E, o);
  }
}

template <int LPT, int NV, bool BF16, bool SIG>
hipError_t balance_launch(const RouteArgs& a, const BalanceArgs& b, hipStream_t s) {
  constexpr int NT = balance_threads<NV>(), NR = NV == 8 ? NT / kWave : 1;
  LRM_LAUNCH(b.chunks, NT, (size_t)(NR + 1) * a.E * 4, s, k_balance<LPT, NV, BF16, SIG>)(a, b);
  return hipGetLastError();
}

template <int LPT, int NV, bool BF16, bool SIG>
hipError_t balance_bwd_launch(const RouteArgs& a, const BalanceBwdArgs& b0, hipStream_t s) {
  constexpr int tpb = (NV > 8 ? kWave : 256) / LPT;
  BalanceBwdArgs b = b0;
  // runs of at least four tokens a place where that leaves four blocks a CU
  const int64_t steps = ((int64_t)a.T + tpb - 1) / tpb;
  const int64_t per = steps > 4096 ? (steps + 4095) / 4096 : (steps > 1024 ? (steps + 1023) / 1024 : 1);
  b.chunk = per * tpb;
  LRM_LAUNCH((unsigned)((steps + per - 1) / per), NV > 8 ? kWave : 256, 0, s,
             k_balance_bwd<LPT, NV, BF16, SIG>)(a, b);
  return hipGetLastError();
}

}  // namespace

// Tokens of a chunk: about kBalanceChunks chunks, of at most 512 tokens (the sums
// over one are fp32).
int balance_chunk(int T) {
  const int64_t c = ((int64_t)T + kBalanceChunks - 1) / kBalanceChunks;
  return c < 32 ? 32 : (c > 512 ? 512 : (int)c);
}

hipError_t launch_balance(const RouteArgs& a, const BalanceArgs& b, hipStream_t s) {
  if (b.chunks > 0) {
    hipError_t e;
#define LRM_CALL4(L, V) \
  (a.bf16 ? (a.softmax ? balance_launch<L, V, true, false>(a, b, s)    \
                       : balance_launch<L, V, true, true>(a, b, s))    \
          : (a.softmax ? balance_launch<L, V, false, false>(a, b, s)   \
                       : balance_launch<L, V, false, true>(a, b, s)))
    auto run = [&]() -> hipError_t { LRM_ROUTE_DISPATCH(LRM_CALL4) };
#undef LRM_CALL4
    e = run();
    if (e != hipSuccess) return e;
  }
  if (a.E <= 64 && b.S == 1) {
    LRM_LAUNCH(1, 1024, 0, s, k_balance_join<64>)(a, b);
  } else if (a.E <= 128 && b.S == 1) {
    LRM_LAUNCH(1, 1024, 0, s, k_balance_join<128>)(a, b);
  } else if (a.E <= 256 && b.S == 1) {
    LRM_LAUNCH(1, 1024, 0, s, k_balance_join<256>)(a, b);
  } else {
    const int tiles = (a.E + kJoinCols - 1) / kJoinCols;
    LRM_LAUNCH(dim3(tiles, b.S < 65535 ? b.S : 65535), 1024, 0, s, k_balance_join<kJoinCols>)(a, b);
    LRM_LAUNCH(1, 1024, 0, s, k_balance_end)((int64_t)b.S * tiles, a.E, b);
  }
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const RouteArgs& a, const BalanceBwdArgs& b, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
#define LRM_CALL4(L, V) \
  (a.bf16 ? (a.softmax ? balance_bwd_launch<L, V, true, false>(a, b, s)    \
                       : balance_bwd_launch<L, V, true, true>(a, b, s))    \
          : (a.softmax ? balance_bwd_launch<L, V, false, false>(a, b, s)   \
                       : balance_bwd_launch<L, V, false, true>(a, b, s)))
  LRM_ROUTE_DISPATCH(LRM_CALL4)
#undef LRM_CALL4
}

}  // namespace lrm
