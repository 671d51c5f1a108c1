// Balance of the experts' load: with p_te the experts' shares of token t
//   balance = coef / S' sum over sequences s, experts e of a_se sum over t of p_te,
//   z = z_coef / n sum over t of (log sum_e exp z_te)^2
// (a_se = M f_se / n_s: see lrm.h) and their gradient
//   d balance / d z_tj = coef / S' p_tj (a_sj - sum_e p_te a_se) [(1 - sigma_j)],
//   d z / d z_tj = 2 z_coef / n log(sum) p_tj
// joined with that of the routing weights.  (The pages take a balanced router as
// given; its counts are those of the controller: page 1, bullet "Квоты до вычислений".)
//
// f_se being the counts' ratios, the loss needs no sums per expert: a token adds
// sum over e of c_se p_te, one number.  So where the counts are at hand the logits are
// read once and every block leaves three numbers; where they are not, a histogram of
// the choice comes first.  A block takes a run of tokens (a chunk); chunk c and
// sequence s meet in row c + s of the scratch: along the tokens one of the two
// grows at a time, so no two pairs share a row and chunks + S rows are enough,
// whatever the offsets (which only the GPU knows).  The last launch adds a
// sequence's rows with a wave, in fp64 and in order.
//
// Measured: 65536 tokens, 128 experts, bf16, counts at hand: 8 us for the 16.8 MB of
// logits and 3 to 4 for the last launch.  About 120 vector instructions for four
// tokens are 3.2 us and the memory's time is 3.3; without any arithmetic the pass takes as
// long: what remains are the launch and a chain of loads (the block's arguments, its
// counts, four rows at once).  16384 tokens, 256 experts, fp32, 13 sequences, from the
// choice: 2 us to clear, 6 to count, 11 for the pass, 5 to join.  256 tokens in one
// launch: 6 us.  Gradient with the routing weights': 65536 x 128 13 to 14.5 us for 38 MB
// (7.3 at a copy's rate; 10.8 without the weights' part, 11.1 without the stores); 15001
// x 161 in fp32, rows not aligned, 9.8.
#include "common.h"
#include "launch.h"
#include "route_util.h"

namespace lrm {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kCountOne = 16384;  // places of slots that one block counts
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ int64_t at_most(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t at_least(int64_t a, int64_t b) { return a > b ? a : b; }

template <typename V>
__device__ __forceinline__ V wave_add(V v) { return group_all<kWave>(v, OpAdd()); }

struct OpMaxF {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// Column of a lane's j-th value.  VEC: aligned rows of a multiple of NV elements,
// NV neighbours a lane, 16 bytes at a time; otherwise the lanes' columns alternate,
// so that single elements load and store whole lines together.
template <int LPT, int NV, bool VEC>
__device__ __forceinline__ int column(int i, int j) { return VEC ? i * NV + j : j * LPT + i; }

// (Loads of single elements are clamped, not guarded: behind a branch each would
// wait for the one before.)
template <int LPT, int NV, bool VEC, bool BF16>
struct Row {
  u32x4 q[VEC ? NV / (BF16 ? 8 : 4) : 1];
  uint32_t x[VEC ? 1 : NV];
  __device__ __forceinline__ void fetch(const void* row, int i, int E) {
    if constexpr (VEC) {
      const int c = i * NV < E ? i * NV : 0;
      if constexpr (BF16) {
        const u32x4* src = reinterpret_cast<const u32x4*>((const uint16_t*)row + c);
#pragma unroll
        for (int p = 0; p < NV / 8; ++p) q[p] = src[p];
      } else {
        const u32x4* src = reinterpret_cast<const u32x4*>((const float*)row + c);
#pragma unroll
        for (int p = 0; p < NV / 4; ++p) q[p] = src[p];
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = column<LPT, NV, VEC>(i, j), cc = c < E ? c : E - 1;
        x[j] = BF16 ? ((const uint16_t*)row)[cc] : ((const uint32_t*)row)[cc];
      }
    }
  }
  // (columns at or past E: -inf)
  __device__ __forceinline__ void values(int i, int E, float (&z)[NV]) const {
    const float none = -__builtin_inff();
    if constexpr (VEC) {
      if constexpr (BF16) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const uint32_t w = q[j / 8][(j & 7) >> 1];
          z[j] = j & 1 ? bf16_hi(w) : bf16_lo(w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) z[j] = __uint_as_float(q[j / 4][j & 3]);
      }
      if (E == LPT * NV) return;
#pragma unroll
      for (int j = 0; j < NV; ++j) z[j] = i * NV < E ? z[j] : none;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        z[j] = column<LPT, NV, VEC>(i, j) < E ? __uint_as_float(BF16 ? x[j] << 16 : x[j]) : none;
    }
  }
};

// A bit for every column of the lane that takes part.
template <int LPT, int NV, bool VEC>
__device__ __forceinline__ uint64_t open_bits(const uint8_t* mask, int i, int E) {
  if (!mask) return ~0ull;
  uint64_t bits = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column<LPT, NV, VEC>(i, j);
    bits |= (uint64_t)(mask[c < E ? c : 0] != 0 ? 1u : 0u) << j;
  }
  return bits;
}

// The lane's entries of a row of E numbers (0 past it).
template <int LPT, int NV, bool VEC, typename V>
__device__ __forceinline__ void numbers_row(const V* row, int i, int E, float (&w)[NV]) {
  V x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column<LPT, NV, VEC>(i, j);
    x[j] = row[c < E ? c : 0];
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) w[j] = column<LPT, NV, VEC>(i, j) < E ? (float)x[j] : 0.f;
}

// A lane's share of a token: the exps f of its eligible logits z (masked: -inf) in
// place of them, with the row's largest taken out, inv one over their sum (0: no
// eligible expert), lse its log.  One rounding in the exponent: f is good to 2^-24
// of the logit's distance from the largest.  SIG: f = sigma, rest = 1 - sigma.
template <int LPT, int NV, bool SIG, bool GRAD>
__device__ __forceinline__ bool shares(float (&z)[NV], float (&rest)[GRAD && SIG ? NV : 1], bool want_lse,
                                       float* inv, float* lse) {
  float top = -__builtin_inff(), sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) top = fmaxf(top, z[j]);
  top = group_all<LPT>(top, OpMaxF());
  const bool live = top > -__builtin_inff();
  if constexpr (SIG) {
    // sigma times e^-m, m = top where every score would be tiny, so that the
    // sum does not underflow
    const float m = live && top < -60.f ? top : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float q = __builtin_amdgcn_exp2f(fabsf(z[j]) * -kLog2e), r = inv_of(1.f + q);
      const float up = m < 0.f ? __builtin_amdgcn_exp2f((z[j] - m) * kLog2e) : q;
      if constexpr (GRAD) rest[j] = z[j] > 0.f ? q * r : r;
      z[j] = z[j] > 0.f ? r : up * r;  // (0 for -inf)
      sum += z[j];
    }
    sum = group_all<LPT>(sum, OpAdd());
    *inv = live ? 1.f / sum : 0.f;
    *lse = 0.f;
  } else {
    const float m = live ? top * kLog2e : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = __builtin_amdgcn_exp2f(fmaf(z[j], kLog2e, -m));
      sum += z[j];
    }
    sum = group_all<LPT>(sum, OpAdd());
    *inv = live ? inv_of(sum) : 0.f;  // (1 .. 4096)
    *lse = want_lse && live ? fmaf(__builtin_amdgcn_logf(sum), kLn2, top) : 0.f;
  }
  return live;
}

// Largest s in [0, S) with seq[s] <= t, or 0 (t the same in a whole wave): 64 places
// are looked at at a time.
__device__ __forceinline__ int sequence_at(const int32_t* seq, int S, int64_t t) {
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + kWave - 1) / kWave, at = lane_id() * step;
    const bool before = at < n && seq[lo + (at < n ? at : 0)] <= t;
    const int c = __popcll(__ballot(before));
    const int k = c > 0 ? (c - 1) * step : 0;
    lo += k;
    n = n - k < step ? n - k : step;
  }
  return lo;
}

// The lane's values into the row that starts at element `at`.
template <int LPT, int NV, bool VEC, bool BF16>
__device__ __forceinline__ void store_row(void* out, bool vec, int64_t at, int i, int E,
                                          const float (&o)[NV]) {
  if (VEC && vec) {
    const int c = i * NV;
    if (c >= E) return;
    if constexpr (BF16) {
      u32x4* dst = reinterpret_cast<u32x4*>((uint16_t*)out + at + c);
#pragma unroll
      for (int q = 0; q < NV / 8; ++q)
        dst[q] = u32x4{cvt_pk_bf16(o[8 * q], o[8 * q + 1]), cvt_pk_bf16(o[8 * q + 2], o[8 * q + 3]),
                       cvt_pk_bf16(o[8 * q + 4], o[8 * q + 5]), cvt_pk_bf16(o[8 * q + 6], o[8 * q + 7])};
    } else {
      f32x4* dst = reinterpret_cast<f32x4*>((float*)out + at + c);
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) dst[q] = f32x4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]};
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column<LPT, NV, VEC>(i, j);
    if (c < E) {
      if constexpr (BF16) ((uint16_t*)out)[at + c] = (uint16_t)(cvt_pk_bf16(o[j], o[j]));
      else ((float*)out)[at + c] = o[j];
    }
  }
}

// -------------------------------------------------------------- histogram
// Slots of tokens [t0, t1) into hist (LDS, clear): kk places a token, the power of 2
// from k on, four tokens a place in flight.
__device__ __forceinline__ void count_slots(const RouteArgs& a, const int32_t* expert, int64_t t0,
                                            int64_t t1, int nt, int log_kk, int* hist) {
  const int i = threadIdx.x & ((1 << log_kk) - 1), step = nt >> log_kk;
  if (i >= a.k) return;
  for (int64_t t = t0 + (threadIdx.x >> log_kk); t < t1; t += 4 * step) {
    int e[4], on[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t tq = t + q * step < t1 ? t + q * step : t;
      e[q] = expert[tq * a.k + i];
      on[q] = a.token_mask ? a.token_mask[tq] : 1;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool named = e[q] >= 0 && e[q] < a.E;
      const int open = a.expert_mask ? a.expert_mask[named ? e[q] : 0] : 1;
      if (t + q * step < t1 && named && on[q] && open) atomicAdd(&hist[e[q]], 1);
    }
  }
}

// Chunks of tokens; integer sums, so their order does not show.  ONE: a single block of a
// single sequence, which writes its counts; otherwise out is clear before.
template <bool ONE>
__global__ __launch_bounds__(ONE ? 1024 : kThreads) void k_balance_count(RouteArgs a, BalanceArgs b,
                                                                         int64_t chunk, int log_kk,
                                                                         int32_t* out) {
  LRM_DYN_SHARED(int, hist);  // [E]
  constexpr int NT = ONE ? 1024 : kThreads;
  const int64_t c0 = (int64_t)blockIdx.x * chunk, c1 = at_most(c0 + chunk, a.T);
  for (int e = threadIdx.x; e < a.E; e += NT) hist[e] = 0;
  for (int s = b.seq ? sequence_at(b.seq, b.S, c0) : 0; s < b.S; ++s) {
    int64_t t0 = c0, t1 = c1;
    if (b.seq) {
      t0 = at_least(c0, b.seq[s]);
      t1 = at_most(c1, b.seq[s + 1]);
      if (ONE) t1 = at_least(t0, t1);
      if (!ONE && b.seq[s] >= c1) break;
      if (!ONE && t0 >= t1) continue;
    }
    __syncthreads();
    count_slots(a, b.expert, t0, t1, NT, log_kk, hist);
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += NT) {
      if constexpr (ONE) out[(int64_t)s * a.E + e] = hist[e];
      else if (hist[e]) atomicAdd(&out[(int64_t)s * a.E + e], hist[e]);
      hist[e] = 0;
    }
  }
}

// ------------------------------------------------------------------- loss
// What a thread adds up over its tokens of [t0, t1), one at least: w the counts of
// its experts.  (fp32 over a chunk's tokens and the lanes of a wave: at most 16 and 6
// additions; fp64 from there.)
struct Sums {
  float dot, lse2;
  int live;
};
__device__ __forceinline__ BalanceRow wave_row(const Sums& v) {
  return BalanceRow{(double)wave_add(v.dot), (double)wave_add(v.lse2), wave_add(v.live), 0};
}
template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
__device__ __forceinline__ Sums pass(const RouteArgs& a, bool z_wanted, int64_t t0, int64_t t1, int tpb,
                                     uint64_t bits, const int32_t* counts) {
  const int i = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
  const bool masked = a.expert_mask || a.token_mask;
  // the place of the thread's next row (tokens behind the last one: the last place again)
  const int64_t stride = (int64_t)tpb * a.ld * (BF16 ? 2 : 4);
  const int n = (int)(t1 - t0);
  int ahead = slot;
  const char* next = (const char*)a.logits + (t0 + (slot < n ? slot : 0)) * a.ld * (BF16 ? 2 : 4);
  auto step = [&] {
    ahead += tpb;
    next += ahead < n ? stride : 0;
  };
  Sums s{0.f, 0.f, 0};
  // DEEP rows of a place on their way at once: a chunk is short, its time the loads' latency
  constexpr int DEEP = NV == 8 ? 4 : 1;
  Row<LPT, NV, VEC, BF16> raw[DEEP];
#pragma unroll
  for (int q = 0; q < DEEP; ++q) {
    raw[q].fetch(next, i, a.E);
    step();
  }
  float w[NV];
  numbers_row<LPT, NV, VEC>(counts, i, a.E, w);
  for (int r = 0; r < n; r += DEEP * tpb) {
#pragma unroll
    for (int q = 0; q < DEEP; ++q) {
      const int t = r + slot + q * tpb;
      const bool in = t < n;
      float z[NV], rest[1], inv, lse, dot = 0.f;
      raw[q].values(i, a.E, z);
      if (r + (q + DEEP) * tpb < n) {
        raw[q].fetch(next, i, a.E);
        step();
      }
      if (q > 0 && r + q * tpb >= n) break;
      if (masked) mask_row<NV>(in && (a.token_mask ? a.token_mask[t0 + (in ? t : 0)] != 0 : true) ? bits : 0, z);
      const bool live = shares<LPT, NV, SIG, false>(z, rest, z_wanted, &inv, &lse) && in;
#pragma unroll
      for (int j = 0; j < NV; ++j) dot = fmaf(z[j], w[j], dot);
      s.dot = fmaf(dot, in ? inv : 0.f, s.dot);
      const bool one = live && i == 0;
      s.live += one ? 1 : 0;
      lse = one ? lse : 0.f;
      s.lse2 = fmaf(lse, lse, s.lse2);
    }
  }
  return s;
}

template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
__global__ __launch_bounds__(kThreads) void k_balance(RouteArgs a, BalanceArgs b) {
  __shared__ BalanceRow part[kThreads / kWave];
  const int i = threadIdx.x & (LPT - 1);
  const uint64_t bits = open_bits<LPT, NV, VEC>(a.expert_mask, i, a.E);
  const int64_t k0 = (int64_t)blockIdx.x * b.chunk;
  const int64_t k1 = at_most(k0 + b.chunk, a.T);
  for (int s = b.seq ? sequence_at(b.seq, b.S, k0) : 0; s < b.S; ++s) {
    int64_t t0 = k0, t1 = k1;
    if (b.seq) {
      t0 = at_least(k0, b.seq[s]);
      t1 = at_most(k1, b.seq[s + 1]);
      if (b.seq[s] >= k1) break;
      if (t0 >= t1) continue;
    }
    const BalanceRow v = wave_row(pass<LPT, NV, SIG, VEC, BF16>(
        a, b.z_coef != 0.f, t0, t1, kThreads / LPT, bits, b.counts + (int64_t)s * a.E));
    __syncthreads();  // (part of the sequence before has been read)
    if (lane_id() == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      BalanceRow x = part[0];
      for (int q = 1; q < kThreads / kWave; ++q) {
        x.dot += part[q].dot;
        x.lse2 += part[q].lse2;
        x.live += part[q].live;
      }
      b.rows[(int64_t)blockIdx.x + s] = x;
    }
  }
}

// Over all sequences: sum of M dot_s / (filled_s n_s), of log^2, of n_s, and how many have tokens.
struct Batch {
  double bal, lse2, live, full;
};
__device__ __forceinline__ void balance_end(const BalanceArgs& b, int E, const Batch& v) {
  const double fb = (double)b.coef / (v.full > 0.0 ? v.full : 1.0);
  const double fz = (double)b.z_coef / (v.live > 0.0 ? v.live : 1.0);
  b.loss[0] = (float)(fb * v.bal);
  b.loss[1] = (float)(fz * v.lse2);
  b.saved[(int64_t)b.S * E] = (float)fb;
  b.saved[(int64_t)b.S * E + 1] = (float)(2.0 * fz);
}

// One wave for a sequence with these sums and counts: its part of saved and of the
// batch (the same in every lane).
__device__ __forceinline__ void sequence_end(const RouteArgs& a, const BalanceArgs& b, int s, double experts,
                                             const BalanceRow& v, const int32_t* counts, Batch* out) {
  double filled = 0.0;
  for (int e = lane_id(); e < a.E; e += 4 * kWave) {
    int n[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) n[q] = counts[e + q * kWave < a.E ? e + q * kWave : e];
#pragma unroll
    for (int q = 0; q < 4; ++q) filled += e + q * kWave < a.E ? (double)n[q] : 0.0;
  }
  filled = wave_add(filled);
  const double f = filled > 0.0 && v.live > 0 ? experts / (filled * (double)v.live) : 0.0;
  for (int e = lane_id(); e < a.E; e += kWave) {
    const int n = counts[e];
    b.saved[(int64_t)s * a.E + e] = (float)(f * (double)n);
    if (b.counts_out) b.counts_out[(int64_t)s * a.E + e] = n;
  }
  out->bal += f * v.dot;
  out->lse2 += v.lse2;
  out->live += (double)v.live;
  out->full += v.live > 0 ? 1.0 : 0.0;
}
__device__ __forceinline__ double open_experts(const RouteArgs& a) {
  if (!a.expert_mask) return (double)a.E;
  int n = 0;
  for (int e = lane_id(); e < a.E; e += kWave) n += a.expert_mask[e] ? 1 : 0;
  return (double)wave_add(n);
}

// A sequence at a time for every wave, or (ALL) one sequence for the block; a single
// block finishes the batch too.
template <bool ALL>
__global__ __launch_bounds__(1024) void k_balance_join(RouteArgs a, BalanceArgs b) {
  __shared__ Batch part[16];
  __shared__ BalanceRow rows[16];
  const int w = threadIdx.x >> 6, l = lane_id();
  const int64_t waves = (int64_t)gridDim.x * 16;
  const double experts = open_experts(a);
  constexpr int step = ALL ? 1024 : kWave;
  Batch mine{0.0, 0.0, 0.0, 0.0};
  for (int64_t s = ALL ? 0 : (int64_t)blockIdx.x * 16 + w; s < b.S; s += waves) {
    // the rows of this sequence (offsets held to the tokens)
    int64_t t0 = 0, t1 = a.T;
    if (b.seq) {
      t0 = at_least(b.seq[s], 0);
      t1 = at_most(b.seq[s + 1], a.T);
    }
    const int64_t r0 = t0 < t1 ? t0 / b.chunk + s : 0;
    const int64_t r1 = t0 < t1 ? (t1 - 1) / b.chunk + s + 1 : 0;
    BalanceRow v{0.0, 0.0, 0, 0};
    for (int64_t rr = r0 + (ALL ? threadIdx.x : l); rr < r1; rr += 4 * step) {
      BalanceRow x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = b.rows[rr + q * step < r1 ? rr + q * step : rr];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool ok = rr + q * step < r1;
        v.dot += ok ? x[q].dot : 0.0;
        v.lse2 += ok ? x[q].lse2 : 0.0;
        v.live += ok ? x[q].live : 0;
      }
    }
    v = BalanceRow{wave_add(v.dot), wave_add(v.lse2), wave_add(v.live), 0};
    if constexpr (ALL) {
      if (l == 0) rows[w] = v;
      __syncthreads();
      if (w > 0) return;
      v = rows[0];
      for (int q = 1; q < 16; ++q) {
        v.dot += rows[q].dot;
        v.lse2 += rows[q].lse2;
        v.live += rows[q].live;
      }
    }
    sequence_end(a, b, (int)s, experts, v, b.counts + s * a.E, &mine);
  }
  if constexpr (ALL) {
    if (l == 0) balance_end(b, a.E, mine);
    return;
  }
  if (l == 0) part[w] = mine;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int q = 1; q < 16; ++q) {
    mine.bal += part[q].bal;
    mine.lse2 += part[q].lse2;
    mine.live += part[q].live;
    mine.full += part[q].full;
  }
  if (gridDim.x == 1) {
    balance_end(b, a.E, mine);
  } else {
    double* o = b.blocks + (int64_t)blockIdx.x * 4;
    o[0] = mine.bal; o[1] = mine.lse2; o[2] = mine.live; o[3] = mine.full;
  }
}

// The blocks of the join, in order.
__global__ __launch_bounds__(64) void k_balance_end(int n, int E, BalanceArgs b) {
  Batch v{0.0, 0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < n; i += kWave) {
    v.bal += b.blocks[4 * i];
    v.lse2 += b.blocks[4 * i + 1];
    v.live += b.blocks[4 * i + 2];
    v.full += b.blocks[4 * i + 3];
  }
  v.bal = wave_add(v.bal);
  v.lse2 = wave_add(v.lse2);
  v.live = wave_add(v.live);
  v.full = wave_add(v.full);
  if (threadIdx.x == 0) balance_end(b, E, v);
}

// Few tokens, one sequence: everything in one launch of one block.
template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
__global__ __launch_bounds__(1024) void k_balance_one(RouteArgs a, BalanceArgs b, int log_kk) {
  LRM_DYN_SHARED(int, hist);  // [E]
  __shared__ BalanceRow part[16];
  const int i = threadIdx.x & (LPT - 1);
  const int64_t t0 = b.seq ? at_least(b.seq[0], 0) : 0, t1 = b.seq ? at_most(b.seq[1], a.T) : a.T;
  for (int e = threadIdx.x; e < a.E; e += 1024) hist[e] = b.counts ? b.counts[e] : 0;
  __syncthreads();
  if (!b.counts) count_slots(a, b.expert, t0, t1, 1024, log_kk, hist);
  __syncthreads();
  BalanceRow v{0.0, 0.0, 0, 0};
  if (t0 < t1)
    v = wave_row(pass<LPT, NV, SIG, VEC, BF16>(a, b.z_coef != 0.f, t0, t1, 1024 / LPT,
                                               open_bits<LPT, NV, VEC>(a.expert_mask, i, a.E), hist));
  if (lane_id() == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x >= kWave) return;
  BalanceRow x = part[0];
  for (int q = 1; q < 16; ++q) {
    x.dot += part[q].dot;
    x.lse2 += part[q].lse2;
    x.live += part[q].live;
  }
  Batch all{0.0, 0.0, 0.0, 0.0};
  sequence_end(a, b, 0, open_experts(a), x, hist, &all);
  if (threadIdx.x == 0) balance_end(b, a.E, all);
}

// --------------------------------------------------------------- gradient
// A block takes a run of tokens; the lanes of a token hold a whole row of p and
// of a.  The chosen slots' part is added in LDS, all slots of a token at once; slot
// after slot where a choice names an expert twice.
template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
__global__ __launch_bounds__(NV > 8 ? kWave : kThreads) void k_balance_bwd(RouteArgs a, BalanceBwdArgs b) {
  constexpr int NT = NV > 8 ? kWave : kThreads, tpb = NT / LPT;
  alignas(16) __shared__ float lds[NT * NV];
  const int i = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
  const bool masked = a.expert_mask || a.token_mask;
  const uint64_t bits = open_bits<LPT, NV, VEC>(a.expert_mask, i, a.E);
  float* row = lds + slot * LPT * NV;
  const float db = (b.dloss ? b.dloss[0] : 1.f) * b.saved[(int64_t)b.S * a.E];
  const float dz = (b.dloss ? b.dloss[1] : 1.f) * b.saved[(int64_t)b.S * a.E + 1];
  bool inside = true;
  const int64_t r0 = (int64_t)blockIdx.x * b.chunk;
  const int64_t r1 = at_most(r0 + b.chunk, a.T);
  int at = 0;        // the sequence of the token, or of the last one before it
  if (b.seq) at = sequence_at(b.seq, b.S, r0);
  // a token's row and slots are on their way while the one before it is worked on
  // (behind the last token: the last place again)
  const int n = (int)(r1 - r0);
  const int64_t t0 = r0 + (slot < n ? slot : 0);
  const char* next = (const char*)a.logits + t0 * a.ld * (BF16 ? 2 : 4);
  int64_t next_slot = t0 * a.k + (i < a.k ? i : 0);
  int64_t out = (r0 + slot) * b.ldd;
  Row<LPT, NV, VEC, BF16> raw;
  int e1 = -1;
  float v1 = 0.f;
  raw.fetch(next, i, a.E);
  if (b.dweight) {
    e1 = b.expert[next_slot];
    v1 = b.dweight[next_slot];
  }
  float w[NV];
  int s = at;        // the sequence whose row is in w
  numbers_row<LPT, NV, VEC>(b.saved + (int64_t)s * a.E, i, a.E, w);
  for (int r = slot; r - slot < n; r += tpb, out += tpb * b.ldd) {
    const int64_t t = r0 + r;
    const bool in = r < n;
    const bool on = in && (a.token_mask ? a.token_mask[in ? t : r0] != 0 : true);
    float z[NV], o[NV], rest[SIG ? NV : 1], inv, lse;
    const int e0 = e1;
    const float v0 = v1;
    raw.values(i, a.E, z);
    if (r - slot + tpb < n) {
      const bool more = r + tpb < n;
      next += more ? (int64_t)tpb * a.ld * (BF16 ? 2 : 4) : 0;
      next_slot += more ? tpb * a.k : 0;
      raw.fetch(next, i, a.E);
      if (b.dweight) {
        e1 = b.expert[next_slot];
        v1 = b.dweight[next_slot];
      }
    }
    if (masked) mask_row<NV>(on ? bits : 0, z);
    int e = -1;
    float zc = -__builtin_inff();
    bool twice = false;
    if (b.dweight) {
      // the chosen logits (masked ones: -inf), and whether a choice names an expert twice
#pragma unroll
      for (int j = 0; j < NV; ++j) row[column<LPT, NV, VEC>(i, j)] = z[j];
      wave_sync();
      const bool named = on && i < a.k && e0 >= 0 && e0 < a.E;
      zc = row[named ? e0 : 0];
      const bool has = named && zc != -__builtin_inff();
      e = has ? e0 : -1;
      zc = has ? zc : -__builtin_inff();
      wave_sync();
      if (has) row[e] = (float)i;
      wave_sync();
      twice = has && row[e] != (float)i;
      wave_sync();
    }
    if (b.seq) {
      while (at + 1 < b.S && b.seq[at + 1] <= t) ++at;
      inside = b.seq[at] <= t && t < b.seq[at + 1];
    }
    if (at != s) {
      s = at;
      numbers_row<LPT, NV, VEC>(b.saved + (int64_t)s * a.E, i, a.E, w);
    }
    shares<LPT, NV, SIG, true>(z, rest, true, &inv, &lse);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) dot = fmaf(z[j], w[j], dot);
    dot = group_all<LPT>(dot, OpAdd()) * inv;
    // the chosen slots' part: d on the slot, and (softmax of all) dw p_j on every expert
    float d = 0.f, dw = 0.f;
    if (b.dweight) {
      const bool has = e >= 0;
      const float v = has ? a.scale * v0 : 0.f;
      if (a.renorm) {
        float m = group_all<LPT>(zc, OpMaxF());
        if (SIG) m = m < 0.f ? m : 0.f;
        float f = 0.f, q = 1.f;
        if (!SIG) {
          f = has ? __builtin_amdgcn_exp2f((zc - m) * kLog2e) : 0.f;
        } else if (has) {
          q = inv_of(1.f + exp_of(zc));  // 1 - sigmoid
          f = zc <= 0.f ? exp_of(zc - m) * q : inv_of(1.f + exp_of(-zc));
        }
        const float sum = group_all<LPT>(f, OpAdd());
        const float n = has ? f * inv_of(sum) : 0.f;  // (sum is 1/2 at least)
        const float nv = group_all<LPT>(n * v, OpAdd());
        d = n * (v - nv) * q;
      } else if (SIG) {
        d = has ? v * inv_of(1.f + exp_of(-zc)) * inv_of(1.f + exp_of(zc)) : 0.f;
      } else {
        // (p of the chosen: log p = z - lse)
        d = has ? __builtin_amdgcn_exp2f((zc - lse) * kLog2e) * v : 0.f;
        dw = group_all<LPT>(d, OpAdd());
      }
    }
    // p_j (gb (w_j - dot) [rest_j] + gz lse - dw)
    const float gb = inside ? db : 0.f, gz = (inside && !SIG ? dz * lse : 0.f) - dw;
    const float pb = gb * inv, pz = (SIG ? 0.f : fmaf(-gb, dot, gz)) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      o[j] = SIG ? z[j] * (pb * (w[j] - dot) * rest[j]) : z[j] * fmaf(pb, w[j], pz);
    if (b.seq) {  // (the shares of a token of no sequence may be no numbers)
#pragma unroll
      for (int j = 0; j < NV; ++j) o[j] = inside || dw != 0.f ? o[j] : 0.f;
    }
    if (b.dweight) {
#pragma unroll
      for (int j = 0; j < NV; ++j) row[column<LPT, NV, VEC>(i, j)] = o[j];
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
      for (int j = 0; j < NV; ++j) o[j] = row[column<LPT, NV, VEC>(i, j)];
      wave_sync();
    }
    if (in) store_row<LPT, NV, VEC, BF16>(b.dlogits, b.vec_out != 0, out, i, a.E, o);
  }
}

int log2_up(int k) {
  int l = 0;
  while ((1 << l) < k) ++l;
  return l;
}

template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
hipError_t balance_launch(const RouteArgs& a, const BalanceArgs& b, hipStream_t s) {
  if constexpr (NV == 8) {
    if (balance_in_one(a.T, a.E, a.k, b.S, b.counts != nullptr)) {
      LRM_LAUNCH(1, 1024, (size_t)a.E * 4, s, k_balance_one<LPT, NV, SIG, VEC, BF16>)(a, b, log2_up(a.k));
      return hipGetLastError();
    }
  }
  LRM_LAUNCH(b.chunks, kThreads, 0, s, k_balance<LPT, NV, SIG, VEC, BF16>)(a, b);
  return hipGetLastError();
}

template <int LPT, int NV, bool SIG, bool VEC, bool BF16>
hipError_t balance_bwd_launch(const RouteArgs& a, const BalanceBwdArgs& b0, hipStream_t s) {
  constexpr int NT = NV > 8 ? kWave : kThreads, tpb = NT / LPT;
  BalanceBwdArgs b = b0;
  // The start of a block weighs as much as a few steps, and so do idle places at the end:
  // 1024, 2048 and 4096 blocks take 13.2, 14.5 and 19.4 us (65536 x 128, 4096 steps), 34.1,
  // 33.5 and 35.3 (65536 x 256 fp32, 8192 steps), 30.3, 27.4 and 26.2 (262144 x 64, 16384 steps).
  const int64_t steps = ((int64_t)a.T + tpb - 1) / tpb;
  const int64_t most = steps <= 4096 ? 1024 : (steps <= 8192 ? 2048 : 4096);
  const int64_t per = (steps + most - 1) / most;
  b.chunk = per * tpb;
  LRM_LAUNCH((unsigned)((steps + per - 1) / per), NT, 0, s, k_balance_bwd<LPT, NV, SIG, VEC, BF16>)(a, b);
  return hipGetLastError();
}

// (whole lanes of aligned elements: rows of a multiple of a lane's V)
#define LRM_BALANCE_TYPE(F, L, V, VEC)                                                         \
  (a.bf16 ? (a.softmax ? F<L, V, false, VEC, true>(a, b, s) : F<L, V, true, VEC, true>(a, b, s)) \
          : (a.softmax ? F<L, V, false, VEC, false>(a, b, s) : F<L, V, true, VEC, false>(a, b, s)))
#define LRM_BALANCE_CALL(F, L, V) \
  (a.vec && a.E % V == 0 ? LRM_BALANCE_TYPE(F, L, V, true) : LRM_BALANCE_TYPE(F, L, V, false))

}  // namespace

// Places of a block of 256 threads: tokens that it holds at once (LRM_ROUTE_DISPATCH).
int balance_places(int E, int k) { return k <= 16 && E <= 128 ? 16 : (k <= 32 && E <= 256 ? 8 : 4); }

// Tokens of a chunk: four of a place and more in about 512 chunks, 16 at most (whose
// sums are fp32).  512, 1024 and 2048 chunks: 65536 x 128 11.2, 11.9 and 11.8 us, 8192 x
// 256 in nine sequences 17.1, 17.5 and 17.4.
int balance_chunk(int T, int E, int k) {
  const int places = balance_places(E, k);
  const int64_t per = (((int64_t)T + 511) / 512 + places - 1) / places;
  return places * (int)(per < 4 ? 4 : (per > 16 ? 16 : per));
}

// One block of 1024 threads for all: few tokens, but some, of one sequence (up to 512
// experts); up to 8 of a place, 16 where the counts would take two more launches.  One
// block against several, counts at hand: 512 x 128 8.1 and 11.1 us, 1024 x 16 13.7 and
// 11.2; from the choice: 512 x 128 9.0 and 17.2, 1024 x 16 14.5 and 17.1, 4096 x 16 47
// and 17.3.
bool balance_in_one(int T, int E, int k, int S, bool counts) {
  return S == 1 && T > 0 && E <= 512 && T <= 4 * balance_places(E, k) * (counts ? 8 : 16);
}

// Blocks of the join: 16 sequences each, 1024 at most.
int balance_join_blocks(int S) { return S <= 64 ? 1 : (S < 16384 ? (S + 15) / 16 : 1024); }

hipError_t launch_balance(const RouteArgs& a, const BalanceArgs& b0, hipStream_t s) {
  BalanceArgs b = b0;
  const bool one = balance_in_one(a.T, a.E, a.k, b.S, b.counts != nullptr);
  if (!one && !b.counts) {
    const int log_kk = log2_up(a.k);
    if (b.S == 1 && a.T > 0 && (int64_t)a.T << log_kk <= kCountOne) {
      LRM_LAUNCH(1, 1024, (size_t)a.E * 4, s, k_balance_count<true>)(a, b, a.T, log_kk, b.cnt);
    } else {
      // about 1024 slots a block, more for over half a million
      int64_t chunk = 1024 >> log_kk;
      if (a.T / chunk > 512) chunk = (a.T / 512 + chunk - 1) / chunk * chunk;
      const hipError_t e =
          launch_fill_u32(reinterpret_cast<uint32_t*>(b.cnt), 0u, (int64_t)b.S * a.E, s);
      if (e != hipSuccess) return e;
      if (a.T > 0)
        LRM_LAUNCH((unsigned)((a.T + chunk - 1) / chunk), kThreads, (size_t)a.E * 4, s,
                   k_balance_count<false>)(a, b, chunk, log_kk, b.cnt);
    }
    b.counts = b.cnt;
  }
  if (one || b.chunks > 0) {
#define LRM_CALL2(L, V) LRM_BALANCE_CALL(balance_launch, L, V)
    auto run = [&]() -> hipError_t { LRM_ROUTE_DISPATCH(LRM_CALL2) };
#undef LRM_CALL2
    const hipError_t e = run();
    if (e != hipSuccess || one) return e;
  }
  const int blocks = balance_join_blocks(b.S);
  if (b.S == 1)
    LRM_LAUNCH(1, 1024, 0, s, k_balance_join<true>)(a, b);
  else
    LRM_LAUNCH(blocks, 1024, 0, s, k_balance_join<false>)(a, b);
  if (blocks > 1) LRM_LAUNCH(1, 64, 0, s, k_balance_end)(blocks, a.E, b);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const RouteArgs& a, const BalanceBwdArgs& b, hipStream_t s) {
  if (a.T <= 0) return hipSuccess;
#define LRM_CALL2(L, V) LRM_BALANCE_CALL(balance_bwd_launch, L, V)
  LRM_ROUTE_DISPATCH(LRM_CALL2)
#undef LRM_CALL2
}

}  // namespace lrm
