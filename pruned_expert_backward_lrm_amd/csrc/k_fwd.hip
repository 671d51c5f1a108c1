// The experts' forward pass: grouped products over the packed pairs of each
// expert with their epilogues, and the join of the pairs' rows per token.
// (LRMoE keeps the forward complete: page 1, section "Что делает LRMoE: полный
// прямой проход, обрезанный обратный".)  For packed row m (pair p = kept[m],
// expert e):
//   GLU:  a = W0_e x, b = W1_e x  -> A[p], B[p] (wanted or not), H[m] = silu(a) b
//   else: z = W0_e x + bias_e     -> Z[p], y = act(z) -> Y[p]
//   join: out[t] = R[t] + sum over the pairs p of t of w_p y_p
// x is row token[p] or p of X, or row m of the packed H.
#include <cstdlib>
#include <type_traits>

#include "common.h"
#include "gemm_util.h"
#include "launch.h"

namespace lrm {

namespace {

__device__ __forceinline__ float act_rt(int act, float z) {
  switch (act) {
    case kActRelu: return act_of<kActRelu, false>(z);
    case kActGelu: return act_of<kActGelu, false>(z);
    case kActSilu: return act_of<kActSilu, false>(z);
  }
  return z;
}

// y between the down product and the join takes 24 bits: its bf16 rounding
// (which is Yp where the caller wants it) and the next 8 bits, a signed byte of
// the difference of the bit patterns.  With bf16 alone Y would carry two
// roundings of half the terms' size on top of its own.  A value half-way between
// two bf16 values goes away from zero, so that the byte is bits 8 .. 15
// themselves, read as signed.  The join adds half of the last place: 2^-16 of
// the value at most.  An infinity (a sum past fp32) stays one: no finite value
// leaves its 16 bits above a byte of zero.  A NaN stays one, since its low 16 bits
// are zero: they come from bf16 inputs or the hardware's own.
__device__ __forceinline__ uint32_t away_bf16x2(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi) + 0x8000u, __float_as_uint(lo) + 0x8000u, 0x07060302u);
}
// bits 8 .. 15 of four values
__device__ __forceinline__ uint32_t next_bytes(f32x4 y) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(y[1]), __float_as_uint(y[0]), 0x00000501u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(y[3]), __float_as_uint(y[2]), 0x00000501u);
  return (lo & 0xffffu) | hi << 16;
}
// INF: an infinity stays one (otherwise it becomes a NaN)
template <bool INF>
__device__ __forceinline__ float join_bits(uint32_t hi16, int lo8) {
  const uint32_t u = (hi16 << 16) + (uint32_t)(lo8 * 256);
  return __uint_as_float(INF && (u << 1) == 0xff000000u ? u : u + 128u);
}

// act of a wave's row of fragments; one loop over registers for each kind
template <int FO, bool FAST>
__device__ __forceinline__ void act_rows(int act, f32x4 (&u)[FO]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int j = 0; j < FO; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) u[j][q] = f(u[j][q]);
  };
  if (act == kActRelu)
    all([](float z) { return act_of<kActRelu, FAST>(z); });
  else if (act == kActGelu)
    all([](float z) { return act_of<kActGelu, FAST>(z); });
  else
    all([](float z) { return act_of<kActSilu, FAST>(z); });
}

// silu for results that are rounded to bf16: the hardware's exp2 and reciprocal
__device__ __forceinline__ float silu_fast(float a) {
  return a * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(a * -1.44269504088896341f));
}

// V consecutive columns of a row, V = 8 in bf16 and 4 in fp32 (16 bytes).
template <bool BF16>
struct Vec {
  static constexpr int V = BF16 ? 8 : 4;
  float v[V];
  __device__ __forceinline__ static Vec load(const void* row, int64_t at) {
    Vec r;
    if constexpr (BF16) {
      const u32x4 x = *reinterpret_cast<const u32x4*>((const uint16_t*)row + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.v[2 * j] = bf16_lo(x[j]);
        r.v[2 * j + 1] = bf16_hi(x[j]);
      }
    } else {
      const f32x4 x = *reinterpret_cast<const f32x4*>((const float*)row + at);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.v[j] = x[j];
    }
    return r;
  }
  __device__ __forceinline__ void store(void* row, int64_t at) const {
    if constexpr (BF16)
      *reinterpret_cast<u32x4*>((uint16_t*)row + at) =
          u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                pack_bf16x2(v[6], v[7])};
    else
      *reinterpret_cast<f32x4*>((float*)row + at) = f32x4{v[0], v[1], v[2], v[3]};
  }
};

// fp32: the outputs of V consecutive columns c .. (c < n, n a multiple of V) of
// packed row m, pair p: u = W0 x, v = W1 x (GLU).
template <bool BF16, bool GLU>
__device__ __forceinline__ void emit(const FwdGemmArgs& g, int e, int m, int p, int c, Vec<BF16> u,
                                     Vec<BF16> v) {
  constexpr int V = Vec<BF16>::V;
  const int64_t pr = (int64_t)p * g.n + c;
  if constexpr (GLU) {
    if (g.A) u.store(g.A, pr);
    if (g.B) v.store(g.B, pr);
#pragma unroll
    for (int j = 0; j < V; ++j) u.v[j] = u.v[j] * sigmoidf_acc(u.v[j]) * v.v[j];
    u.store(g.H, (int64_t)m * g.n + c);
  } else {
    if (g.bias) {
      const Vec<BF16> b = Vec<BF16>::load(g.bias, (int64_t)e * g.n + c);
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] += b.v[j];
    }
    if (g.Z) u.store(g.Z, pr);
    if (!g.Y) return;
    if (g.act != kActNone) {
#pragma unroll
      for (int j = 0; j < V; ++j) u.v[j] = act_rt(g.act, u.v[j]);
    }
    u.store(g.Y, pr);
  }
}

// ------------------------------------------------------------- tiled kernel
//
// Output tiles of BM packed rows of one expert x BN weight rows (GLU: BN/2 of
// W0 and the same BN/2 of W1, so that a lane holds a and b of the same
// elements).  Both operands have k contiguous in memory: 128-byte pieces of
// their rows (64 k in bf16, 32 in fp32) go straight from memory into LDS
// (dma16), kStages deep; a row gathered through the pairs costs nothing more,
// since every lane brings its own offset.  Lanes past an expert's rows, past
// the columns or past K take an offset outside the bound and write zeros.
// Granule G (16 bytes) of row r sits at G ^ swz128(r): the four 16-lane passes
// of a 16-byte LDS read then hit 16 distinct slots of the banks each.  Whole
// lines of 128 bytes matter: the loads alone take 445 us for the gate/up
// product of 131072 rows, 2048 x 2 x 768, and 580 in pieces of 64 bytes.
//
// Pipeline: a stage is multiplied in four quarters (half of the wave's rows x
// half of k); each quarter reads from LDS what the next one multiplies.  A part
// of a stage is loaded again as soon as every wave has its fragments: B and the
// first half of A after the first quarter, the second half of A after the third,
// 1.5 stages before they are needed (96 KB in flight per CU).  Waits name how
// many younger memory instructions may stand (the counter retires in order), so
// that neither the loads behind a part nor a finished tile's stores are waited
// for.  The down product (768 x 2048, 131072 rows) takes 534 us, with four
// stages of 64 bytes it took 647.  A copy without its 805 MB of stores took 406 us
// when it took 546, one that stores to a few lines in the L2 505: 100 us are the
// store code's, 40 the memory's.  The matrix pipes are busy 43 % of its cycles,
// and 60 % of the gate/up product's.
//
// Persistent blocks: each XCD (block b runs on XCD b mod 8) owns a contiguous
// eighth of the tiles, in which an expert's tiles lie 8 row tiles high, column
// by column, so that the tiles running on it at a time share operand panels in
// its L2 (1.09 GB fetched for 0.8 GB of weights and rows gathered 8 times from 67 MB).
//
// fp32 runs v_mfma_f32_16x16x4: a lane's 16-byte granule holds four k, and
// step s multiplies the s-th of every lane.  Which k those are is the same for
// both operands, so every k is met once.  Its sums restart every kRestart stages
// (256 k) and are added up apart: the roundings of a long sum stay below those
// of a library's split sums, for an addition in 64 products (bf16 inputs round
// by far more).
constexpr int kStages = 2, kRestart = 8;

template <int BM_, int BN_, int WGM_, int WGN_>
struct FwdCfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NW = WGM * WGN, NT = 64 * NW;
  static constexpr int TM = BM / WGM, TN = BN / WGN, FM = TM / 16, FN = TN / 16;
  static constexpr int QA = BM / 16 / NW, QB = BN / 8 / NW;  // 1 KB loads per wave: half of A, B
  static constexpr int L = 2 * QA + QB;                      // and of a stage
  static constexpr int SA = BM * 128, SS = (BM + BN) * 128;  // bytes of a stage
  static_assert(BM % (16 * NW) == 0 && BN % (8 * NW) == 0 && TN % 32 == 0 && TM % 32 == 0, "tile");
};

__device__ __forceinline__ int swz128(int r) { return (r >> 1) & 7; }

struct FwdJob {
  int e, m0, rows, n0;
};

// Position t of an expert-major tile list with nc column tiles: expert e holds
// positions [mt_off[e] nc, mt_off[e+1] nc).  e: start of the search (an expert
// at or before the right one; experts of later positions come later).
__device__ __forceinline__ FwdJob fwd_job(const FwdGemmArgs& g, int t, int nc, int e, int bm, int bno) {
  constexpr int kHigh = 8;
  const int mt = t / nc;
  int next = ld_table(g.mt_off, e + 1);
  while (next <= mt) next = ld_table(g.mt_off, ++e + 1);
  const int first = ld_table(g.mt_off, e), high = next - first;
  const int local = t - first * nc;
  const int grp = local / (kHigh * nc), rem = local - grp * kHigh * nc;
  const int h = high - grp * kHigh < kHigh ? high - grp * kHigh : kHigh;
  const int col = rem / h, row = grp * kHigh + rem - col * h;
  FwdJob j;
  j.e = e;
  j.m0 = ld_table(g.offsets, e) + row * bm;
  j.rows = min(bm, ld_table(g.offsets, e + 1) - j.m0);
  j.n0 = col * bno;
  return j;
}

template <bool BF16>
__device__ __forceinline__ f32x4 mma(u32x4 b, u32x4 a, f32x4 c) {
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

// Waits until at most n of this wave's memory instructions are outstanding (n
// rounded down to a value of the ladder; L loads make a stage) and all its LDS
// reads have arrived, then the barrier.  The empty asm statements keep memory
// accesses on their side.
template <int L>
__device__ __forceinline__ void stage_barrier(int n) {
  asm volatile("" ::: "memory");
  if (n == L) wait_vm<L>();
  else if (n >= 56) wait_vm<56>();
  else if (n >= 40) wait_vm<40>();
  else if (n >= 32) wait_vm<32>();
  else if (n >= 24) wait_vm<24>();
  else if (n >= 16) wait_vm<16>();
  else if (n >= L) wait_vm<L>();
  else wait_vm<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- tile store
// A wave stores its sub-tile 16 rows at a time through a piece of LDS of its
// own (kStoreBytes; no other wave waits), so that 8 lanes write 128 bytes of a
// row (fewer where the wave's sub-tile is narrower): in the MFMA layout a bf16
// store writes 16 rows x 8 bytes, at a quarter of the rate (measured for the
// backward products' tiles).  The LDS serves a wave in order, so the next
// piece is written as soon as this one's reads are issued.  Granules of 16
// bytes are swizzled by the row.  Lanes outside the tile store to a dump in
// the workspace instead of being masked off: every store is then issued, and
// their number, which the function returns, is known to the waits.
//
// fp32 lanes hold 16 bytes of a row and store them directly (not counted: 0).
constexpr int kStoreBytes = 2048;

// 16 rows of FO * 16 bf16 columns from the MFMA layout (v: four columns a
// fragment) to granules: lane l then holds granule l % (2 FO) of rows
// l / (2 FO) + q * 32 / FO in out[q] (FO = 1: lanes 0 .. 31 only).
template <int FO>
struct Piece {
  static constexpr int GR = 2 * FO, NQ = FO > 1 ? FO / 2 : 1, STEP = 64 / GR;
  static_assert(16 * GR * 16 <= kStoreBytes, "the piece of LDS holds 16 rows");
  __device__ __forceinline__ static int row(int l, int q) { return (l / GR + q * STEP) & 15; }
  __device__ __forceinline__ static void pass(char* buf, int l, const u32x2 (&v)[FO], u32x4 (&out)[NQ]) {
    const int lrow = l & 15, lq = l >> 4;
#pragma unroll
    for (int j = 0; j < FO; ++j)
      *reinterpret_cast<u32x2*>(buf + lrow * (GR * 16) + (((j * 2 + (lq >> 1)) ^ (lrow & (GR - 1))) << 4) +
                                (lq & 1) * 8) = v[j];
    wave_sync();
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = row(l, q);
      out[q] = *reinterpret_cast<const u32x4*>(buf + r * (GR * 16) + (((l % GR) ^ (r & (GR - 1))) << 4));
    }
    wave_sync();
  }
};

__device__ __forceinline__ u32x2 pack4(f32x4 v) {
  return u32x2{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
}

// EPI: with a bias, an activation or Z (not GLU)
template <class C, bool BF16, bool GLU, bool EPI>
__device__ __forceinline__ int fwd_store(const FwdGemmArgs& g, const FwdJob& job,
                                         const f32x4 (&acc)[C::FM][C::FN], char* buf, const int* prow,
                                         int w, int l) {
  constexpr int FO = GLU ? C::FN / 2 : C::FN;  // output fragments of a wave row
  typedef Piece<FO> P;
  const int wm = w / C::WGN, wn = w % C::WGN;
  const int cw = job.n0 + wn * FO * 16;  // first column of the wave
  const int lrow = l & 15, lq = l >> 4;  // MFMA layout: row, four columns
  char* const dump = (char*)g.dump + l * 16;
  int stores = 0;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int r0 = wm * C::TM + i * 16;
    if (r0 >= job.rows) break;
    if constexpr (!BF16) {
      if (r0 + lrow >= job.rows) continue;
#pragma unroll
      for (int j = 0; j < FO; ++j) {
        const int c = cw + j * 16 + lq * 4;
        if (c >= g.n) continue;
        Vec<BF16> u, v;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u.v[q] = acc[i][j][q];
          v.v[q] = acc[i][GLU ? j + FO : j][q];
        }
        emit<BF16, GLU>(g, job.e, job.m0 + r0 + lrow, prow[r0 + lrow], c, u, v);
      }
    } else {
      // the lane's rows and columns of a piece
      int64_t at[P::NQ];  // element in a PAIR output
      bool in[P::NQ];
      const int c = cw + l % P::GR * 8;
#pragma unroll
      for (int q = 0; q < P::NQ; ++q) {
        const int r = r0 + P::row(l, q);
        in[q] = r < job.rows && c < g.n && (FO > 1 || l < 32);
        at[q] = (int64_t)prow[r] * g.n + c;
      }
      auto put = [&](void* base, const u32x2 (&v)[FO]) {
        u32x4 out[P::NQ];
        P::pass(buf, l, v, out);
#pragma unroll
        for (int q = 0; q < P::NQ; ++q)
          *reinterpret_cast<u32x4*>(in[q] ? (char*)base + at[q] * 2 : dump) = out[q];
        stores += P::NQ;
      };
      u32x2 v[FO];
      if constexpr (GLU) {
        if (g.A) {
#pragma unroll
          for (int j = 0; j < FO; ++j) v[j] = pack4(acc[i][j]);
          put(g.A, v);
        }
        if (g.B) {
#pragma unroll
          for (int j = 0; j < FO; ++j) v[j] = pack4(acc[i][j + FO]);
          put(g.B, v);
        }
#pragma unroll
        for (int j = 0; j < FO; ++j) {
          const f32x4 x = acc[i][j], y = acc[i][j + FO];
          f32x4 h;
#pragma unroll
          for (int q = 0; q < 4; ++q) h[q] = silu_fast(x[q]) * y[q];
          v[j] = pack4(h);
        }
#pragma unroll
        for (int q = 0; q < P::NQ; ++q) at[q] = (int64_t)(job.m0 + r0 + P::row(l, q)) * g.n + c;
        put(g.H, v);
      } else {
        f32x4 u[FO];
#pragma unroll
        for (int j = 0; j < FO; ++j) u[j] = acc[i][j];
        if (EPI && g.bias) {
#pragma unroll
          for (int j = 0; j < FO; ++j) {
            const int cb = cw + j * 16 + lq * 4;
            const u32x2 b = *reinterpret_cast<const u32x2*>((const uint16_t*)g.bias +
                                                            (int64_t)job.e * g.n + (cb < g.n ? cb : 0));
            u[j] += f32x4{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
          }
        }
        if (EPI && g.Z) {
#pragma unroll
          for (int j = 0; j < FO; ++j) v[j] = pack4(u[j]);
          put(g.Z, v);
        }
        if (!EPI || g.Y) {
          if (EPI && g.act != kActNone) act_rows<FO, true>(g.act, u);
#pragma unroll
          for (int j = 0; j < FO; ++j)
            v[j] = u32x2{away_bf16x2(u[j][0], u[j][1]), away_bf16x2(u[j][2], u[j][3])};
          put(g.Y, v);
          if (g.Ylo) {
            // 16 rows of FO * 16 bytes: lane l holds 16 columns of row l / FO
#pragma unroll
            for (int j = 0; j < FO; ++j)
              *reinterpret_cast<uint32_t*>(buf + lrow * (FO * 16) + ((j ^ (lrow >> 1 & (FO - 1))) << 4) +
                                           lq * 4) = next_bytes(u[j]);
            wave_sync();
            const int r = l / FO & 15, cl = cw + l % FO * 16;
            const u32x4 lo = *reinterpret_cast<const u32x4*>(buf + r * (FO * 16) +
                                                             (((l % FO) ^ (r >> 1 & (FO - 1))) << 4));
            wave_sync();
            const bool inl = r0 + r < job.rows && cl < g.n && l < 16 * FO;
            char* d = (char*)g.Ylo + (int64_t)prow[r0 + r] * g.n + cl;
            if (g.n % 16 == 0) {
              *reinterpret_cast<u32x4*>(inl ? d : dump) = lo;
              ++stores;
            } else {  // n is a multiple of 8: so are the bytes' addresses
              *reinterpret_cast<u32x2*>(inl ? d : dump) = u32x2{lo[0], lo[1]};
              *reinterpret_cast<u32x2*>(inl && cl + 8 < g.n ? d + 8 : dump) = u32x2{lo[2], lo[3]};
              stores += 2;
            }
          }
        }
      }
    }
  }
  return stores;
}

// The operand fragments of a stage, 16 bytes per lane each: k half h (32 k in
// bf16) of the wave's columns (b) and of the upper and the lower half of its
// rows (a[0], a[1]).
template <class C>
struct Frags {
  static constexpr int HM = C::FM / 2;
  u32x4 a[2][2][HM], b[2][C::FN];
  // o: the lane's offset of fragment 0 in k half 0 (the swizzle is the same 16
  // rows on, and the other half of k 4 granules off)
  __device__ __forceinline__ void read_a(const char* stage, int o, int half, int h) {
#pragma unroll
    for (int i = 0; i < HM; ++i)
      a[half][h][i] = *reinterpret_cast<const u32x4*>(stage + (o ^ h * 64) + (half * HM + i) * 2048);
  }
  __device__ __forceinline__ void read_b(const char* stage, int o, int h) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
      b[h][j] = *reinterpret_cast<const u32x4*>(stage + C::SA + (o ^ h * 64) + j * 2048);
  }
  template <bool BF16>
  __device__ __forceinline__ void multiply(f32x4 (&acc)[C::FM][C::FN], int half, int h) const {
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
        acc[half * HM + i][j] = mma<BF16>(b[h][j], a[half][h][i], acc[half * HM + i][j]);
  }
};

// LDS reads one by one between the products that run meanwhile.
template <int READS, bool BF16>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int q = 0; q < READS; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);           // an LDS read
    __builtin_amdgcn_sched_group_barrier(0x008, BF16 ? 1 : 4, 0);  // MFMAs
  }
}

// Where the loads stand: a tile, its k-tile and what the next load takes.
template <class C>
struct FwdFeed {
  FwdJob job;
  int k;
  dma_rsrc a, w0, w1;  // the operands' rows from k = 0, to their ends
  int off[2][C::QA];
};

template <class C, bool BF16, bool GLU, bool EPI>
__global__ __launch_bounds__(C::NT, 2) void k_fwd_tile(FwdGemmArgs g) {
  constexpr int ES = BF16 ? 2 : 4, KT = 128 / ES;  // k per stage
  constexpr int BNO = GLU ? C::BN / 2 : C::BN;    // output columns of a tile
  constexpr int HN = C::TN / 2;                   // GLU: a wave's columns of each product
  __shared__ __attribute__((aligned(1024))) char lds[kStages * C::SS];
  __shared__ __attribute__((aligned(16))) char sbuf[BF16 ? C::NW * kStoreBytes : 16];
  __shared__ __attribute__((aligned(16))) int prow[4][C::BM];  // pair of every row, by tile
  __shared__ __attribute__((aligned(16))) int xrow[2][C::BM];  // its row of X
  const int nc = (g.n + BNO - 1) / BNO;
  const int ntiles = ld_table(g.mt_off, g.E) * nc;
  const int x = blockIdx.x & 7, nb = gridDim.x >> 3;
  const int tend = (int)((int64_t)ntiles * (x + 1) / 8);
  int t = (int)((int64_t)ntiles * x / 8) + (int)(blockIdx.x >> 3);
  if (t >= tend) return;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), l = lane_id();
  const int wm = w / C::WGN, wn = w % C::WGN;
  // stages of a tile, zeros past K: three at least, so that the feed is never
  // more than one tile ahead and the rows of the next tile, asked for when the
  // feed enters this one, are there when it leaves it
  const int nk = max((g.K + KT - 1) / KT, 3);
  const int64_t kb = (int64_t)g.K * ES;  // bytes of a weight row

  // this lane's place in the 1 KB blocks (8 rows) that its wave loads
  const int lr = l >> 3;
  auto gran = [&](int r) { return ((l & 7) ^ swz128(r)) * 16; };
  auto arow = [&](int half, int q) {  // the upper or lower half of every wave's rows
    const int r = (w * C::QA + q) * 8, in = r % (C::TM / 2);
    return r / (C::TM / 2) * C::TM + half * (C::TM / 2) + in;
  };
  auto brow = [&](int q) { return (w * C::QB + q) * 8; };
  int boff[C::QB];
#pragma unroll
  for (int q = 0; q < C::QB; ++q) {
    const int r = brow(q) + lr, in = r % C::TN;
    const int col = GLU ? (r / C::TN) * HN + in % HN : r;
    boff[q] = (int)(col * kb) + gran(r);
  }
  // and in the fragments that it multiplies
  const int fr = l & 15, fo = fr * 128 + (((l >> 4) ^ swz128(fr)) << 4);
  const int ao = wm * C::TM * 128 + fo, bo = wn * C::TN * 128 + fo;

  int vm = 0;  // memory instructions of this wave so far
  FwdFeed<C> f;
  FwdJob next, cur;   // the tile after the feed's; the one being multiplied
  bool more = true;   // `next` is a tile
  int entered = -1;   // tiles that the feed has entered, less one
  auto look = [&]() {  // the rows of `next`, straight into LDS
    if (w * 64 < C::BM) {
      const int at = next.m0 + w * 64, slot = entered + 1;
      dma4(uniform(make_dma_rsrc((const char*)(g.kept + at), (int64_t)(g.N - at) * 4)),
           &prow[slot & 3][w * 64], l * 4);
      dma4(uniform(make_dma_rsrc((const char*)(g.rows + at), (int64_t)(g.N - at) * 4)),
           &xrow[slot & 1][w * 64], l * 4);
      vm += 2;
    }
  };
  auto enter = [&]() {  // the feed moves on to `next`
    ++entered;
    f.job = next;
    f.k = 0;
    const char* xa = (const char*)g.X + (g.gather ? 0 : (int64_t)next.m0 * g.ldx * ES);
    f.a = uniform(make_dma_rsrc(xa, g.gather ? g.x_bytes
                                             : ((int64_t)(next.rows - 1) * g.ldx + g.K) * ES));
    const int64_t wat = (int64_t)next.e * g.w_stride * ES + next.n0 * kb;
    const int64_t wleft = min<int64_t>((g.n - next.n0) * kb, kOobOff);
    f.w0 = uniform(make_dma_rsrc((const char*)g.W0 + wat, wleft));
    if constexpr (GLU) f.w1 = uniform(make_dma_rsrc((const char*)g.W1 + wat, wleft));
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int q = 0; q < C::QA; ++q) {
        const int r = arow(half, q) + lr;
        const int row = g.gather ? xrow[entered & 1][r] : r;
        f.off[half][q] = r < next.rows ? row * (int)(g.ldx * ES) + gran(r) : kOobOff;
      }
    t += nb;
    more = t < tend;
    if (more) {
      next = fwd_job(g, t, nc, next.e, C::BM, BNO);
      look();
    }
  };
  bool fed = false;  // the feed is past the last tile
  // stage s <- the feed's k-tile, B and the first half of A or the second half
  auto feed = [&](int s, auto second) {
    if (fed) return;
    char* base = lds + s * C::SS;
    const int at = f.k * 128, left = (int)kb - at;  // bytes of a row before and from this k-tile
    auto load = [&](auto tail) {
      constexpr int half = second;
#pragma unroll
      for (int q = 0; q < C::QA; ++q) {
        const int r = arow(half, q);
        dma16(f.a, reinterpret_cast<uint16_t*>(base + r * 128),
              tail && gran(r + lr) >= left ? kOobOff : f.off[half][q], at);
      }
      if constexpr (!half) {
#pragma unroll
        for (int q = 0; q < C::QB; ++q) {
          const int r = brow(q);
          const bool up = GLU && r % C::TN >= HN;
          dma16(up ? f.w1 : f.w0, reinterpret_cast<uint16_t*>(base + C::SA + r * 128),
                tail && gran(r + lr) >= left ? kOobOff : boff[q], at);
        }
      }
    };
    if (left >= 128)
      load(std::false_type());
    else
      load(std::true_type());
    vm += second ? C::QA : C::QA + C::QB;
    if (second && ++f.k == nk) {
      fed = !more;
      if (more) enter();
    }
  };

  next = fwd_job(g, t, nc, find_expert(g.mt_off, g.E, t / nc), C::BM, BNO);
  look();
  stage_barrier<C::L>(0);
  cur = next;
  enter();
  std::false_type first;
  std::true_type second;
  // mk[i]: vm just after the loads of the i-th oldest half stage in flight
  int mk[3];
  feed(0, first);
  const int m0 = vm;
  feed(0, second);
  mk[0] = vm;
  feed(1, first);
  mk[1] = vm;
  feed(1, second);
  mk[2] = vm;
  auto shift = [&]() {
    mk[0] = mk[1];
    mk[1] = mk[2];
    mk[2] = vm;
  };
  stage_barrier<C::L>(vm - m0);
  Frags<C> f01;
  f01.read_a(lds, ao, 0, 0);
  f01.read_b(lds, bo, 0);
  int st = 0;
  for (int done = 0;; ++done) {
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 total[BF16 ? 1 : C::FM][C::FN] = {};  // fp32: of the finished runs of stages
    // Four quarters, each reading what the next one multiplies.  A wave enters
    // with the first one's fragments read (or on their way).
    for (int k = 0; k < nk; ++k) {
      const char* stage = lds + st * C::SS;
      f01.read_a(stage, ao, 0, 1);
      f01.read_b(stage, bo, 1);
      f01.template multiply<BF16>(acc, 0, 0);
      interleave<C::FM / 2 + C::FN, BF16>();
      // every wave has B and the first half of A; the second half is there
      stage_barrier<C::L>(vm - mk[0]);
      f01.read_a(stage, ao, 1, 0);
      f01.template multiply<BF16>(acc, 0, 1);
      interleave<C::FM / 2, BF16>();
      feed(st, first);  // behind the products: before them 935 us for gate/up instead of 870
      shift();
      f01.read_a(stage, ao, 1, 1);
      f01.template multiply<BF16>(acc, 1, 0);
      interleave<C::FM / 2, BF16>();
      // every wave has the second half; the next stage's B and first half are there
      stage_barrier<C::L>(vm - mk[0]);
      const char* behind = lds + (st ^ 1) * C::SS;
      f01.read_a(behind, ao, 0, 0);
      f01.read_b(behind, bo, 0);
      f01.template multiply<BF16>(acc, 1, 1);
      interleave<C::FM / 2 + C::FN, BF16>();
      feed(st, second);
      shift();
      st ^= 1;
      if constexpr (!BF16) {
        if (k % kRestart == kRestart - 1 || k == nk - 1) {
          const bool last = k == nk - 1;
#pragma unroll
          for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
              total[i][j] += acc[i][j];
              acc[i][j] = last ? total[i][j] : f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
      }
    }
    vm += fwd_store<C, BF16, GLU, EPI>(g, cur, acc, sbuf + (BF16 ? w * kStoreBytes : 0), prow[done & 3], w,
                                         l + opaque_uniform(0));
    if (done == entered) break;
    cur = f.job;
  }
}

// The rows of X in packed order (X too large for the 32-bit offsets of the
// gathering loads): one wave per row, 16 bytes a lane.
__global__ __launch_bounds__(256) void k_fwd_pack(FwdGemmArgs g, char* out) {
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= g.offsets[g.E]) return;
  const int64_t es = g.bf16 ? 2 : 4, row = g.rows[m];
  const u32x4* src = reinterpret_cast<const u32x4*>((const char*)g.X + row * g.ldx * es);
  u32x4* dst = reinterpret_cast<u32x4*>(out + (int64_t)m * g.K * es);
  for (int c = lane_id(); c < g.K * es / 16; c += kWave) dst[c] = src[c];
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

// One wave per token and 512 (bf16) or 256 (fp32) columns.  Bound by memory: 16384
// tokens of 8 pairs, 2048 columns, take 186 us for 872 MB, the rate of a large
// copy; asking for four pairs' rows at once changed nothing.
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
  Vec<BF16> sum;
  float (&acc)[V] = sum.v;
  auto add_up = [&](auto inf) {
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    if (a.R) sum = Vec<BF16>::load(a.R, (int64_t)t * a.ldr + c);
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
          acc[j] = fmaf(w, join_bits<inf>(hi, l8), acc[j]);
        }
      } else {
        const f32x4 x = *reinterpret_cast<const f32x4*>((const float*)a.Y + at);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, x[j], acc[j]);
      }
    }
  };
  add_up(std::false_type());
  if constexpr (BF16) {
    // a NaN may have been an infinity: once more (the test for one in every term
    // took 5 us of the 1450 of a 16384-token call)
    bool nan = false;
#pragma unroll
    for (int j = 0; j < V; ++j) nan |= acc[j] != acc[j];
    if (nan) add_up(std::true_type());
  }
  sum.store(a.out, (int64_t)t * a.d + c);
}

}  // namespace

namespace {

// Rows x columns, and waves: a GLU wave holds half as many output columns, so
// its sub-tile is wider (64 output columns a wave, 128 bytes a row, for L).
template <bool GLU> using FwdL = FwdCfg<256, 256, GLU ? 4 : 2, GLU ? 2 : 4>;
template <bool GLU> using FwdM = FwdCfg<128, 128, 2, 2>;
template <bool GLU> using FwdS = FwdCfg<64, 128, GLU ? 2 : 1, GLU ? 2 : 4>;

template <class C, bool BF16, bool GLU, bool EPI>
hipError_t launch_tiles(const FwdGemmArgs& g, hipStream_t s) {
  constexpr int bno = GLU ? C::BN / 2 : C::BN;
  const int64_t tiles = ((int64_t)g.N / C::BM + g.E) * ((g.n + bno - 1) / bno);
  if (tiles > 0x7fffffffll) return hipErrorInvalidValue;
  const int cap = grid_cap_of<k_fwd_tile<C, BF16, GLU, EPI>, C::NT>() & ~7;
  const int64_t want = (tiles + 7) & ~7ll;
  const int grid = (int)(want < cap ? want : cap < 8 ? 8 : cap);
  LRM_LAUNCH(grid, C::NT, 0, s, k_fwd_tile<C, BF16, GLU, EPI>)(g);
  return hipGetLastError();
}

template <template <bool> class C>
hipError_t launch_f32(const FwdGemmArgs& g, hipStream_t s) {
  return g.glu ? launch_tiles<C<true>, false, true, false>(g, s)
               : launch_tiles<C<false>, false, false, true>(g, s);
}

template <template <bool> class C>
hipError_t launch_bf16(const FwdGemmArgs& g, hipStream_t s) {
  if (g.glu) return launch_tiles<C<true>, true, true, false>(g, s);
  return g.bias || g.Z || g.act != kActNone ? launch_tiles<C<false>, true, false, true>(g, s)
                                            : launch_tiles<C<false>, true, false, false>(g, s);
}

}  // namespace

int fwd_tile_forced() {
  const char* env = getenv("LRM_FWD_TILE");
  const int v = env ? atoi(env) : 0;
  return v == 64 || v == 128 || v == 256 ? v : 0;
}

// Rows of a tile: by the rows of an average expert.  bf16 (both products of a
// Qwen3-shaped layer, 128 experts): 128 rows an expert 350 us with tiles of 128
// and 377 with 256, 187 rows 420 and 417, 256 rows 560 and 502 (tiles of 64 are
// within 3 % of 128 from 1 to 32 rows an expert: there are none).  fp32 (1024 x
// 1408, 8 experts): 128 rows an expert 55 us with tiles of 64 and 93 with 128,
// 1024 rows 251 and 250, 4096 rows 870 and 862.
int fwd_tile_rows(const FwdGemmArgs& g) {
  const int v = fwd_tile_forced(), avg = g.N / g.E;
  if (!g.bf16) return v ? (v < 128 ? v : 128) : avg >= 1536 ? 128 : 64;
  if (v) return v < 128 ? 128 : v;
  return avg >= 192 ? 256 : 128;
}

hipError_t launch_fwd_gemm(const FwdGemmArgs& g, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  if (g.gather && g.x_bytes > kFwdGatherMax) return hipErrorInvalidValue;
  const int rows = fwd_tile_rows(g);
  if (!g.bf16) return rows == 128 ? launch_f32<FwdM>(g, s) : launch_f32<FwdS>(g, s);
  return rows == 256 ? launch_bf16<FwdL>(g, s) : launch_bf16<FwdM>(g, s);
}

hipError_t launch_fwd_pack(const FwdGemmArgs& g, void* out, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  LRM_LAUNCH((g.N + 3) / 4, 256, 0, s, k_fwd_pack)(g, (char*)out);
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
