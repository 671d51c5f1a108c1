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

#include "common.h"
#include "gemm_util.h"
#include "launch.h"

namespace lrm {

namespace {

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

// The outputs of V consecutive columns c .. (c < n, n a multiple of V) of
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
    if constexpr (BF16) {
      if (g.Ylo) {
        uint32_t lo[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          lo[j >> 2] |= split_lo(u.v[j], f32_to_bf16_bits(u.v[j])) << (8 * (j & 3));
        *reinterpret_cast<u32x2*>(g.Ylo + pr) = u32x2{lo[0], lo[1]};
      }
    }
  }
}

// ------------------------------------------------------------- tiled kernel
//
// Output tiles of BM packed rows of one expert x BN weight rows (GLU: BN/2 of
// W0 and the same BN/2 of W1, so that a lane holds a and b of the same
// elements).  Both operands have k contiguous in memory: 128-byte pieces of
// their rows (64 k in bf16, 32 in fp32) go straight from memory into LDS
// (dma16), two stages deep, in the swizzled granule order of lds_off; a row
// gathered through kept and token costs nothing more, since every lane brings
// its own offset.  Lanes past an expert's rows, past the columns or past K
// take an offset outside the bound and write zeros.
//
// Persistent blocks: each XCD (block b runs on XCD b mod 8) owns a contiguous
// eighth of the tiles, in which an expert's tiles lie 8 row tiles high, column
// by column, so that the tiles running on it at a time share operand panels in
// its L2.  The next tile's rows are looked up during the current one, and its
// first loads are in flight while the current tile is stored.
//
// fp32 runs v_mfma_f32_16x16x4: a lane's 16-byte granule holds four k, and
// step s multiplies the s-th of every lane.  Which k those are is the same for
// both operands, so every k is met once.
template <int BM_, int BN_, int WGM_, int WGN_>
struct FwdCfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NW = WGM * WGN, NT = 64 * NW;
  static constexpr int TM = BM / WGM, TN = BN / WGN, FM = TM / 16, FN = TN / 16;
  static constexpr int QA = BM / 8 / NW, QB = BN / 8 / NW;  // 1 KB loads per wave and stage
  static constexpr int SA = BM * 128, SS = (BM + BN) * 128;  // bytes of a stage
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && TN % 32 == 0 && TM % 16 == 0, "tile");
};

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

// All of this wave's loads into LDS have arrived, and every wave's have.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  wait_vm<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- tile store
// The sums of a tile go through LDS (the stage just consumed, in passes of two
// fragment rows of every wave), so that the epilogue works on whole rows: a
// thread takes 16 output bytes of a row, its neighbours the next ones.  In the
// MFMA layout a store would write 16 rows x 8 bytes, at a quarter of the rate
// (measured for the backward products' tiles).  LDS rows hold the BN sums of a
// row, granules of four swizzled by the row.
template <class C, bool BF16, bool GLU>
__device__ __forceinline__ void fwd_store(const FwdGemmArgs& g, const FwdJob& job,
                                          const f32x4 (&acc)[C::FM][C::FN], char* buf, const int* prow,
                                          int w, int l) {
  constexpr int BNO = GLU ? C::BN / 2 : C::BN, HN = C::TN / 2;
  constexpr int V = Vec<BF16>::V, QR = BNO / V, RB = C::BN * 4, ROWS = C::WGM * 32;
  static_assert(ROWS * RB <= C::SS, "a pass fits a stage");
  const int wm = w / C::WGN, wn = w % C::WGN;
#pragma unroll
  for (int i0 = 0; i0 < C::FM; i0 += 2) {
    __syncthreads();  // the buffer's readers are done
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = wm * 32 + i * 16 + (l & 15);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        // column of the sums in the LDS row: W0's, then W1's
        const int c = !GLU ? wn * C::TN + j * 16
                           : (j * 16 >= HN ? BNO - HN : 0) + wn * HN + j * 16;
        const int q = c / 4 + (l >> 4);
        *reinterpret_cast<f32x4*>(buf + r * RB + ((q ^ (r & 15)) << 4)) = acc[i0 + i][j];
      }
    }
    __syncthreads();
    for (int u = threadIdx.x; u < ROWS * QR; u += C::NT) {
      const int r = u / QR, c = u % QR * V;
      const int row = (r >> 5) * C::TM + i0 * 16 + (r & 31);  // row of the tile
      if (row >= job.rows || job.n0 + c >= g.n) continue;
      auto sums = [&](int col) {
        Vec<BF16> x;
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(buf + r * RB + (((col / 4 + q) ^ (r & 15)) << 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) x.v[4 * q + j] = y[j];
        }
        return x;
      };
      emit<BF16, GLU>(g, job.e, job.m0 + row, prow[row], job.n0 + c, sums(c), sums(GLU ? BNO + c : c));
    }
  }
}

template <class C, bool BF16, bool GLU>
__global__ __launch_bounds__(C::NT, 2) void k_fwd_tile(FwdGemmArgs g) {
  constexpr int ES = BF16 ? 2 : 4, KT = 128 / ES;  // k per stage
  constexpr int BNO = GLU ? C::BN / 2 : C::BN;     // output columns of a tile
  constexpr int HN = C::TN / 2;                    // GLU: a wave's columns of each product
  __shared__ __attribute__((aligned(1024))) char lds[2 * C::SS];
  __shared__ int prow[2][C::BM];  // pair of every row of the tile
  const int nc = (g.n + BNO - 1) / BNO;
  const int ntiles = ld_table(g.mt_off, g.E) * nc;
  const int x = blockIdx.x & 7, nb = gridDim.x >> 3;
  const int tend = (int)((int64_t)ntiles * (x + 1) / 8);
  int t = (int)((int64_t)ntiles * x / 8) + (int)(blockIdx.x >> 3);
  if (t >= tend) return;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), l = lane_id();
  const int wm = w / C::WGN, wn = w % C::WGN;
  const int nk = (g.K + KT - 1) / KT;
  const int64_t kb = (int64_t)g.K * ES;  // bytes of a weight row

  // this lane's granule of the 1 KB blocks that its wave loads
  const int lr = l >> 3;  // row inside a block
  int agran[C::QA], bgran[C::QB], boff[C::QB];
#pragma unroll
  for (int q = 0; q < C::QA; ++q)
    agran[q] = ((l & 7) ^ lds_swz((w * C::QA + q) * 8 + lr)) * 16;
#pragma unroll
  for (int q = 0; q < C::QB; ++q) {
    const int r = (w * C::QB + q) * 8 + lr;
    bgran[q] = ((l & 7) ^ lds_swz(r)) * 16;
    const int in = r % C::TN;
    const int col = GLU ? (r / C::TN) * HN + in % HN : r;
    boff[q] = (int)(col * kb) + bgran[q];
  }
  // fragment offsets: row bits 4 and 5 flip granule bits 0 and 2
  const int fa = wm * C::TM + (l & 15), fb = wn * C::TN + (l & 15);
  int ao[4], bo[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int flip = (v & 1) | (v & 2) << 1;
    ao[v] = fa * 128 + ((((l >> 4) ^ lds_swz(fa)) ^ flip) << 4);
    bo[v] = fb * 128 + ((((l >> 4) ^ lds_swz(fb)) ^ flip) << 4);
  }

  FwdJob cur = fwd_job(g, t, nc, find_expert(g.mt_off, g.E, t / nc), C::BM, BNO), nxt = cur;
  bool more = false;
  int aoff[C::QA], noff[C::QA], np[C::QA], npr = 0;
  // rows of a tile, in two dependent steps
  auto rows1 = [&](const FwdJob& j) {
#pragma unroll
    for (int q = 0; q < C::QA; ++q) {
      const int r = (w * C::QA + q) * 8 + lr;
      np[q] = g.gather && r < j.rows ? g.kept[j.m0 + r] : 0;
    }
    if ((int)threadIdx.x < C::BM) npr = (int)threadIdx.x < j.rows ? g.kept[j.m0 + threadIdx.x] : 0;
  };
  auto rows2 = [&](const FwdJob& j, int par) {
#pragma unroll
    for (int q = 0; q < C::QA; ++q) {
      const int r = (w * C::QA + q) * 8 + lr;
      const int64_t row = g.gather ? (g.x_pair ? np[q] : g.token[np[q]]) : r;
      noff[q] = r < j.rows ? (int)(row * g.ldx * ES) + agran[q] : kOobOff;
    }
    if ((int)threadIdx.x < C::BM) prow[par][threadIdx.x] = npr;
  };
  // stage s <- k-tile k of tile j with row offsets off
  auto issue = [&](const FwdJob& j, const int (&off)[C::QA], int k, int s) {
    const int kbyte = k * 128;
    const char* abase = (const char*)g.X + (g.gather ? 0 : (int64_t)j.m0 * g.ldx * ES) + kbyte;
    const int64_t abytes = g.gather ? g.x_bytes : ((int64_t)(j.rows - 1) * g.ldx + g.K) * ES;
    const int64_t wat = (int64_t)j.e * g.w_stride * ES + j.n0 * kb + kbyte;
    const int64_t wbytes = min<int64_t>((g.n - j.n0) * kb - kbyte, kOobOff);
    const dma_rsrc ra = uniform(make_dma_rsrc(abase, abytes - kbyte));
    const dma_rsrc r0 = uniform(make_dma_rsrc((const char*)g.W0 + wat, wbytes));
    dma_rsrc r1 = r0;
    if constexpr (GLU) r1 = uniform(make_dma_rsrc((const char*)g.W1 + wat, wbytes));
    char* base = lds + s * C::SS;
    const bool tail = kbyte + 128 > kb;
#pragma unroll
    for (int q = 0; q < C::QA; ++q)
      dma16(ra, reinterpret_cast<uint16_t*>(base + (w * C::QA + q) * 1024),
            tail && kbyte + agran[q] >= kb ? kOobOff : off[q]);
#pragma unroll
    for (int q = 0; q < C::QB; ++q) {
      const bool up = GLU && (w * C::QB + q) * 8 % C::TN >= HN;
      dma16(up ? r1 : r0, reinterpret_cast<uint16_t*>(base + C::SA + (w * C::QB + q) * 1024),
            tail && kbyte + bgran[q] >= kb ? kOobOff : boff[q]);
    }
  };

  rows1(cur);
  rows2(cur, 0);
#pragma unroll
  for (int q = 0; q < C::QA; ++q) aoff[q] = noff[q];
  issue(cur, aoff, 0, 0);
  int st = 0, par = 0;
  for (;;) {
    f32x4 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < nk; ++k) {
      stage_barrier();
      if (k == 0) {
        t += nb;
        more = t < tend;
        if (more) {
          nxt = fwd_job(g, t, nc, cur.e, C::BM, BNO);
          rows1(nxt);
        }
      }
      if (k == (nk > 1 ? 1 : 0) && more) rows2(nxt, par ^ 1);
      if (k + 1 < nk)
        issue(cur, aoff, k + 1, st ^ 1);
      else if (more)
        issue(nxt, noff, 0, st ^ 1);
      const char* As = lds + st * C::SS;
      const char* Bs = As + C::SA;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 af[C::FM], bf[C::FN];
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
          bf[j] = *reinterpret_cast<const u32x4*>(Bs + bo[(j & 1) | ((((j >> 1) & 1) ^ h) << 1)] + j * 2048);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
          af[i] = *reinterpret_cast<const u32x4*>(As + ao[(i & 1) | ((((i >> 1) & 1) ^ h) << 1)] + i * 2048);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j) acc[i][j] = mma<BF16>(bf[j], af[i], acc[i][j]);
      }
      st ^= 1;
    }
    // lane l of fragment (i, j): row 16 i + (l & 15), columns 16 j + 4 (l >> 4)
    // .. + 3 of the wave's sub-tile
    fwd_store<C, BF16, GLU>(g, cur, acc, lds + (st ^ 1) * C::SS, prow[par], w, l);
    if (!more) break;
    cur = nxt;
    par ^= 1;
#pragma unroll
    for (int q = 0; q < C::QA; ++q) aoff[q] = noff[q];
  }
}

// The rows of X in packed order (X too large for the 32-bit offsets of the
// gathering loads): one wave per row, 16 bytes a lane.
__global__ __launch_bounds__(256) void k_fwd_pack(FwdGemmArgs g, char* out) {
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= g.offsets[g.E]) return;
  const int p = g.kept[m];
  const int64_t es = g.bf16 ? 2 : 4, row = g.x_pair ? p : g.token[p];
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
  Vec<BF16> sum;
#pragma unroll
  for (int j = 0; j < V; ++j) sum.v[j] = 0.f;
  if (a.R) sum = Vec<BF16>::load(a.R, (int64_t)t * a.ldr + c);
  float (&acc)[V] = sum.v;
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
  sum.store(a.out, (int64_t)t * a.d + c);
}

}  // namespace

namespace {

typedef FwdCfg<256, 256, 2, 4> FwdL;
typedef FwdCfg<128, 128, 2, 2> FwdM;
typedef FwdCfg<64, 128, 1, 4> FwdS;

template <class C, bool BF16, bool GLU>
hipError_t launch_tiles(const FwdGemmArgs& g, hipStream_t s) {
  constexpr int bno = GLU ? C::BN / 2 : C::BN;
  const int64_t tiles = ((int64_t)g.N / C::BM + g.E) * ((g.n + bno - 1) / bno);
  if (tiles > 0x7fffffffll) return hipErrorInvalidValue;
  const int cap = grid_cap_of<k_fwd_tile<C, BF16, GLU>, C::NT>() & ~7;
  const int64_t want = (tiles + 7) & ~7ll;
  const int grid = (int)(want < cap ? want : cap < 8 ? 8 : cap);
  LRM_LAUNCH(grid, C::NT, 0, s, k_fwd_tile<C, BF16, GLU>)(g);
  return hipGetLastError();
}

template <class C>
hipError_t launch_cfg(const FwdGemmArgs& g, hipStream_t s) {
  if (g.bf16) return g.glu ? launch_tiles<C, true, true>(g, s) : launch_tiles<C, true, false>(g, s);
  return g.glu ? launch_tiles<C, false, true>(g, s) : launch_tiles<C, false, false>(g, s);
}

}  // namespace

// Rows of a tile: by the rows of an average expert.
int fwd_tile_rows(const FwdGemmArgs& g) {
  if (const char* env = getenv("LRM_FWD_TILE")) {
    const int v = atoi(env);
    if (v == 64 || v == 128 || v == 256) return v;
  }
  const int avg = g.N / g.E;
  return avg >= 512 ? 256 : avg >= 96 ? 128 : 64;
}

hipError_t launch_fwd_gemm(const FwdGemmArgs& g, hipStream_t s) {
  if (g.N <= 0) return hipSuccess;
  if (g.gather && g.x_bytes > kFwdGatherMax) return hipErrorInvalidValue;
  switch (fwd_tile_rows(g)) {
    case 256: return launch_cfg<FwdL>(g, s);
    case 128: return launch_cfg<FwdM>(g, s);
  }
  return launch_cfg<FwdS>(g, s);
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
