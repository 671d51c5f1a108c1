// Building blocks of the tiled products: table reads, buffer resources, the
// swizzled LDS operand tile, loads straight into LDS, waits.
#pragma once

#include <atomic>

#include "common.h"

namespace lrm {

// Read of the per-expert tables (kept offsets, dX row-tile prefix) that no
// GEMM kernel writes.  Through the constant address space a wave-uniform index
// becomes a scalar load, which waits on its own counter; a vector load would
// also wait for every store the wave issued before it (one counter covers
// vector loads and stores, retired in order), so the first table read after a
// tile's stores would hold the wave until those stores reach the cache.
#ifdef LRM_CPU_EMU
__device__ __forceinline__ int ld_table(const int32_t* p, int i) { return p[i]; }
#else
typedef const __attribute__((address_space(4))) int32_t* table_ptr;
__device__ __forceinline__ int ld_table(const int32_t* p, int i) {
  return ((table_ptr)(uintptr_t)p)[i];
}
#endif

__device__ __forceinline__ int xcd_remap(int b, int G) {
  // hardware places block b on XCD b % 8; give each XCD a contiguous range
  return (b & 7) * (G >> 3) + (b >> 3);
}

// Largest e with mt_off[e] <= mt (mt < mt_off[E]).
__device__ __forceinline__ int find_expert(const int32_t* mt_off, int E, int mt) {
  int lo = 0, hi = E;  // invariant: mt_off[lo] <= mt < mt_off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ld_table(mt_off, mid) <= mt) lo = mid; else hi = mid;
  }
  return lo;
}

// LDS operand tile: R rows x 64 k (bf16), 128-byte rows, no padding.  The
// 16-byte granule G of row r sits at granule G ^ f(r), with f built from row
// bits as (r4, r3, r1 ^ r5).  On gfx950 a ds_read_b128 is served in four
// passes of 16 lanes ({0-3, 12-15, 20-23, 24-27}, {4-7, 8-11, 16-19, 28-31}
// and the same +32) over 64 four-byte banks, and a ds_write_b64 in passes of
// 16 consecutive lanes over 32 banks (both measured with bank-conflict
// counters).  With this f the fragment reads (16 consecutive rows, granules
// g and g+1 in a pass) and the transposed 8-byte stores (16 lanes: 8 rows 8
// apart x both halves of a granule) hit 16 distinct bank slots per pass.
constexpr int BK = 64;
__device__ __forceinline__ int lds_swz(int r) {
  return ((r >> 4) & 1) | (r & 8) >> 2 | (((r >> 1) ^ (r >> 5)) & 1) << 2;
}
// element offset of 8-byte half-granule h (0..15) of row r
__device__ __forceinline__ int lds_off(int r, int h) {
  return r * BK + ((h ^ (lds_swz(r) << 1)) << 2);
}

// Operand panels are read with buffer loads: a buffer resource per k-tile
// (scalar base and byte bound) plus per-lane byte offsets fixed for the whole
// output tile.  Loads past the bound return zero in hardware, which pads the
// k tail of a segment and the rows past an expert's block without any
// per-lane masking or address arithmetic inside the k loop.
typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kRsrcWord3 = 0x00020000;

__device__ __forceinline__ rsrc_t make_rsrc(const char* base, int64_t nbytes) {
  const int n = nbytes <= 0 ? 0 : (nbytes > 0x7ffffff0ll ? 0x7ffffff0 : (int)nbytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, n, kRsrcWord3);
}
// AUX: cache policy of the load (0 default, kStreamAux non-temporal)
template <int AUX = 0>
__device__ __forceinline__ u32x4 bload(rsrc_t r, int off) {
  return (u32x4)__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, AUX);
}
constexpr int kStreamAux = 2;  // the nt bit

// A byte offset past every bound that it is used with
constexpr int kOobOff = 0x7fff0000;

// A wave-uniform value the compiler cannot see through: offsets built from it
// are computed where the stores are, not hoisted out of the tile loop (where
// the 32 per-store offsets would take 32 live registers).
#ifdef LRM_CPU_EMU
__device__ __forceinline__ int opaque_uniform(int x) { return x; }
#else
__device__ __forceinline__ int opaque_uniform(int x) {
  asm volatile("" : "+s"(x));
  return x;
}
#endif

#ifdef LRM_CPU_EMU
typedef void* lds_vptr;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef s16x4* lds_s16x4;
#else
typedef __attribute__((address_space(3))) void* lds_vptr;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;
#endif

// 16 bytes per lane from r at byte voff into LDS at lds + 16 * lane (lds is
// wave-uniform); past the bound the lane writes zeros (measured).  Written
// as inline asm so that the compiler, which does not track these loads, does
// not wait for every one in flight before each LDS read: the kernel orders
// them itself (dma_barrier).  The LDS address goes in M0 as an input operand.
// Five wait states stand before the load: the compiler does not look inside the
// asm for the hazard of a scalar register written by a vector instruction
// (v_readfirstlane, or v_readlane from a spilled register) and read by a memory
// instruction, and may put such a write right before it.
#ifdef LRM_CPU_EMU
typedef rsrc_t dma_rsrc;
__device__ __forceinline__ dma_rsrc make_dma_rsrc(const char* base, int64_t nbytes) {
  return make_rsrc(base, nbytes);
}
__device__ __forceinline__ void dma16(dma_rsrc r, uint16_t* lds, int voff) {
  const u32x4 v = bload(r, voff);
  std::memcpy(reinterpret_cast<char*>(lds) + 16 * lane_id(), &v, 16);
}
// the same at byte voff + soff (soff wave-uniform)
__device__ __forceinline__ void dma16(dma_rsrc r, uint16_t* lds, int voff, int soff) {
  dma16(r, lds, voff + soff);
}
// 4 bytes per lane, to LDS at lds + 4 * lane
__device__ __forceinline__ void dma4(dma_rsrc r, int* lds, int voff) {
  int v = 0;
  if (voff + 4 <= r.n) std::memcpy(&v, r.base + voff, 4);
  lds[lane_id()] = v;
}
__device__ __forceinline__ dma_rsrc uniform(dma_rsrc r) { return r; }
#else
typedef u32x4 dma_rsrc;  // buffer resource words: base, bound, raw access
__device__ __forceinline__ dma_rsrc make_dma_rsrc(const char* base, int64_t nbytes) {
  const int n = nbytes <= 0 ? 0 : (nbytes > 0x7ffffff0ll ? 0x7ffffff0 : (int)nbytes);
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return dma_rsrc{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)n, (uint32_t)kRsrcWord3};
}
__device__ __forceinline__ void dma16(dma_rsrc r, uint16_t* lds, int voff) {
  const uint32_t la = (uint32_t)(uintptr_t)(lds_vptr)lds;
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "{m0}"(la)
               : "memory");
}
// the same at byte voff + soff (soff wave-uniform)
__device__ __forceinline__ void dma16(dma_rsrc r, uint16_t* lds, int voff, int soff) {
  const uint32_t la = (uint32_t)(uintptr_t)(lds_vptr)lds;
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(r), "s"(soff), "{m0}"(la)
               : "memory");
}
// 4 bytes per lane, to LDS at lds + 4 * lane
__device__ __forceinline__ void dma4(dma_rsrc r, int* lds, int voff) {
  const uint32_t la = (uint32_t)(uintptr_t)(lds_vptr)lds;
  asm volatile("s_nop 4\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "{m0}"(la)
               : "memory");
}
// A resource whose words are the same in every lane, in scalar registers (the
// asm operand has to be; the compiler may keep uniform values in vector ones).
__device__ __forceinline__ dma_rsrc uniform(dma_rsrc r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
  return r;
}
#endif

// s_waitcnt vmcnt(N) lgkmcnt(0) (expcnt not waited on)
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Resident blocks of a GEMM kernel on the current device, cached for the
// first 16 devices (concurrent callers may both compute it; they store the
// same value).
template <auto Kern, int NTH>
inline int grid_cap_of() {
  static std::atomic<int> cap[16];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 0;
  if (dev < 16) {
    const int c = cap[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int cus = 0, occ = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0)
    cus = 256;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, Kern, NTH, 0) != hipSuccess || occ <= 0)
    occ = 1;
  const int c = cus * occ;
  if (dev < 16) cap[dev].store(c, std::memory_order_relaxed);
  return c;
}

}  // namespace lrm
