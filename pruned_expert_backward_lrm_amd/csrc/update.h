// What the update of the parameters shares between host and device: the table of
// tensors in GPU memory, the step's numbers and the random numbers' key.
#pragma once

#include <stdint.h>

#include "platform.h"

namespace lrm {

constexpr int kChunk = 2048;       // elements of a chunk: 8 for each thread of a block
constexpr int kMomentBlock = 32;   // elements that share an exponent
constexpr int kMaxTensors = 65536;

struct ParamEntry {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  uint8_t* m_exp;
  uint8_t* v_exp;
  int64_t n;
  int64_t chunk0;  // chunks of the tensors before
  int64_t block0;  // blocks of the tensors before (places of the random numbers)
  float lr, decay;
  int32_t vec;     // every array starts on a boundary of its 8 elements (16 bytes at most)
  int32_t _pad;
};

// The table: n entries, then chunk0 of each once more, and all chunks.
struct ParamTable {
  int32_t n;
  const ParamEntry* entry;
  const int64_t* chunk0;  // [n + 1]
};

constexpr int kTableBatch = 32;
struct TableBatch {
  ParamEntry entry[kTableBatch];
};

struct AdamArgs {
  double grad_scale;
  double over;  // max_norm / |grad_scale|, infinite without clipping
  double beta1, beta2;
  float lr, b1, d1, b2, d2, eps;  // betas and one less them
  // of a step that the host counts: 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t), the key
  float bias, root;
  uint32_t key;
  // of one that the GPU counts
  double ln1, ln2;  // logarithms of the betas
  uint64_t seed;
  const double* sumsq;
  int n_sumsq;
  const float* lr_dev;
  const int64_t* steps;
};

// Random numbers of the roundings: multiply-xorshift mixing; the constants are the
// fractional bits of the golden ratio and of the square roots of 2 and 3.
constexpr uint32_t kGold = 0x9E3779B9u, kRoot2 = 0x6A09E667u, kRoot3 = 0xBB67AE85u;
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= kRoot2;
  x ^= x >> 15;
  x *= kRoot3;
  return x ^ (x >> 16);
}
__host__ __device__ inline uint32_t step_key(uint64_t seed, uint64_t step) {
  uint32_t k = mix32((uint32_t)seed + kGold);
  k = mix32((k ^ (uint32_t)(seed >> 32)) + kGold);
  k = mix32((k ^ (uint32_t)step) + kGold);
  return mix32((k ^ (uint32_t)(step >> 32)) + kGold);
}

constexpr int kSumBlocks = 2048;  // persistent blocks of the sum, at most

hipError_t launch_params_table(const TableBatch& b, int first, int count, int n, int64_t chunks,
                               void* table, hipStream_t s);
hipError_t launch_grad_sumsq(const ParamTable& t, int64_t chunks, int g_bf16, double* part,
                             double* sumsq, hipStream_t s);
// p: 0 fp32, 1 bf16, 2 bf16 with fp32 masters
hipError_t launch_adamw(const ParamTable& t, int64_t chunks, int p, int g_bf16, int eight,
                        const AdamArgs& a, int64_t* steps, hipStream_t s);
hipError_t launch_moment_read(int64_t n, int second, const uint8_t* codes, const uint8_t* exps,
                              int bf16, void* out, hipStream_t s);

}  // namespace lrm
