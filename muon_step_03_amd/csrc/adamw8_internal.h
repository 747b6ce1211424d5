// Structures of AdamW with 8-bit states shared by its host file
// (adamw8_abi.hip) and kernels (k_adamw8.hip).
#pragma once

#include "layer_internal.h"

namespace muon {

// As many tensors as the 4 KB of a launch's arguments hold: a launch more costs the
// host 5 us (49 short vectors in two launches 35 us with their moments, in one 26).
constexpr int kAdam8Segs = MUON_ADAMW8_TENSORS_PER_LAUNCH;
constexpr int kAdam8Vec = 8;                   // elements per thread and vector
constexpr int kAdam8PerThread = 2;             // vectors per thread
constexpr int kAdam8Chunk = 256 * kAdam8Vec * kAdam8PerThread;   // elements per block

struct Adam8Seg {
  void* P;
  const void* G;
  uint8_t* m_q;
  uint8_t* m_scale;
  uint8_t* r_q;
  uint8_t* r_scale;
  int64_t n;
  float decay;          // 1 - lr*wd
  float step_size;      // lr / (1 - beta1^t)
  uint32_t seed;
  uint32_t begin;       // its first block
};
struct Adam8Batch {
  Adam8Seg seg[kAdam8Segs];
  int nseg;
  uint32_t blocks;
  float beta1, beta2, eps;
  float one_minus_beta1, one_minus_beta2;      // rounded once from double
  float inv_sqrt_bc2;                          // 1 / sqrt(1 - beta2^t)
};
static_assert(sizeof(Adam8Batch) <= 4096, "kernel arguments");

// States to read back; P and G of a segment are where its m and r go.
hipError_t launch_adamw8(const Adam8Batch& bt, bool bf16, hipStream_t s);
hipError_t launch_adamw8_moments(const Adam8Batch& bt, bool bf16, hipStream_t s);

}  // namespace muon
