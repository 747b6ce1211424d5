// Activation checkpoints: x -> 8-bit q with one power-of-two scale per block of
// 32 columns, and back.  HBM-bound: 2 (or 4) bytes in and 33/32 out per
// element, and the reverse.  32768 x 4096 bf16 to e4m3 on one MI355X: 84 us
// (4.8 TB/s; 69 and 5.9 after a restore has left the caches alone), back 62 (6.6; a
// 1 GiB copy moves 5.45).
//
// A vector is 16 bytes of x (8 bf16 or 4 float32), so 4 or 8 consecutive lanes
// hold a block and find its largest magnitude with two or three lane exchanges.
#include "layer_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;   // vectors in flight per thread

// Vectors per row, padding included: whole scale words, so that the lanes
// past the row write the padding of q and scale.
__host__ __device__ __forceinline__ uint32_t vecs_per_row(const Ckpt& c, int n) {
  return uint32_t(c.s_pitch * MUON_CKPT_BLOCK / n);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void save_kernel(const void* x, int64_t ldx, Ckpt c,
                                                        int64_t tokens, int cols) {
  using R = RowVec<BF16>;
  constexpr int N = R::N;
  const uint32_t vpr = vecs_per_row(c, N);
  const int64_t total = tokens * int64_t(vpr);
  for (int64_t base = int64_t(blockIdx.x) * (kThreads * kPerThread); base < total;
       base += int64_t(gridDim.x) * (kThreads * kPerThread)) {
    const int64_t row0 = base / vpr;
    const uint32_t rem = uint32_t(base - row0 * vpr);
    u32x4_t w[kPerThread];
    int64_t row[kPerThread];
    int col[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint32_t at = rem + j * kThreads + threadIdx.x;
      const uint32_t r = at / vpr;
      row[j] = row0 + r;
      col[j] = int((at - r * vpr) * N);
      w[j] = u32x4_t{0, 0, 0, 0};
      if (row[j] < tokens)
        w[j] = load_raw<BF16>(static_cast<const typename R::T*>(x) + row[j] * ldx, col[j], cols);
    }
    // blocks of a row never straddle a wave (vpr is a multiple of 16), and the
    // lanes of one block lie in one row: they all pass the test below together
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (row[j] < tokens) ckpt_store<BF16>(c, row[j], col[j], cols, w[j]);
  }
}

template <bool BF16, bool STREAM>
__global__ __launch_bounds__(kThreads) void restore_kernel(Ckpt c, void* x, int64_t tokens,
                                                           int cols) {
  using R = RowVec<BF16>;
  constexpr int N = R::N;
  const uint32_t vpr = uint32_t((cols + N - 1) / N);
  const int64_t total = tokens * int64_t(vpr);
  for (int64_t base = int64_t(blockIdx.x) * (kThreads * kPerThread); base < total;
       base += int64_t(gridDim.x) * (kThreads * kPerThread)) {
    const int64_t row0 = base / vpr;
    const uint32_t rem = uint32_t(base - row0 * vpr);
    CkptVec<N> r8[kPerThread];
    int64_t row[kPerThread];
    int col[kPerThread];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint32_t at = rem + j * kThreads + threadIdx.x;
      const uint32_t r = at / vpr;
      row[j] = row0 + r;
      col[j] = int((at - r * vpr) * N);
      if (row[j] < tokens) r8[j] = ckpt_load<N>(c, row[j], col[j]);
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (row[j] < tokens) {
        float v[N];
        ckpt_values<N>(r8[j], c.fmt, v);
        store_vec<BF16, STREAM>(static_cast<typename R::T*>(x) + row[j] * cols, col[j], cols, v);
      }
  }
}

// Enough blocks to fill the chip several times over; larger inputs loop.
unsigned grid_for(int64_t vectors) {
  const int64_t b = (vectors + kThreads * kPerThread - 1) / (kThreads * kPerThread);
  return unsigned(b < 65536 ? b : 65536);
}

}  // namespace

hipError_t launch_ckpt_save(const void* x, int64_t ldx, bool bf16, const Ckpt& c, int64_t tokens,
                            int cols, hipStream_t s) {
  const int64_t vecs = tokens * int64_t(vecs_per_row(c, bf16 ? 8 : 4));
  if (bf16)
    hipLaunchKernelGGL(save_kernel<true>, dim3(grid_for(vecs)), dim3(kThreads), 0, s, x, ldx, c,
                       tokens, cols);
  else
    hipLaunchKernelGGL(save_kernel<false>, dim3(grid_for(vecs)), dim3(kThreads), 0, s, x, ldx, c,
                       tokens, cols);
  return hipGetLastError();
}

hipError_t launch_ckpt_restore(const Ckpt& c, void* x, bool bf16, int64_t tokens, int cols,
                               hipStream_t s) {
  const int n = bf16 ? 8 : 4;
  const int64_t vecs = tokens * int64_t((cols + n - 1) / n);
  // More than half of the 256 MB Infinity Cache streams past it: save and restore
  // of 32768 x 4096 bf16 156 -> 131 us, with a reader of the values 164 -> 152;
  // for 16384 x 4096 the reader loses more than the 8 us that the restore gains.
  const bool stream = tokens * int64_t(cols) * (bf16 ? 2 : 4) > (int64_t(1) << 27);
  const dim3 grid(grid_for(vecs)), block(kThreads);
  if (bf16 && stream)
    hipLaunchKernelGGL((restore_kernel<true, true>), grid, block, 0, s, c, x, tokens, cols);
  else if (bf16)
    hipLaunchKernelGGL((restore_kernel<true, false>), grid, block, 0, s, c, x, tokens, cols);
  else if (stream)
    hipLaunchKernelGGL((restore_kernel<false, true>), grid, block, 0, s, c, x, tokens, cols);
  else
    hipLaunchKernelGGL((restore_kernel<false, false>), grid, block, 0, s, c, x, tokens, cols);
  return hipGetLastError();
}

}  // namespace muon
