// Weights in 8 bits: e4m3 with one power-of-two scale per block of 128 x 128,
// kept both as they are and with rows and columns exchanged, so that forward
// product (along the columns) and input gradient (along the rows) both read
// runs of k.  The square block gives both the same numbers.
//
// A block of threads takes one block of the weight: read once, its largest
// magnitude found, converted, written, and written again exchanged through LDS.
// HBM-bound: 2 (or 4) bytes in and 2 out per element.  Measured on one MI355X: bf16
// 4096 x 1024 6.7 us; 5 float32 weights of 1411 x 777 13.0 us with loads that a
// branch guards, 9.6 with loads clamped into the row and shifted, as here.
#include "linear_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256, SIDE = MUON_WEIGHT_BLOCK;
constexpr int PITCH = SIDE + 4;   // bytes: rows start on different banks

// INSIDE: a row holds a vector at least.
template <bool BF16, bool INSIDE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const Weight8 p) {
  using R = RowVec<BF16>;
  constexpr RowEnd END = INSIDE ? END_INSIDE : END_SHORT;
  constexpr int N = R::N, LANES = SIDE / N, ROWS = kThreads / LANES, PASSES = SIDE / ROWS;
  __shared__ uint32_t most[kThreads / 64];
  __shared__ __attribute__((aligned(16))) uint8_t tile[SIDE * PITCH];
  const int t = threadIdx.x;
  const int bc = (p.cols + SIDE - 1) / SIDE, br = (p.rows + SIDE - 1) / SIDE;
  const int64_t which = blockIdx.x / (uint32_t(bc) * br);
  const int block = int(blockIdx.x % (uint32_t(bc) * br));
  const int r0 = block / bc * SIDE, c0 = block % bc * SIDE;
  const typename R::T* W = static_cast<const typename R::T*>(p.W) + which * p.rows * int64_t(p.cols);

  u32x4_t raw[PASSES];
  const int col = t % LANES * N;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t row = min(r0 + i * ROWS + t / LANES, p.rows - 1);
    raw[i] = load_ahead<BF16, END>(W + row * p.cols, c0 + col, p.cols);
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    settle<BF16, END>(raw[i], c0 + col, p.cols);
    if (r0 + i * ROWS + t / LANES >= p.rows) raw[i] = u32x4_t{0, 0, 0, 0};
    float v[N];
    unpack_raw<BF16>(raw[i], v);
#pragma unroll
    for (int j = 0; j < N; ++j) a = max(a, __float_as_uint(v[j]) & 0x7fffffffu);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) a = max(a, uint32_t(__shfl_xor(int(a), off, 64)));
  if ((t & 63) == 0) most[t >> 6] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) a = max(a, most[i]);
  const int byte = ckpt_scale_byte(a, MUON_CKPT_E4M3);
  const float down = ckpt_down(byte);
  if (t == 0) p.scale[which * bc * br + block] = uint8_t(byte);

  const int64_t q_pitch = int64_t(bc) * SIDE, qt_pitch = int64_t(br) * SIDE;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int in = i * ROWS + t / LANES;
    float v[N];
    unpack_raw<BF16>(raw[i], v);
    uint32_t q[N / 4];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      // only at the largest exponent may a value be out of range: it saturates
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __builtin_amdgcn_fmed3f(v[4 * j + k] * down, -448.f, 448.f);
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
      q[j] = byte == 255 ? 0u : uint32_t(w);
      *reinterpret_cast<uint32_t*>(tile + in * PITCH + col + 4 * j) = q[j];
    }
    if (r0 + in < p.rows) {
      uint8_t* to = p.q + (which * p.rows + r0 + in) * q_pitch + c0 + col;
      if constexpr (N == 8)
        *reinterpret_cast<uint2*>(to) = uint2{q[0], q[1]};
      else
        *reinterpret_cast<uint32_t*>(to) = q[0];
    }
  }
  __syncthreads();
  // Exchanged: a thread turns 4 x 4 bytes at a time; 8 lanes write a run of 128.
#pragma unroll
  for (int i = 0; i < SIDE / 4 / (kThreads / 8); ++i) {
    const int c = (i * (kThreads / 8) + t / 8) * 4, r = t % 8 * 16;
    uint32_t o[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const uint32_t*>(tile + (r + 4 * j + k) * PITCH + c);
      const uint32_t a01 = __builtin_amdgcn_perm(m[1], m[0], 0x05010400u), a23 = __builtin_amdgcn_perm(m[3], m[2], 0x05010400u);
      const uint32_t b01 = __builtin_amdgcn_perm(m[1], m[0], 0x07030602u), b23 = __builtin_amdgcn_perm(m[3], m[2], 0x07030602u);
      o[0][j] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
      o[1][j] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
      o[2][j] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
      o[3][j] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + c + k < p.cols)
        *reinterpret_cast<u32x4_t*>(p.q_t + (which * p.cols + c0 + c + k) * qt_pitch + r0 + r) =
            u32x4_t{o[k][0], o[k][1], o[k][2], o[k][3]};
  }
}

}  // namespace

hipError_t launch_weight_quantize(const Weight8& p, bool bf16, hipStream_t s) {
  const int64_t blocks = p.count * ((p.rows + SIDE - 1) / SIDE) * ((p.cols + SIDE - 1) / SIDE);
  const auto kernel = bf16 ? (p.cols >= 8 ? quantize_kernel<true, true> : quantize_kernel<true, false>)
                           : (p.cols >= 4 ? quantize_kernel<false, true> : quantize_kernel<false, false>);
  hipLaunchKernelGGL(kernel, dim3(unsigned(blocks)), dim3(kThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace muon
