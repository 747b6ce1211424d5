// Layer norm over the columns of a tokens x cols matrix, forward and backward.
//
//   forward   mean = avg x, rstd = (avg (x - mean)^2 + eps)^-1/2,
//             y = (x - mean) rstd gain + bias
//   backward  xhat = (x - mean) rstd, a = gain dy,
//             dx = rstd (a - avg a - xhat avg(a xhat)),
//             dgain = sum_t dy xhat, dbias = sum_t dy
//
// HBM-bound: each matrix is read or written once; a row stays in registers
// between its sums and its outputs.  LPR lanes hold a row, V values each: a
// wave for rows up to 2048 columns (its sums need no LDS), 256 lanes up to
// 8192 and 1024 above.  Statistics and sums are float32: the variance is
// summed from the centred values, so nothing cancels.
#include "layer_internal.h"

namespace muon {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sum of K values over the LPR lanes of a row, the same in every lane.  `red`
// holds K floats per wave of the block; a caller's consecutive calls use
// different arrays, so that one barrier per call is enough.
template <int LPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x >> 6, first = wave / W * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[wave * K + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[(first + w) * K + k];
      v[k] = s;
    }
  }
}

// Rows of a block of the forward pass, and of the backward pass.
template <int LPR>
constexpr int fwd_threads() { return LPR < 256 ? 256 : LPR; }
template <int LPR>
constexpr int bwd_threads() { return LPR < 1024 ? 512 : 1024; }

template <bool BF16, int LPR, int V>
__global__ __launch_bounds__(fwd_threads<LPR>()) void ln_forward_kernel(const LnForward p) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  constexpr int N = R::N, NV = V / N, RPB = fwd_threads<LPR>() / LPR;
  __shared__ float red[2][fwd_threads<LPR>() / 64];
  const int lane = threadIdx.x % LPR;
  // every lane of a block makes the same number of passes (barriers inside)
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.tokens;
       row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + threadIdx.x / LPR;
    const bool live = row < p.tokens;
    const T* x = static_cast<const T*>(p.x) + (live ? row : p.tokens - 1) * p.ldx;
    float v[NV][N];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_vec<BF16>(x, (j * LPR + lane) * N, p.cols, v[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += v[j][i];
    }
    row_sum<LPR, 1>(s, red[0]);
    const float mean = s[0] * p.inv_cols;
    if (p.xc.fmt >= 0 && live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ckpt_store<N>(p.xc, row, (j * LPR + lane) * N, p.cols, v[j]);
    }
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int left = p.cols - (j * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[j][i] = i < left ? v[j][i] - mean : 0.f;
        q[0] = __builtin_fmaf(v[j][i], v[j][i], q[0]);
      }
    }
    row_sum<LPR, 1>(q, red[1]);
    const float rstd = 1.f / __builtin_sqrtf(q[0] * p.inv_cols + p.eps);
    if (!live) continue;
    if (lane == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * LPR + lane) * N;
      float g[N], b[N];
      load_params<N>(p.gain, p.param_bf16, col, p.cols, g);
      if (p.bias) {
        load_params<N>(p.bias, p.param_bf16, col, p.cols, b);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) b[i] = 0.f;
      }
      float o[N];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(v[j][i] * rstd, g[i], b[i]);
      store_vec<BF16>(y, col, p.cols, o);
      if (p.yc.fmt >= 0) {
        // the checkpoint holds y as the next layer reads it
        const int left = p.cols - col;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if constexpr (BF16) o[i] = bf2f(f2bf(o[i]));
          if (i >= left) o[i] = 0.f;
        }
        ckpt_store<N>(p.yc, row, col, p.cols, o);
      }
    }
  }
}

template <bool BF16, int LPR, int V>
__global__ __launch_bounds__(bwd_threads<LPR>()) void ln_backward_kernel(const LnBackward p) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  constexpr int N = R::N, NV = V / N, NT = bwd_threads<LPR>(), RPB = NT / LPR;
  __shared__ float red[2][2 * NT / 64];
  __shared__ float join[RPB > 1 ? RPB : 1][RPB > 1 ? LPR * N : 1];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float dg[NV][N], db[NV][N], gain[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_params<N>(p.gain, p.param_bf16, (j * LPR + lane) * N, p.cols, gain[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) dg[j][i] = db[j][i] = 0.f;
  }
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.tokens;
       row0 += int64_t(gridDim.x) * RPB) {
    const int64_t row = row0 + sub;
    const bool live = row < p.tokens;
    const int64_t at = live ? row : p.tokens - 1;
    const float mean = p.mean[at], rstd = p.rstd[at];
    const T* dy = static_cast<const T*>(p.dy) + at * p.lddy;
    float a[NV][N], xh[NV][N];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * LPR + lane) * N;
      load_vec<BF16>(dy, col, p.cols, a[j]);
      if (p.x)
        load_vec<BF16>(static_cast<const T*>(p.x) + at * p.ldx, col, p.cols, xh[j]);
      else
        ckpt_load<N>(p.xc, at, col, xh[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int left = p.cols - (j * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = a[j][i];
        const float h = i < left ? (xh[j][i] - mean) * rstd : 0.f;
        if (live) {
          dg[j][i] = __builtin_fmaf(d, h, dg[j][i]);
          db[j][i] += d;
        }
        xh[j][i] = h;
        a[j][i] = d * gain[j][i];
        s[0] += a[j][i];
        s[1] = __builtin_fmaf(a[j][i], h, s[1]);
      }
    }
    row_sum<LPR, 2>(s, red[turn]);
    turn ^= 1;
    if (live) {
      const float c0 = s[0] * p.inv_cols, c1 = s[1] * p.inv_cols;
      T* dx = static_cast<T*>(p.dx) + row * p.cols;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = rstd * (a[j][i] - c0 - xh[j][i] * c1);
        store_vec<BF16>(dx, (j * LPR + lane) * N, p.cols, o);
      }
    }
  }
  // One row of partial sums per block: the block's rows are added in order.
  float* out = p.partial + int64_t(blockIdx.x) * 2 * p.cols;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float(&acc)[N] = k ? db[j] : dg[j];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) join[sub][lane * N + i] = acc[i];
        __syncthreads();
        for (int c = threadIdx.x; c < LPR * N; c += NT) {
          float t = 0.f;
#pragma unroll
          for (int r = 0; r < RPB; ++r) t += join[r][c];
          const int col = j * LPR * N + c;
          if (col < p.cols) out[k * p.cols + col] = t;
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int col = (j * LPR + lane) * N + i;
          if (col < p.cols) out[k * p.cols + col] = acc[i];
        }
      }
    }
  }
}

// Sums the blocks' rows of partial sums: 32 columns by 32 rows of threads per
// block (grid.y: gain, bias), each thread every 32nd row in order.
__global__ __launch_bounds__(1024) void ln_params_kernel(const LnBackward p) {
  __shared__ float part[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + tx, k = blockIdx.y;
  float t = 0.f;
  if (col < p.cols) {
    const float* in = p.partial + int64_t(k) * p.cols + col;
#pragma unroll 4
    for (int b = ty; b < p.blocks; b += 32) t += in[int64_t(b) * 2 * p.cols];
  }
  part[ty][tx] = t;
  __syncthreads();
  if (ty == 0 && col < p.cols) {
    t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][tx];
    void* out = k ? p.dbias : p.dgain;
    if (p.param_bf16) {
      uint16_t* o = static_cast<uint16_t*>(out) + col;
      *o = f2bf(p.accumulate ? bf2f(*o) + t : t);
    } else {
      float* o = static_cast<float*>(out) + col;
      *o = p.accumulate ? *o + t : t;
    }
  }
}

// Lanes and values per lane of a row.
struct RowShape {
  int lpr, v;
};
RowShape row_shape(int64_t cols) {
  const int lpr = cols <= 2048 ? 64 : cols <= 8192 ? 256 : 1024;
  const int64_t per_lane = (cols + lpr - 1) / lpr;
  return {lpr, per_lane <= 8 ? 8 : per_lane <= 16 ? 16 : 32};
}

template <bool BF16, int LPR, int V>
hipError_t forward(const LnForward& p, hipStream_t s) {
  constexpr int NT = fwd_threads<LPR>(), RPB = NT / LPR;
  const int64_t want = (p.tokens + RPB - 1) / RPB;
  const int64_t cap = 256 * (2048 / NT);   // the waves that fill the chip
  hipLaunchKernelGGL((ln_forward_kernel<BF16, LPR, V>), dim3(unsigned(want < cap ? want : cap)),
                     dim3(NT), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int LPR, int V>
hipError_t backward(const LnBackward& p, hipStream_t s) {
  hipLaunchKernelGGL((ln_backward_kernel<BF16, LPR, V>), dim3(unsigned(p.blocks)),
                     dim3(bwd_threads<LPR>()), 0, s, p);
  return hipGetLastError();
}

}  // namespace

// Two blocks of 512 threads per CU, or one of 1024.
int ln_backward_blocks(int64_t tokens, int64_t cols) {
  const int lpr = row_shape(cols).lpr, nt = lpr < 1024 ? 512 : 1024;
  const int64_t want = (tokens + nt / lpr - 1) / (nt / lpr);
  const int64_t cap = 256 * (1024 / nt);
  return int(want < cap ? want : cap);
}

#define MUON_LN_SHAPES(CALL)                                   \
  const RowShape r = row_shape(p.cols);                        \
  if (r.lpr == 64) {                                           \
    if (r.v == 8) return bf16 ? CALL<true, 64, 8>(p, s) : CALL<false, 64, 8>(p, s);     \
    if (r.v == 16) return bf16 ? CALL<true, 64, 16>(p, s) : CALL<false, 64, 16>(p, s);  \
    return bf16 ? CALL<true, 64, 32>(p, s) : CALL<false, 64, 32>(p, s);                 \
  }                                                            \
  if (r.lpr == 256) {                                          \
    if (r.v == 16) return bf16 ? CALL<true, 256, 16>(p, s) : CALL<false, 256, 16>(p, s); \
    return bf16 ? CALL<true, 256, 32>(p, s) : CALL<false, 256, 32>(p, s);               \
  }                                                            \
  if (r.v == 16) return bf16 ? CALL<true, 1024, 16>(p, s) : CALL<false, 1024, 16>(p, s); \
  return bf16 ? CALL<true, 1024, 32>(p, s) : CALL<false, 1024, 32>(p, s)

hipError_t launch_ln_forward(const LnForward& p, bool bf16, hipStream_t s) {
  MUON_LN_SHAPES(forward);
}
hipError_t launch_ln_backward(const LnBackward& p, bool bf16, hipStream_t s) {
  MUON_LN_SHAPES(backward);
}

hipError_t launch_ln_params(const LnBackward& p, hipStream_t s) {
  hipLaunchKernelGGL(ln_params_kernel, dim3(unsigned((p.cols + 31) / 32), p.dbias ? 2 : 1),
                     dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace muon
