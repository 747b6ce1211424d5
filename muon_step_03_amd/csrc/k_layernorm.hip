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
// 4096 and 1024 above.  Statistics and sums are float32: the variance is
// summed from the centred values, so nothing cancels.  Measured on one MI355X
// (a 1 GiB copy: 5.45 TB/s): 16384 x 1024 bf16, forward with a checkpoint of y
// 17.8 us (4.8 TB/s), backward from one 17.3 and 3.7 for the parameters' sums;
// 16384 x 4096 bf16, forward 46 (5.9 TB/s), backward 84 (4.8); 16384 x 1411
// float32, forward 35 (5.3), backward 51 (5.4).
#include "layer_internal.h"

namespace muon {
namespace {

// Sum over 32 or 64 lanes, the same in every lane: exchanges within rows of
// 16 lanes, then swaps of rows and of halves (no LDS).
template <int LANES>
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kMirror8>(__float_as_uint(v)));
  v += __uint_as_float(dpp<kMirror16>(__float_as_uint(v)));
  const uint32_t u = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  if constexpr (LANES == 64) {
    const uint32_t t = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(t, t, false, false);
    v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  }
  return v;
}

// Sum of K values over the LPR lanes of a row, the same in every lane.  `red`
// holds K floats per wave of the block; a caller's consecutive calls use
// different arrays, so that one barrier per call is enough.
template <int LPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum<LPR == 32 ? 32 : 64>(v[k]);
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

// s / n with inv = 1 / n rounded: the quotient is corrected by its remainder,
// which an infinite one does not have.
__device__ __forceinline__ float over(float s, float n, float inv) {
  const float q = s * inv;
  const float c = __builtin_fmaf(__builtin_fmaf(-q, n, s), inv, q);
  return __builtin_fabsf(q) < __builtin_inff() ? c : q;
}

// 1 / sqrt(v) within half a step and a little: the hardware's estimate (one
// step off) and a Newton correction, its residual in fused multiply-adds.
// Tiny v is scaled up first (the estimate flushes subnormals); zero and
// infinity give infinity and zero.
__device__ __forceinline__ float inv_sqrt(float v) {
  const bool tiny = v < 0x1p-96f;
  if (tiny) v *= 0x1p96f;
  float r = __builtin_amdgcn_rsqf(v);
  const float t = v * r, d = __builtin_fmaf(v, r, -t);
  const float e = __builtin_fmaf(-d, r, __builtin_fmaf(-t, r, 1.f));   // 1 - v r^2
  const float c = __builtin_fmaf(0.5f * r, e, r);
  r = r > 0.f && r < __builtin_inff() ? c : r;
  return tiny ? r * 0x1p48f : r;
}

// Whether a lane holds its gains (and biases) and the next row's loads in
// registers: not for the longest rows, whose 16 and 32 values a lane leave no
// room for them in the 128 registers of a 1024-thread block.
template <int LPR, int V>
constexpr bool hold() { return LPR < 1024 || V < 16; }

// Threads of a block of the forward pass, and of the backward pass.
template <int LPR>
constexpr int fwd_threads() { return LPR < 256 ? 256 : LPR; }
template <int LPR>
constexpr int bwd_threads() { return LPR < 1024 ? 512 : 1024; }

// Whether two blocks of the backward pass share a CU: their threads do, and the
// registers (128 each) hold all but float32 rows of 16 values a lane.
constexpr bool bwd_two_blocks(bool bf16, int lpr, int v) { return lpr < 1024 && (bf16 || v < 16); }

// A sum of a parameter's gradient, to where it belongs.
__device__ __forceinline__ void store_param(const LnBackward& p, int k, int col, float t) {
  void* out = k ? p.dbias : p.dgain;
  if (!out) return;
  if (p.param_bf16) {
    uint16_t* o = static_cast<uint16_t*>(out) + col;
    *o = f2bf(p.accumulate ? bf2f(*o) + t : t);
  } else {
    float* o = static_cast<float*>(out) + col;
    *o = p.accumulate ? *o + t : t;
  }
}

// END: how rows end (with a whole vector where cols is a multiple of N).
template <bool BF16, RowEnd END, int LPR, int V>
__global__ __launch_bounds__(fwd_threads<LPR>()) void ln_forward_kernel(const LnForward p) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  constexpr int N = R::N, NV = V / N, RPB = fwd_threads<LPR>() / LPR;
  __shared__ float red[2][fwd_threads<LPR>() / 64];
  const int lane = threadIdx.x % LPR;
  const float n = float(p.cols), inv = 1.f / n;
  constexpr bool HOLD = hold<LPR, V>();
  float gain[HOLD ? NV : 1][N], bias[HOLD ? NV : 1][N];
  auto load_affine = [&](int j, float (&g)[N], float (&b)[N]) {
    load_params<N>(p.gain, p.param_bf16, (j * LPR + lane) * N, p.cols, g);
#pragma unroll
    for (int i = 0; i < N; ++i) b[i] = 0.f;
    if (p.bias) load_params<N>(p.bias, p.param_bf16, (j * LPR + lane) * N, p.cols, b);
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_affine(j, gain[j], bias[j]);
  }
  const int64_t stride = int64_t(gridDim.x) * RPB;
  auto load = [&](int64_t row, u32x4_t (&w)[NV]) {
    const T* x = static_cast<const T*>(p.x) + (row < p.tokens ? row : p.tokens - 1) * p.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j) w[j] = load_ahead<BF16, END>(x, (j * LPR + lane) * N, p.cols);
  };
  u32x4_t next[HOLD ? NV : 1];
  const int64_t first = int64_t(blockIdx.x) * RPB + threadIdx.x / LPR;
  if constexpr (HOLD) load(first, next);
  // every lane of a block makes the same number of passes (barriers inside);
  // the next row is on its way while one is worked on
  for (int64_t row = first; row - threadIdx.x / LPR < p.tokens; row += stride) {
    const bool live = row < p.tokens;
    u32x4_t w[NV];
    if constexpr (HOLD) {
#pragma unroll
      for (int j = 0; j < NV; ++j) w[j] = next[j];
      if (row - threadIdx.x / LPR + stride < p.tokens) load(row + stride, next);
    } else {
      load(row, w);
    }
    float v[NV][N];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      settle<BF16, END>(w[j], (j * LPR + lane) * N, p.cols);
      unpack_raw<BF16>(w[j], v[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += v[j][i];
    }
    row_sum<LPR, 1>(s, red[0]);
    const float mean = over(s[0], n, inv);
    if (p.xc.fmt >= 0 && live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ckpt_store<BF16>(p.xc, row, (j * LPR + lane) * N, p.cols, w[j]);
    }
    float q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int left = p.cols - (j * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) v[j][i] -= mean;
      float t = 0.f;
      if constexpr (END != END_WHOLE) {
        if (left < N) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i >= left) v[j][i] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) t = __builtin_fmaf(v[j][i], v[j][i], t);
      q[0] += left > 0 ? t : 0.f;
    }
    row_sum<LPR, 1>(q, red[1]);
    const float rstd = inv_sqrt(over(q[0], n, inv) + p.eps);
    if (!live) continue;
    if (lane == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * LPR + lane) * N;
      float o[N];
      if constexpr (!HOLD) load_affine(j, gain[0], bias[0]);
      const int k = HOLD ? j : 0;
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(v[j][i] * rstd, gain[k][i], bias[k][i]);
      u32x4_t out = pack_raw<BF16>(o);
      store_raw<BF16, END == END_WHOLE>(y, col, p.cols, out);
      // the checkpoint holds y as the next layer reads it
      if (p.yc.fmt >= 0) {
        if (col >= p.cols) out = u32x4_t{0, 0, 0, 0};
        ckpt_store<BF16>(p.yc, row, col, p.cols, out);
      }
    }
  }
}

// CK: x from its checkpoint.
template <bool BF16, RowEnd END, bool CK, int LPR, int V>
__global__ __launch_bounds__(bwd_threads<LPR>(), bwd_two_blocks(BF16, LPR, V) ? 4 : 1)
void ln_backward_kernel(const LnBackward p) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  constexpr int N = R::N, NV = V / N, NT = bwd_threads<LPR>(), RPB = NT / LPR;
  __shared__ float red[2][2 * NT / 64];
  __shared__ float join[RPB > 1 ? RPB : 1][RPB > 1 ? LPR * N : 1];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const float n = float(p.cols), inv = 1.f / n;
  constexpr bool HOLD = hold<LPR, V>();
  float dg[NV][N], db[NV][N], gain[HOLD ? NV : 1][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (HOLD) load_params<N>(p.gain, p.param_bf16, (j * LPR + lane) * N, p.cols, gain[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) dg[j][i] = db[j][i] = 0.f;
  }
  // A row's loads; the next row's are on their way while one is worked on.
  struct Row {
    u32x4_t dy[NV];
    u32x4_t x[CK ? 1 : NV];
    CkptVec<N> c[CK ? NV : 1];
    float mean, rstd;
  } next;
  auto load = [&](int64_t row, Row& r) {
    const int64_t at = row < p.tokens ? row : p.tokens - 1;
    r.mean = p.mean[at];
    r.rstd = p.rstd[at];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int col = (j * LPR + lane) * N;
      r.dy[j] = load_ahead<BF16, END>(static_cast<const T*>(p.dy) + at * p.lddy, col, p.cols);
      if constexpr (CK)
        r.c[j] = ckpt_load<N>(p.xc, at, col);
      else
        r.x[j] = load_ahead<BF16, END>(static_cast<const T*>(p.x) + at * p.ldx, col, p.cols);
    }
  };
  const int64_t stride = int64_t(gridDim.x) * RPB;
  if constexpr (HOLD) load(int64_t(blockIdx.x) * RPB + sub, next);
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPB; row0 < p.tokens; row0 += stride) {
    const int64_t row = row0 + sub;
    const bool live = row < p.tokens;
    Row cur;
    if constexpr (HOLD) {
      cur = next;
      if (row0 + stride < p.tokens) load(row + stride, next);
    } else {
      load(row, cur);
    }
    float a[NV][N], xh[NV][N];
    float s[2] = {0.f, 0.f};
    // past the row's end dy is zero, and so is every term of the sums
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      settle<BF16, END>(cur.dy[j], (j * LPR + lane) * N, p.cols);
      unpack_raw<BF16>(cur.dy[j], a[j]);
      if constexpr (CK) {
        ckpt_values<N>(cur.c[j], p.xc.fmt, xh[j]);
      } else {
        settle<BF16, END>(cur.x[j], (j * LPR + lane) * N, p.cols);
        unpack_raw<BF16>(cur.x[j], xh[j]);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) xh[j][i] = (xh[j][i] - cur.mean) * cur.rstd;
      if (live) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dg[j][i] = __builtin_fmaf(a[j][i], xh[j][i], dg[j][i]);
          db[j][i] += a[j][i];
        }
      }
      const int k = HOLD ? j : 0;
      if constexpr (!HOLD) load_params<N>(p.gain, p.param_bf16, (j * LPR + lane) * N, p.cols, gain[0]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        a[j][i] *= gain[k][i];
        s[0] += a[j][i];
        s[1] = __builtin_fmaf(a[j][i], xh[j][i], s[1]);
      }
    }
    row_sum<LPR, 2>(s, red[turn]);
    turn ^= 1;
    if (live) {
      const float c0 = over(s[0], n, inv), c1 = over(s[1], n, inv);
      T* dx = static_cast<T*>(p.dx) + row * p.cols;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = cur.rstd * (a[j][i] - c0 - xh[j][i] * c1);
        store_raw<BF16, END == END_WHOLE>(dx, (j * LPR + lane) * N, p.cols, pack_raw<BF16>(o));
      }
    }
  }
  // One row of partial sums per block, the block's rows added in order; a
  // single block's are the gradients.
  float* out = p.partial + int64_t(blockIdx.x) * 2 * p.cols;
  auto put = [&](int k, int col, float t) {
    if (col >= p.cols) return;
    if (p.blocks == 1)
      store_param(p, k, col, t);
    else
      out[k * p.cols + col] = t;
  };
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
          put(k, j * LPR * N + c, t);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) put(k, (j * LPR + lane) * N + i, acc[i]);
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
    // 16 loads in flight whatever the number of rows (500 rows of 1411: 7.5 us
    // when the last ones were loaded one by one)
    for (int b0 = ty; b0 < p.blocks; b0 += 512) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int b = b0 + 32 * i;
        v[i] = in[int64_t(b < p.blocks ? b : b0) * 2 * p.cols];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) t += b0 + 32 * i < p.blocks ? v[i] : 0.f;
    }
  }
  part[ty][tx] = t;
  __syncthreads();
  if (ty == 0 && col < p.cols) {
    t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][tx];
    store_param(p, k, col, t);
  }
}

// Lanes and values per lane of a row: the least that hold it.  Three vectors a
// lane in half a wave fit rows of 768 (forward 20.1 -> 15.7 us at 16384 rows in
// bf16), but cost the backward more registers than they save lanes (20.4
// -> 23.2); a wave of three vectors a lane for 1411 float32 columns was slower
// than 256 lanes of two in both (18.9 against 17.1, 24.0 against 19.8).
struct RowShape {
  int lpr, v;
};
RowShape row_shape(int64_t cols, bool backward) {
  constexpr RowShape all[] = {{32, 8}, {64, 8}, {32, 24}, {64, 16}, {256, 8},
                              {256, 16}, {1024, 8}, {1024, 16}, {1024, 32}};
  for (const RowShape& r : all)
    if (cols <= r.lpr * r.v && !(backward && r.v == 24)) return r;
  return all[8];
}

template <bool BF16, int LPR, int V>
hipError_t forward(const LnForward& p, hipStream_t s) {
  constexpr int NT = fwd_threads<LPR>(), RPB = NT / LPR;
  const int64_t want = (p.tokens + RPB - 1) / RPB;
  const int64_t cap = 256 * (2048 / NT);   // the waves that fill the chip
  const dim3 grid(unsigned(want < cap ? want : cap)), block(NT);
  const RowEnd end = row_end(p.cols, RowVec<BF16>::N);
  if (end == END_WHOLE)
    hipLaunchKernelGGL((ln_forward_kernel<BF16, END_WHOLE, LPR, V>), grid, block, 0, s, p);
  else if (end == END_INSIDE)
    hipLaunchKernelGGL((ln_forward_kernel<BF16, END_INSIDE, LPR, V>), grid, block, 0, s, p);
  else if constexpr (LPR * V == 256)   // the shape of the shortest rows
    hipLaunchKernelGGL((ln_forward_kernel<BF16, END_SHORT, LPR, V>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <bool BF16, RowEnd END, int LPR, int V>
hipError_t backward_of(const LnBackward& p, hipStream_t s) {
  const dim3 grid(unsigned(p.blocks)), block(bwd_threads<LPR>());
  if (p.x)
    hipLaunchKernelGGL((ln_backward_kernel<BF16, END, false, LPR, V>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((ln_backward_kernel<BF16, END, true, LPR, V>), grid, block, 0, s, p);
  return hipGetLastError();
}
template <bool BF16, int LPR, int V>
hipError_t backward(const LnBackward& p, hipStream_t s) {
  const RowEnd end = row_end(p.cols, RowVec<BF16>::N);
  if (end == END_WHOLE) return backward_of<BF16, END_WHOLE, LPR, V>(p, s);
  if (end == END_INSIDE) return backward_of<BF16, END_INSIDE, LPR, V>(p, s);
  if constexpr (LPR * V == 256) return backward_of<BF16, END_SHORT, LPR, V>(p, s);   // the shortest rows
  return hipErrorInvalidValue;
}

}  // namespace

// The blocks that the CUs hold at once (a third one would only wait: float32
// rows of 1024, 4099 of them, 14.9 us with 512 blocks, one per CU at a time, 11.6
// with 256).  A few passes of a block are left to a single one, which spares the
// second launch.  Measured in bf16, eager calls in a row and one of a captured
// graph, one block against two launches:
//   12 rows of 768, 2 passes     13.5 and 4.8 us against 17.8 and 6.2
//   64 rows of 768, 8 passes     13.4 and 11.0   against 17.9 and 6.5
//   16 rows of 4096, 8 passes    14.8 and 14.8   against 17.5 and 8.1
//   3 rows of 8192               13.0 and 12.2   against 17.3 and 12.6
//   2 rows of 16384              22.1 and 22.0   against 23.8 and 23.2
//   3 rows of 16384              25.0 and 24.9   against 23.7 and 23.3
//   2 rows of 32768              56.9 and 56.8   against 52.2 and 51.8
// Up to 4096 columns 8 passes hide behind the host's time for a call; a captured
// graph, where more than 3 lose, would sum in another order than the eager call if
// it took two launches.  Above, where a pass is one row, one block is taken while it
// is ahead in both.
int64_t one_block_passes(int64_t cols) { return cols <= 4096 ? 8 : 1 + 16384 / cols; }
int ln_backward_blocks(int64_t tokens, int64_t cols, bool bf16) {
  const RowShape r = row_shape(cols, true);
  const int nt = r.lpr < 1024 ? 512 : 1024, rows = nt / r.lpr;
  const int64_t want = (tokens + rows - 1) / rows;
  const int64_t cap = bwd_two_blocks(bf16, r.lpr, r.v) ? 512 : 256;
  return int(want < 1 ? 0 : want <= one_block_passes(cols) ? 1 : want < cap ? want : cap);
}

#define MUON_LN_SHAPE(CALL, LPR, V) \
  if (r.lpr == LPR && r.v == V) return bf16 ? CALL<true, LPR, V>(p, s) : CALL<false, LPR, V>(p, s)
#define MUON_LN_SHAPES(CALL)              \
  MUON_LN_SHAPE(CALL, 32, 8);             \
  MUON_LN_SHAPE(CALL, 64, 8);             \
  MUON_LN_SHAPE(CALL, 64, 16);            \
  MUON_LN_SHAPE(CALL, 256, 8);            \
  MUON_LN_SHAPE(CALL, 256, 16);           \
  MUON_LN_SHAPE(CALL, 1024, 8);           \
  MUON_LN_SHAPE(CALL, 1024, 16);          \
  MUON_LN_SHAPE(CALL, 1024, 32);          \
  return hipErrorInvalidValue

hipError_t launch_ln_forward(const LnForward& p, bool bf16, hipStream_t s) {
  const RowShape r = row_shape(p.cols, false);
  MUON_LN_SHAPE(forward, 32, 24);
  MUON_LN_SHAPES(forward);
}
hipError_t launch_ln_backward(const LnBackward& p, bool bf16, hipStream_t s) {
  const RowShape r = row_shape(p.cols, true);
  MUON_LN_SHAPES(backward);
}

hipError_t launch_ln_params(const LnBackward& p, hipStream_t s) {
  hipLaunchKernelGGL(ln_params_kernel, dim3(unsigned((p.cols + 31) / 32), p.dbias ? 2 : 1),
                     dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace muon
