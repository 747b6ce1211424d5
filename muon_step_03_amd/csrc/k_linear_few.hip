// The linear products along a weight's rows for few tokens per matrix: bound by
// reading the weights once.
//
// A block of 4 waves computes 16 outputs for up to 16 tokens.  The waves take k by
// turns, each lane loading its part of the 16 x 16 matrix instructions' operands
// straight to registers, many steps at once, and add their sums through LDS at
// the end.  A step is 128 bytes of a row, two chunks of 16 per lane: side by side,
// an order of k that is the same for both operands; for e4m3 64 bytes apart,
// where the instruction wants them for its scales.  Rows start at any element;
// what follows a row's end is zero (e4m3: the padding of the weight).
//
// Measured on one MI355X, launch included: a token of 5632 x 2048 7.3 us from e4m3
// (11.5 MB), 9.2 from bf16; of 4096 x 1024 5.6 and 6.3.
#include <algorithm>

#include "linear_device.h"

namespace muon {
namespace {

constexpr int THREADS = 256, WAVES = THREADS / 64, OUT = 16, TOKENS = 16;
constexpr int CHUNKS = 2, AT_ONCE = 4;     // chunks per lane and step, steps in flight per wave

template <LinearType TYPE>
__global__ __launch_bounds__(THREADS) void linear_few_kernel(const Linear p, int tiles_n) {
  constexpr bool E4M3 = TYPE >= LIN_E4M3, BF16 = TYPE == LIN_BF16;
  constexpr int ES = TYPE == LIN_BF16 ? 2 : TYPE == LIN_F32 ? 4 : 1, STEP = ROWB / ES;
  __shared__ int bounds_lds[kBoundsWords];
  __shared__ float sums[WAVES][TOKENS][OUT + 1];
  Bounds bounds{};
  bounds.tiles = cdiv_d(int(p.tokens), TOKENS);
  if (p.offsets) bounds = find_bounds<THREADS, true>(p, TOKENS, (LDS_AS int*)bounds_lds);
  const int64_t id = xcd_order(blockIdx.x, uint32_t(bounds.tiles) * tiles_n);
  if (id < 0) return;
  const Place at = place_of(p, bounds, TOKENS, tiles_n, int(id));
  const int t = threadIdx.x, lane = t & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int t0 = at.begin + at.tm * TOKENS, n0 = at.tn * OUT;

  f32x4_t acc = {0, 0, 0, 0};
  if (at.e >= 0) {
    // rows past the last output or token repeat it: what they give is not stored
    const char* w = static_cast<const char*>(p.W) + at.e * p.w_stride + int64_t(min(n0 + r, p.n - 1)) * p.ldw;
    const int64_t row = min(t0 + r, at.end - 1);
    const char* x = static_cast<const char*>(p.x) + row * p.ldx;
    const uint8_t *xs = nullptr, *ws = nullptr;
    if constexpr (E4M3) {
      xs = p.x_scale + row * p.xs_pitch;
      ws = p.w_scale + at.e * p.ws_stride + int64_t(n0 / SIDE) * p.ws_row;
    }

    struct Step {
      u32x4_t w[CHUNKS], x[CHUNKS];
      uint32_t ws, xs;
    };
    auto load = [&](Step& s, int k) __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        if constexpr (E4M3) {
          const int64_t off = int64_t(k) * ROWB + c * 64 + g * 16;
          s.w[c] = *reinterpret_cast<const u32x4_t*>(w + off);
          s.x[c] = *reinterpret_cast<const u32x4_t*>(x + min(off, p.ldx - 16));
        } else {
          using Raw = typename RowVec<BF16>::Raw;
          const int64_t off = int64_t(k) * ROWB + g * 32 + c * 16;
          const Raw u = *reinterpret_cast<const Raw*>(w + off), v = *reinterpret_cast<const Raw*>(x + off);
          s.w[c] = u32x4_t{u[0], u[1], u[2], u[3]};
          s.x[c] = u32x4_t{v[0], v[1], v[2], v[3]};
        }
      }
      if constexpr (E4M3) {
        s.ws = ws[k * p.ws_col];
        s.xs = *reinterpret_cast<const uint32_t*>(xs + k * 4);
      }
    };
    // the step that crosses the row's end: its vectors are loaded from the row's
    // last elements and shifted down (rows shorter than a vector: one by one)
    auto load_last = [&](Step& s, int k, int left) __attribute__((always_inline)) {
      constexpr int N = RowVec<BF16>::N;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const int in = g * 2 * N + c * N, from = k * STEP + in, by = max(in + N - left, 0);
        auto vec = [&](const char* base) __attribute__((always_inline)) {
          if (p.k < N) return load_raw<BF16>(base, from, p.k);
          using Raw = typename RowVec<BF16>::Raw;
          const Raw v = *reinterpret_cast<const Raw*>(base + int64_t(min(from, p.k - N)) * ES);
          u32x4_t o = {v[0], v[1], v[2], v[3]};
          shift_down<BF16>(o, by);
          return o;
        };
        s.w[c] = vec(w);
        s.x[c] = vec(x);
      }
    };
    auto multiply = [&](const Step& s) __attribute__((always_inline)) {
      if constexpr (TYPE == LIN_E4M3) {
        // a lane's first chunk is of block g / 2, its second of 2 + g / 2; the
        // instruction takes the scale of block b from the lanes of group b
        auto both = [](const u32x4_t& lo, const u32x4_t& hi) {
          return i32x8_t{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                         int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
        };
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(both(s.w[0], s.w[1]), both(s.x[0], s.x[1]), acc, 0, 0,
                                                               0, int(s.ws), 0, int(s.xs >> (8 * g)));
        return;
      }
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        if constexpr (TYPE == LIN_BF16) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, s.w[c]),
                                                        __builtin_bit_cast(bf16x8_t, s.x[c]), acc, 0, 0, 0);
        } else if constexpr (TYPE == LIN_F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(s.w[c][i]), __uint_as_float(s.x[c][i]), acc,
                                                       0, 0, 0);
        } else {
          bf16x8_t wv[2], xv[2];
          widen(s.w[c], s.ws, wv);
          widen(s.x[c], s.xs >> (8 * (2 * c + (g >> 1))) & 0xff, xv);
#pragma unroll
          for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[h], xv[h], acc, 0, 0, 0);
        }
      }
    };

    const int whole = E4M3 ? cdiv_d(p.k, STEP) : p.k / STEP;
    const int left = E4M3 ? 0 : p.k - whole * STEP;     // elements of the last, partial step
    Step s[AT_ONCE];
    int k = wave;
    for (; k + (AT_ONCE - 1) * WAVES < whole; k += AT_ONCE * WAVES) {
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) load(s[i], k + i * WAVES);
#pragma unroll
      for (int i = 0; i < AT_ONCE; ++i) multiply(s[i]);
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE - 1; ++i)
      if (k + i * WAVES < whole) load(s[i], k + i * WAVES);
#pragma unroll
    for (int i = 0; i < AT_ONCE - 1; ++i)
      if (k + i * WAVES < whole) multiply(s[i]);
    if constexpr (!E4M3) {
      if (left > 0 && wave == whole % WAVES) {
        load_last(s[0], whole, left);
        multiply(s[0]);
      }
    }
  }
  // lane l, register i of the block holds output 4 (l / 16) + i, token l % 16
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[wave][r][4 * g + i] = acc[i];
  __syncthreads();
  const int row = t / OUT, col = t % OUT;
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) v += sums[i][row][col];
  if (t0 + row < at.end && n0 + col < p.n) {
    const int64_t to = int64_t(t0 + row) * p.n + n0 + col;
    if (p.y_bf16)
      static_cast<uint16_t*>(p.y)[to] = f2bf(v);
    else
      static_cast<float*>(p.y)[to] = v;
  }
}

template <LinearType TYPE>
hipError_t launch_few(const Linear& p, hipStream_t s) {
  const int64_t tiles_n = (p.n + OUT - 1) / OUT;
  // of the matrices, only those with tokens have tiles, and the tokens of none
  const int64_t tiles_m = p.offsets ? p.tokens / TOKENS + std::min<int64_t>(p.count + 2, p.tokens)
                                    : (p.tokens + TOKENS - 1) / TOKENS;
  const dim3 grid(unsigned((tiles_m * tiles_n + 7) / 8 * 8));
  hipLaunchKernelGGL(linear_few_kernel<TYPE>, grid, dim3(THREADS), 0, s, p, int(tiles_n));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_few(const Linear& p, LinearType type, hipStream_t s) {
  switch (type) {
    case LIN_BF16: return launch_few<LIN_BF16>(p, s);
    case LIN_F32: return launch_few<LIN_F32>(p, s);
    case LIN_E4M3: return launch_few<LIN_E4M3>(p, s);
    default: return launch_few<LIN_E4M3_EXACT>(p, s);
  }
}

}  // namespace muon
