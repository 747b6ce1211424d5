// Structures and device helpers of the layer operators (layer norm,
// activation checkpoints, weight gradients) shared by their host file
// (layer_abi.hip) and kernels.
#pragma once

#include "muon_internal.h"

namespace muon {

// ------------------------------------------------------------- checkpoints
// A checkpoint as the kernels see it; fmt < 0: none.
struct Ckpt {
  uint8_t* q;
  uint8_t* scale;
  int64_t q_pitch, s_pitch;
  int fmt;
};

// Scale exponents: a block stands for q * 2^e, e >= kCkptEMin, so that the
// smallest step (2^-9 * 2^e for e4m3) is a normal float32 and bfloat16
// number; the largest e keeps the largest q finite.
constexpr int kCkptEMin = -117;
constexpr int kCkptEMaxE4m3 = 119, kCkptEMaxInt8 = 121;
constexpr uint32_t kInfBits = 0x7f800000u;

// Scale byte of a block whose largest magnitude has the bit pattern `a`
// (an infinity or NaN anywhere in the block makes a >= kInfBits): e + 127, e
// the smallest exponent with a <= 448 * 2^e = 1.75 * 2^(8+e) (e4m3) or
// 127 * 2^e = 1.984375 * 2^(6+e) (int8).
__device__ __forceinline__ int ckpt_scale_byte(uint32_t a, int fmt) {
  const int field = int(a >> 23);            // exponent + 127 (0: subnormal or zero)
  const int over = (a & 0x7fffffu) > (fmt == MUON_CKPT_E4M3 ? 0x600000u : 0x7e0000u) ? 1 : 0;
  int e = field - 127 - (fmt == MUON_CKPT_E4M3 ? 8 : 6) + over;
  e = e < kCkptEMin ? kCkptEMin : e;
  const int top = fmt == MUON_CKPT_E4M3 ? kCkptEMaxE4m3 : kCkptEMaxInt8;
  e = e > top ? top : e;
  return a >= kInfBits ? 255 : e + 127;
}

// The factor that brings a block into the format's range: 2^-e; 0 for a
// marked block, whose q are zeros.
__device__ __forceinline__ float ckpt_down(int byte) {
  return byte == 255 ? 0.f : __uint_as_float(uint32_t(254 - byte) << 23);
}
// The factor that brings it back: 2^e; NaN for a marked block (a NaN factor
// makes the whole block NaN), 0 for the padding's scale byte 0.
__device__ __forceinline__ float ckpt_up(int byte) {
  return __uint_as_float(byte == 255 ? 0x7fc00000u : uint32_t(byte) << 23);
}

// Four values -> four q bytes.  A marked block's values are not finite, so
// they are replaced, not multiplied, by zero.
__device__ __forceinline__ uint32_t ckpt_pack4(const float* v, float down, int fmt) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = down == 0.f ? 0.f : v[i] * down;
  if (fmt == MUON_CKPT_E4M3) {
    // only values that the largest exponent cannot hold are clamped
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = __builtin_amdgcn_fmed3f(s[i], -448.f, 448.f);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], w, true);
    return uint32_t(w);
  }
  // adding 1.5 * 2^23 leaves the integer, rounded half to even, in the low byte
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b[i] = __float_as_uint(__builtin_amdgcn_fmed3f(s[i], -127.f, 127.f) + 12582912.f) & 0xffu;
  return b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
}

// Four q bytes -> four values, exact.
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, float up, int fmt, float* v) {
  if (fmt == MUON_CKPT_E4M3) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    v[0] = lo[0] * up;
    v[1] = lo[1] * up;
    v[2] = hi[0] * up;
    v[3] = hi[1] * up;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = float(int(w << (24 - 8 * i)) >> 24) * up;
  }
}

// ------------------------------------------------------- rows of 16-byte vectors
// A vector of a row: 8 bf16 or 4 float32.  Rows start at any element, so the
// 16-byte accesses are only element-aligned (global memory takes them so).
template <bool BF16>
struct RowVec;
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
template <>
struct RowVec<true> {
  using T = uint16_t;
  using Raw = u32x4_a2;
  static constexpr int N = 8;
};
template <>
struct RowVec<false> {
  using T = float;
  using Raw = u32x4_a4;
  static constexpr int N = 4;
};

// Elements [col, col + N) of a row of `cols`, those past its end as zero.
template <bool BF16>
__device__ __forceinline__ void load_vec(const void* row, int col, int cols, float* v) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  const T* p = static_cast<const T*>(row) + col;
  if (col + R::N <= cols) {
    const typename R::Raw w = *reinterpret_cast<const typename R::Raw*>(p);
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::N; ++i) v[i] = col + i < cols ? Elem<BF16>::load(p + i) : 0.f;
  }
}

// The same for `n` = BF16 ? 8 : 4 values starting at any column, of either
// parameter type chosen at run time.
template <int N>
__device__ __forceinline__ void load_params(const void* base, bool bf16, int col, int cols,
                                            float* v) {
  if (bf16) {
    if constexpr (N == 8) {
      load_vec<true>(base, col, cols, v);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = col + i < cols ? bf2f(static_cast<const uint16_t*>(base)[col + i]) : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) load_vec<false>(base, col + i, cols, v + i);
  }
}

template <bool BF16>
__device__ __forceinline__ void store_vec(void* row, int col, int cols, const float* v) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  T* p = static_cast<T*>(row) + col;
  if (col + R::N <= cols) {
    typename R::Raw w;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = f2bf2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    }
    *reinterpret_cast<typename R::Raw*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < R::N; ++i)
      if (col + i < cols) p[i] = Elem<BF16>::cvt(v[i]);
  }
}

// Quantises the N values of this lane at columns [col, col + N) of a row;
// the 32 / N consecutive lanes that hold a block take part together.  The
// lanes past the row's end write the padding (q and scale zero).
template <int N>
__device__ __forceinline__ void ckpt_store(const Ckpt& c, int64_t row, int col, int cols,
                                           const float* v) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    a = a > b ? a : b;
  }
#pragma unroll
  for (int off = 1; off < MUON_CKPT_BLOCK / N; off <<= 1) {
    const uint32_t b = __shfl_xor(a, off, 64);
    a = a > b ? a : b;
  }
  const int byte = ckpt_scale_byte(a, c.fmt);
  const float down = ckpt_down(byte);
  if (col < c.q_pitch) {
    uint32_t* q = reinterpret_cast<uint32_t*>(c.q + row * c.q_pitch + col);
    if constexpr (N == 8) {
      const uint2 w = {ckpt_pack4(v, down, c.fmt), ckpt_pack4(v + 4, down, c.fmt)};
      *reinterpret_cast<uint2*>(q) = w;
    } else {
      *q = ckpt_pack4(v, down, c.fmt);
    }
  }
  if (col % MUON_CKPT_BLOCK == 0 && col / MUON_CKPT_BLOCK < c.s_pitch)
    c.scale[row * c.s_pitch + col / MUON_CKPT_BLOCK] = uint8_t(col < cols ? byte : 0);
}

// N values of a checkpoint's row from column `col` on (a multiple of N; zero
// past the row's pitch).
template <int N>
__device__ __forceinline__ void ckpt_load(const Ckpt& c, int64_t row, int col, float* v) {
  if (col < c.q_pitch) {
    const float up = ckpt_up(c.scale[row * c.s_pitch + col / MUON_CKPT_BLOCK]);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(c.q + row * c.q_pitch + col);
    if constexpr (N == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      ckpt_unpack4(w.x, up, c.fmt, v);
      ckpt_unpack4(w.y, up, c.fmt, v + 4);
    } else {
      ckpt_unpack4(*q, up, c.fmt, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
  }
}

// ------------------------------------------------------------- layer norm
struct LnForward {
  const void* x;
  int64_t ldx;          // elements
  const void* gain;
  const void* bias;     // or null
  void* y;
  float* mean;
  float* rstd;
  int64_t tokens;
  int cols;
  int param_bf16;
  float eps;
  float inv_cols;
  Ckpt xc, yc;          // checkpoints of x and y to write (fmt < 0: none)
};

struct LnBackward {
  const void* dy;
  int64_t lddy;
  const void* x;        // or null: from the checkpoint
  int64_t ldx;
  Ckpt xc;
  const void* gain;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dgain;
  void* dbias;          // or null
  float* partial;       // [blocks][2][cols]
  int64_t tokens;
  int cols;
  int param_bf16;
  int accumulate;
  int blocks;           // of the first launch (0: no tokens)
  float inv_cols;
};

// Blocks of the backward's first launch: each leaves one row of partial sums.
int ln_backward_blocks(int64_t tokens, int64_t cols);

hipError_t launch_ln_forward(const LnForward& p, bool bf16, hipStream_t s);
hipError_t launch_ln_backward(const LnBackward& p, bool bf16, hipStream_t s);
hipError_t launch_ln_params(const LnBackward& p, hipStream_t s);
hipError_t launch_ckpt_save(const void* x, int64_t ldx, bool bf16, const Ckpt& c, int64_t tokens,
                            int cols, hipStream_t s);
hipError_t launch_ckpt_restore(const Ckpt& c, void* x, bool bf16, int64_t tokens, int cols,
                               hipStream_t s);

// ----------------------------------------------------------- weight gradient
struct WeightGrad {
  const void* dy;
  int64_t lddy;
  Ckpt x;
  const int64_t* offsets;  // device, or null
  int64_t tokens;
  int count, rows, cols;
  void* G;
  int g_bf16, accumulate;
  float* partial;          // [slot][rows][cols]
  // A matrix's tokens are cut into pieces of `chunk`; a matrix of more than
  // one piece leaves partial sums in consecutive slots.
  uint32_t chunk;
  int64_t pieces;          // upper bound over all matrices
  void* table;             // with offsets: the pieces and the split matrices
  uint16_t* repack;        // workspace for dy in aligned bf16 rows
  // dy as the 256 x 256 tiles read it
  const uint16_t* y;
  int64_t y_ld;            // elements
  int64_t y_part;          // bytes between the parts of float32 dy
  int y_cols;              // columns that may be read
};
// The cut of the tokens, which also sizes the workspace: partial sums, then
// (ragged) the table, then dy repacked.
constexpr int kWeightGradPieceBytes = 32, kWeightGradSplitBytes = 16;
struct WeightGradPlan {
  uint32_t chunk;
  int64_t pieces, slots;
  bool wide;               // 256 x 256 tiles, where dy's rows allow
  size_t partial_bytes, table_bytes, repack_bytes;
};
WeightGradPlan weight_grad_plan(int64_t count, int64_t tokens, int64_t rows, int64_t cols,
                                bool ragged, bool bf16);
hipError_t launch_weight_grad(const WeightGrad& p, const WeightGradPlan& plan, bool bf16,
                              hipStream_t s);
hipError_t launch_weight_grad_join(const WeightGrad& p, const WeightGradPlan& plan, hipStream_t s);

}  // namespace muon
