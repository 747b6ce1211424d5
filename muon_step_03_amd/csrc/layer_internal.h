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

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// The 16 bytes of elements [col, col + N) of a row of `cols`, those past its
// end as zero.  EVEN: cols is a multiple of N, so no vector crosses the end.
template <bool BF16, bool EVEN = false>
__device__ __forceinline__ u32x4_t load_raw(const void* row, int col, int cols) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  const T* p = static_cast<const T*>(row) + col;
  u32x4_t w = {0, 0, 0, 0};
  if (col + R::N <= cols) {
    const typename R::Raw r = *reinterpret_cast<const typename R::Raw*>(p);
    w = u32x4_t{r[0], r[1], r[2], r[3]};
  } else if constexpr (!EVEN) {
#pragma unroll
    for (int i = 0; i < R::N; ++i)
      if (col + i < cols) {
        if constexpr (BF16)
          w[i / 2] |= uint32_t(p[i]) << (16 * (i & 1));
        else
          w[i] = __float_as_uint(p[i]);
      }
  }
  return w;
}

// How rows end: with a whole vector; inside a vector of a row that holds one
// at least; before the first vector's end.
enum RowEnd { END_WHOLE, END_INSIDE, END_SHORT };
inline RowEnd row_end(int64_t cols, int n) {
  return cols % n == 0 ? END_WHOLE : cols >= n ? END_INSIDE : END_SHORT;
}
// load_raw in two halves, for loads in flight: what is loaded, and, once it is
// used, the elements that were asked for.  A vector that crosses the row's end
// (or lies past it) is loaded from the row's last N elements and shifted down:
// a load that no lane's branch guards, which nothing has to wait for before its
// use (16384 rows of 1411 float32, forward: 44 us with guarded elements, 35 so).
template <bool BF16, RowEnd END>
__device__ __forceinline__ u32x4_t load_ahead(const void* row, int col, int cols) {
  if constexpr (END != END_INSIDE) return load_raw<BF16, END == END_WHOLE>(row, col, cols);
  using R = RowVec<BF16>;
  const int at = col < cols - R::N ? col : cols - R::N;
  const typename R::Raw r =
      *reinterpret_cast<const typename R::Raw*>(static_cast<const typename R::T*>(row) + at);
  return u32x4_t{r[0], r[1], r[2], r[3]};
}
// A vector without its first `by` elements, zeros behind the last.
template <bool BF16>
__device__ __forceinline__ void shift_down(u32x4_t& w, int by) {
  if constexpr (BF16) {
    if (by & 1)
      w = u32x4_t{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
    by >>= 1;
  }
  if (by & 1) w = u32x4_t{w[1], w[2], w[3], 0};
  if (by & 2) w = u32x4_t{w[2], w[3], 0, 0};
  if (by >= 4) w = u32x4_t{0, 0, 0, 0};
}
template <bool BF16, RowEnd END>
__device__ __forceinline__ void settle(u32x4_t& w, int col, int cols) {
  if constexpr (END != END_INSIDE) return;
  const int by = col - (cols - RowVec<BF16>::N);
  if (by > 0) shift_down<BF16>(w, by);
}
template <bool BF16>
__device__ __forceinline__ void unpack_raw(u32x4_t w, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}
template <bool BF16>
__device__ __forceinline__ u32x4_t pack_raw(const float* v) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = BF16 ? f2bf2(v[2 * i], v[2 * i + 1]) : __float_as_uint(v[i]);
  return w;
}
// STREAM: the caches need not keep it.
template <bool BF16, bool EVEN = false, bool STREAM = false>
__device__ __forceinline__ void store_raw(void* row, int col, int cols, u32x4_t w) {
  using R = RowVec<BF16>;
  using T = typename R::T;
  T* p = static_cast<T*>(row) + col;
  if (col + R::N <= cols) {
    const typename R::Raw r = {w[0], w[1], w[2], w[3]};
    if constexpr (STREAM)
      __builtin_nontemporal_store(r, reinterpret_cast<typename R::Raw*>(p));
    else
      *reinterpret_cast<typename R::Raw*>(p) = r;
  } else if constexpr (!EVEN) {
#pragma unroll
    for (int i = 0; i < R::N; ++i)
      if (col + i < cols) {
        if constexpr (BF16)
          p[i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
        else
          p[i] = __uint_as_float(w[i]);
      }
  }
}

// Elements [col, col + N) of a row of `cols`, those past its end as zero.
template <bool BF16>
__device__ __forceinline__ void load_vec(const void* row, int col, int cols, float* v) {
  unpack_raw<BF16>(load_raw<BF16>(row, col, cols), v);
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

template <bool BF16, bool STREAM = false>
__device__ __forceinline__ void store_vec(void* row, int col, int cols, const float* v) {
  store_raw<BF16, false, STREAM>(row, col, cols, pack_raw<BF16>(v));
}

// Lane exchanges within a row of 16 lanes (data-parallel-primitive moves).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, false));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;             // quad_perm
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;    // row_half_mirror, row_mirror

// Quantises a vector of 16 bytes at columns [col, col + N) of a row; the 32 / N
// consecutive lanes that hold a block take part together.  The lanes past
// the row's end (their elements zero) write the padding.
template <bool BF16>
__device__ __forceinline__ void ckpt_store(const Ckpt& c, int64_t row, int col, int cols,
                                           u32x4_t w) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  constexpr int N = RowVec<BF16>::N;
  // the block's largest magnitude as a bit pattern (the order of floats is
  // that of their patterns)
  uint32_t a;
  if constexpr (BF16) {
    u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7fff7fffu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    a = uint32_t(m[0] > m[1] ? m[0] : m[1]) << 16;
  } else {
    a = w[0] & 0x7fffffffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) a = max(a, w[i] & 0x7fffffffu);
  }
  a = max(a, dpp<kXor1>(a));
  a = max(a, dpp<kXor2>(a));
  if constexpr (N == 4) a = max(a, dpp<kMirror8>(a));
  const int byte = ckpt_scale_byte(a, c.fmt);
  const int top = 127 + (c.fmt == MUON_CKPT_E4M3 ? kCkptEMaxE4m3 : kCkptEMaxInt8);
  uint32_t q[N / 4];
  if (c.fmt == MUON_CKPT_E4M3 && byte != top) {
    // the conversion divides by 2^e and rounds to nearest even: in range here
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float up = __uint_as_float(uint32_t(byte) << 23);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      s16x2 r = {0, 0};
      if constexpr (BF16) {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, uint32_t(w[2 * i])), up, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2_t, uint32_t(w[2 * i + 1])), up, true);
      } else {
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[0]), __uint_as_float(w[1]), up, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, __uint_as_float(w[2]), __uint_as_float(w[3]), up, true);
      }
      q[i] = __builtin_bit_cast(uint32_t, r);
    }
  } else {
    // at the largest exponent a value may still be out of range: it saturates
    const float down = ckpt_down(byte);
    float v[N];
    unpack_raw<BF16>(w, v);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float* x = v + 4 * i;
      if (c.fmt == MUON_CKPT_E4M3) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(x[0] * down, -448.f, 448.f),
                                                __builtin_amdgcn_fmed3f(x[1] * down, -448.f, 448.f), 0, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(x[2] * down, -448.f, 448.f),
                                            __builtin_amdgcn_fmed3f(x[3] * down, -448.f, 448.f), r, true);
        q[i] = uint32_t(r);
      } else {
        // adding 1.5 * 2^23 leaves the integer, rounded half to even, in the
        // low byte; the clamp only acts at the largest exponent
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = __float_as_uint(__builtin_amdgcn_fmed3f(x[j] * down, -127.f, 127.f) + 12582912.f);
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
        q[i] = lo | hi;
      }
    }
  }
  if (byte == 255) {   // a marked block
#pragma unroll
    for (int i = 0; i < N / 4; ++i) q[i] = 0;
  }
  if (col < c.q_pitch) {
    uint32_t* to = reinterpret_cast<uint32_t*>(c.q + row * c.q_pitch + col);
    if constexpr (N == 8)
      *reinterpret_cast<uint2*>(to) = uint2{q[0], q[1]};
    else
      *to = q[0];
  }
  if (col % MUON_CKPT_BLOCK == 0 && col / MUON_CKPT_BLOCK < c.s_pitch)
    c.scale[row * c.s_pitch + col / MUON_CKPT_BLOCK] = uint8_t(col < cols ? byte : 0);
}

// N = 8 or 4 values of a checkpoint's row from column `col` on (a multiple of
// N; zero past the row's pitch): loaded, then brought back.
template <int N>
struct CkptVec {
  uint32_t w[N / 4];
  int byte;
};
template <int N>
__device__ __forceinline__ CkptVec<N> ckpt_load(const Ckpt& c, int64_t row, int col) {
  CkptVec<N> r;
  r.byte = 0;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) r.w[i] = 0;
  if (col < c.q_pitch) {
    r.byte = c.scale[row * c.s_pitch + col / MUON_CKPT_BLOCK];
    const uint32_t* q = reinterpret_cast<const uint32_t*>(c.q + row * c.q_pitch + col);
    if constexpr (N == 8) {
      const uint2 w = *reinterpret_cast<const uint2*>(q);
      r.w[0] = w.x;
      r.w[1] = w.y;
    } else {
      r.w[0] = *q;
    }
  }
  return r;
}
template <int N>
__device__ __forceinline__ void ckpt_values(const CkptVec<N>& r, int fmt, float* v) {
  const float up = ckpt_up(r.byte);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) ckpt_unpack4(r.w[i], up, fmt, v + 4 * i);
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
};

// Blocks of the backward's first launch: each leaves one row of partial sums.
int ln_backward_blocks(int64_t tokens, int64_t cols, bool bf16);   // bf16: at least float32's

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
  uint16_t* repack;        // workspace for dy in aligned rows
  // dy as the 256 x 256 tiles read it
  const uint16_t* y;
  int64_t y_ld;            // elements
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
