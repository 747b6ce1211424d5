// Products of linear layers, forward y = x W^T and input gradient dx = dy W,
// dense or with a matrix per expert over ragged tokens: tiles of outputs from
// LDS on the matrix cores.
//
// Every operand is staged in tiles of rows of 128 bytes of k: 64 bf16, 128 e4m3
// or 32 float32, 8 chunks of 16 bytes.  A lane of a 32 x 32 fragment takes the
// chunks 2 s + lane / 32, s = 0 .. 3, which is the order of k that the
// instructions of all three types want: bf16 multiplies a chunk at a time (k =
// 16), e4m3 two (k = 64, the first 16 bytes of both halves of the lanes being
// one block of 32 with its scale, the second ones the next), float32 four times
// two k, in an order of k that is the same for both operands.  The weight of the
// input gradient runs along n: its tile holds rows of k, which bf16 reads with
// transposing LDS reads and float32 by the element.
#include <algorithm>
#include <type_traits>

#include "lds_tiles.h"
#include "linear_internal.h"

namespace muon {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int ROWB = 128;    // bytes of k per row and step
constexpr int SIDE = MUON_WEIGHT_BLOCK;

int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
__device__ __forceinline__ int cdiv_d(int x, int m) { return (x + m - 1) / m; }

// Chunk c of row r lies at chunk c ^ swz(r): the 16 lanes that a 16-byte read
// serves at once (four quads of every other quad) then use all 64 banks once.
__device__ __forceinline__ int swz(int r) { return (r >> 1 & 1) | (r >> 3 & 3) << 1; }

// ------------------------------------------------------------ tiles and tokens
// The tokens [begin, end) of matrix e (e < 0: of none, whose outputs are zero),
// and this block's tile among theirs.
struct Place {
  int e, begin, end;
  int tm, tn;
};

// Tile number -> tile row and column: groups of 8 tile rows, columns first
// within a group, so that 32 consecutive tiles (an XCD's compute units) share
// their operands.
__device__ __forceinline__ void place_tile(int tile, int tiles_m, int tiles_n, int& ti, int& tj) {
  const int group = tile / (8 * tiles_n), r = tile - group * 8 * tiles_n;
  const int rows = tiles_m - group * 8 < 8 ? tiles_m - group * 8 : 8;
  tj = r / rows;
  ti = group * 8 + r - tj * rows;
}

// Number of block b among `total`: the hardware deals blocks to the 8 XCDs in
// turn; XCD x takes a contiguous eighth.
__device__ __forceinline__ int64_t xcd_order(uint32_t b, uint32_t total) {
  const uint32_t per = (total + 7) / 8, turn = b >> 3, id = (b & 7) * per + turn;
  return turn < per && id < total ? int64_t(id) : -1;
}

// The place of this block.  With offsets, every block finds the bounds itself:
// segment 0 lies before the first offset, segment s holds matrix s - 1, the last
// one the tokens behind the last offset.  Offsets are clamped to [0, tokens] and
// read as the largest so far, so that no place leaves the buffers.  `lds`: 2
// kLinearMaxSegs + 64 words.
template <int THREADS>
__device__ __forceinline__ bool find_place(const Linear& p, int bm, int tiles_n, LDS_AS int* lds,
                                           Place& out) {
  const int t = threadIdx.x, T = int(p.tokens);
  if (!p.offsets) {
    const int tiles_m = cdiv_d(T, bm);
    const int64_t id = xcd_order(blockIdx.x, uint32_t(tiles_m) * tiles_n);
    if (id < 0) return false;
    out.e = out.begin = 0;
    out.end = T;
    place_tile(int(id), tiles_m, tiles_n, out.tm, out.tn);
    return true;
  }
  constexpr int WAVES = THREADS / 64;
  const int lane = t & 63, wave = t >> 6, segs = p.count + 2;
  LDS_AS int *ends = lds, *firsts = lds + kLinearMaxSegs, *wave_top = firsts + kLinearMaxSegs,
             *wave_sum = wave_top + 16, *found = wave_sum + 16;
  int top = 0, tiles = 0;   // of the segments before this group
  for (int base = 0; base < segs; base += THREADS) {
    const int s = base + t;
    int hi = 0;
    if (s <= p.count) {
      const int64_t v = p.offsets[s];
      hi = int(v < 0 ? 0 : v > T ? T : v);
    } else if (s < segs) {
      hi = T;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(hi, off, 64);
      if (lane >= off && o > hi) hi = o;
    }
    if (lane == 63) wave_top[wave] = hi;
    __syncthreads();
    int before = top;
    for (int w = 0; w < wave; ++w) before = before > wave_top[w] ? before : wave_top[w];
    hi = hi > before ? hi : before;
    int lo = __shfl_up(hi, 1, 64);
    if (lane == 0) lo = before;
    const int n = s < segs ? cdiv_d(hi - lo, bm) : 0;
    int sum = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off, 64);
      if (lane >= off) sum += o;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    int first = tiles + sum - n;
    for (int w = 0; w < wave; ++w) first += wave_sum[w];
    if (s < segs) {
      ends[s] = hi;
      firsts[s] = first;
    }
    for (int w = 0; w < WAVES; ++w) {
      top = top > wave_top[w] ? top : wave_top[w];
      tiles += wave_sum[w];
    }
    __syncthreads();
  }
  const int64_t id = xcd_order(blockIdx.x, uint32_t(tiles) * tiles_n);
  if (id < 0) return false;
  for (int s = t; s < segs; s += THREADS) {
    const int64_t a = int64_t(firsts[s]) * tiles_n,
                  b = int64_t(s + 1 < segs ? firsts[s + 1] : tiles) * tiles_n;
    if (id >= a && id < b) *found = s;
  }
  __syncthreads();
  const int s = __builtin_amdgcn_readfirstlane(*found);
  const int first = __builtin_amdgcn_readfirstlane(firsts[s]);
  const int next = __builtin_amdgcn_readfirstlane(s + 1 < segs ? firsts[s + 1] : tiles);
  out.e = s > p.count ? -1 : s - 1;
  out.begin = __builtin_amdgcn_readfirstlane(s > 0 ? ends[s - 1] : 0);
  out.end = __builtin_amdgcn_readfirstlane(ends[s]);
  place_tile(int(id - int64_t(first) * tiles_n), next - first, tiles_n, out.tm, out.tn);
  __syncthreads();      // the tiles overwrite what was read here
  return true;
}

// ---------------------------------------------------------------- the epilogue
// Writes a wave's 32 MT tokens (from t0) x 32 NT outputs (from n0) through a
// window of LDS of its own, 32 tokens at a time, so that lanes store whole runs
// of a row.  Lane l, register 4 g + i of a 32 x 32 block holds token l % 32,
// output 8 g + 4 (l / 32) + i.
template <int NT>
constexpr int window_bytes() { return 32 * (32 * NT + 4) * 4; }
template <int MT, int NT>
__device__ __forceinline__ void store_tile(const Linear& p, int t0, int end, int n0,
                                           const f32x16_t (&acc)[MT][NT], LDS_AS char* window,
                                           int lane) {
  constexpr int PITCH = 32 * NT + 4;
  LDS_AS float* w = (LDS_AS float*)window;
#pragma unroll
  for (int a = 0; a < MT; ++a) {
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(LDS_AS f32x4_t*)(w + (lane & 31) * PITCH + b * 32 + 8 * g + 4 * (lane >> 5)) =
            f32x4_t{acc[a][b][4 * g], acc[a][b][4 * g + 1], acc[a][b][4 * g + 2],
                    acc[a][b][4 * g + 3]};
    wave_lds_sync();
    auto rows = [&](auto bf16) {
      constexpr int N = RowVec<decltype(bf16)::value>::N;
      constexpr int LANES = 32 * NT / N;   // per row
#pragma unroll
      for (int r = 0; r < 32 * LANES / 64; ++r) {
        const int row = r * (64 / LANES) + lane / LANES, col = lane % LANES * N;
        const int t = t0 + a * 32 + row, n = n0 + col;
        if (t < end && n < p.n) {
          float v[N];
#pragma unroll
          for (int i = 0; i < N; i += 4) {
            const f32x4_t x = *(const LDS_AS f32x4_t*)(w + row * PITCH + col + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = x[j];
          }
          using T = typename RowVec<decltype(bf16)::value>::T;
          store_vec<decltype(bf16)::value>(static_cast<T*>(p.y) + int64_t(t) * p.n + n, 0, p.n - n, v);
        }
      }
    };
    if (p.y_bf16)
      rows(std::true_type{});
    else
      rows(std::false_type{});
    wave_lds_sync();
  }
}

// ------------------------------------------------------------------- the tiles
template <int BM_, int BN_, int WM_, int WN_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;   // tokens, outputs, waves
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MT = BM / WM / 32, NT = BN / WN / 32;     // 32 x 32 blocks per wave
};
using Tile128 = Shape<128, 128, 2, 2>;
using Tile256 = Shape<256, 256, 2, 4>;

template <LinearType TYPE>
constexpr int elem_bytes() { return TYPE == LIN_BF16 ? 2 : TYPE == LIN_F32 ? 4 : 1; }

// ACROSS: the weight's rows are k (dx = dy W).  DIRECT: both operands' rows
// start on 16 bytes and hold whole chunks, so that they go straight to LDS;
// otherwise they pass through registers, where what follows a row's end becomes
// zero.
template <LinearType TYPE, bool ACROSS, bool DIRECT, class S>
__global__ __launch_bounds__(S::THREADS, S::NW == 8 ? 1 : 2) void linear_kernel(const Linear p, int tiles_n) {
  constexpr int ES = elem_bytes<TYPE>(), BK = ROWB / ES;
  constexpr int BM = S::BM, BN = S::BN, MT = S::MT, NT = S::NT, THREADS = S::THREADS;
  constexpr bool E4M3 = TYPE >= LIN_E4M3;
  static_assert(!(E4M3 && ACROSS), "8-bit weights are kept both ways");
  constexpr int X_BYTES = BM * ROWB, W_BYTES = BN * ROWB;
  constexpr int XS_BYTES = E4M3 ? S::NW * 256 : 0;        // x scales of a step
  constexpr int STAGE = X_BYTES + W_BYTES + XS_BYTES;
  constexpr int WS_AT = 2 * STAGE, WS_BYTES = E4M3 ? BN / SIDE * (MUON_MAX_DIM / SIDE) : 0;
  constexpr int LDS_BYTES = WS_AT + WS_BYTES;
  static_assert(LDS_BYTES <= (S::NW == 8 ? 160 : 80) * 1024, "LDS");
  static_assert(S::NW * window_bytes<NT>() <= LDS_BYTES, "the epilogue's windows");
  __shared__ __attribute__((aligned(1024))) char smem_raw[LDS_BYTES];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;
  const uint32_t smem_base = uint32_t(reinterpret_cast<uintptr_t>(smem));

  Place at;
  if (!find_place<THREADS>(p, BM, tiles_n, (LDS_AS int*)smem, at)) return;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int t0 = at.begin + at.tm * BM, n0 = at.tn * BN;

  f32x16_t acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  const int steps = at.e < 0 ? 0 : cdiv_d(p.k, BK);
  const int last_k = p.k - (steps - 1) * BK;     // of the last step
  const int last_chunks = cdiv_d(last_k * ES, 16);
  const char* x = static_cast<const char*>(p.x) + int64_t(t0) * p.ldx;
  const char* w = static_cast<const char*>(p.W) + (at.e < 0 ? 0 : at.e) * p.w_stride +
                  (ACROSS ? int64_t(n0) * ES : int64_t(n0) * p.ldw);
  const int rows_x = at.end - t0 < BM ? at.end - t0 : BM, rows_w = p.n - n0 < BN ? p.n - n0 : BN;

  // This thread's chunks of a step.  x, and w along k: chunk `at` is row at / 8,
  // place at % 8.  w across: rows of k of BN outputs.
  constexpr int XI = X_BYTES / 16 / THREADS, WI = W_BYTES / 16 / THREADS;
  constexpr int WPR = BN * ES / 16;              // chunks per k row of a w across
  auto x_at = [&](int i) { return DIRECT ? (wave * XI + i) * 64 + lane : i * THREADS + t; };
  auto w_at = [&](int i) { return DIRECT ? (wave * WI + i) * 64 + lane : i * THREADS + t; };
  // where chunk c of row k of a w across lies
  auto w_swz = [](int k) { return TYPE == LIN_BF16 ? gswz(k) : (k >> 2 & 1) << 3; };

  // ---- loads straight to LDS
  uint32_t x_off[XI], w_off[WI];
  if constexpr (DIRECT) {
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int r = x_at(i) / 8;
      x_off[i] = uint32_t(r < rows_x ? r : rows_x - 1) * uint32_t(p.ldx) + ((x_at(i) % 8) ^ swz(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      if constexpr (ACROSS) {
        const int k = w_at(i) / WPR, c = (w_at(i) % WPR) ^ w_swz(k);
        w_off[i] = uint32_t(k) * uint32_t(p.ldw) + (c * 16 < rows_w * ES ? c * 16 : rows_w * ES - 16);
      } else {
        const int r = w_at(i) / 8;
        w_off[i] = uint32_t(r < rows_w ? r : rows_w - 1) * uint32_t(p.ldw) + ((w_at(i) % 8) ^ swz(r)) * 16;
      }
    }
  }
  // x scales: a word per row and step.
  const uint32_t xs_row = (wave * 64 + lane) % BM;
  const uint32_t xs_off = E4M3 ? uint32_t(int(xs_row) < rows_x ? int(xs_row) : rows_x - 1) * uint32_t(p.xs_pitch) : 0;
  const char* xs = E4M3 ? reinterpret_cast<const char*>(p.x_scale) + int64_t(t0) * p.xs_pitch : nullptr;

  // END: the step may be the last one, whose chunks past the row's end read its
  // last chunk instead (and are cleared when they have come; e4m3's weight has
  // zeros there, and x the scale of a padding).
  auto issue = [&](auto end, int buf, int k) __attribute__((always_inline)) {
    const bool tail = decltype(end)::value && k == steps - 1;
    const uint32_t base = smem_base + buf * STAGE;
    const char* xk = x + int64_t(k) * ROWB;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      uint32_t off = x_off[i];
      if (tail) {
        const int c = (x_at(i) % 8) ^ swz(x_at(i) / 8);
        if (c >= last_chunks) off -= (c - last_chunks + 1) * 16;
      }
      dma16(off, xk, base + (wave * XI + i) * WAVE_BYTES);
    }
    const char* wk = w + (ACROSS ? int64_t(k) * BK * p.ldw : int64_t(k) * ROWB);
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      uint32_t off = w_off[i];
      if constexpr (ACROSS) {
        const int kr = w_at(i) / WPR;
        if (tail && kr >= last_k) off -= uint32_t(kr - last_k + 1) * uint32_t(p.ldw);
      } else if constexpr (!E4M3) {
        const int c = (w_at(i) % 8) ^ swz(w_at(i) / 8);
        if (tail && c >= last_chunks) off -= (c - last_chunks + 1) * 16;
      }
      dma16(off, wk, base + X_BYTES + (wave * WI + i) * WAVE_BYTES);
    }
    if constexpr (E4M3) dma4(xs_off, xs + int64_t(k) * 4, base + X_BYTES + W_BYTES + wave * 256);
  };
  // This thread's chunks of the last step that lie past the end.
  auto clear_tail = [&](int buf) {
    LDS_AS char* s = smem + buf * STAGE;
#pragma unroll
    for (int i = 0; i < XI; ++i)
      if (((x_at(i) % 8) ^ swz(x_at(i) / 8)) >= last_chunks)
        *reinterpret_cast<LDS_AS u32x4_t*>(s + x_at(i) * 16) = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const bool past = ACROSS ? w_at(i) / WPR >= last_k
                               : ((w_at(i) % 8) ^ swz(w_at(i) / 8)) >= last_chunks;
      if (past) *reinterpret_cast<LDS_AS u32x4_t*>(s + X_BYTES + w_at(i) * 16) = u32x4_t{0, 0, 0, 0};
    }
  };

  // ---- loads through registers (float32 and bf16)
  using R = RowVec<TYPE == LIN_BF16>;
  u32x4_t xr[DIRECT ? 1 : XI], wr[DIRECT ? 1 : WI];
  auto load = [&](int k) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
      const bool whole = k < steps - 1 || last_k == BK;
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int r = x_at(i) / 8, c = x_at(i) % 8;
        const char* row = x + int64_t(r < rows_x ? r : rows_x - 1) * p.ldx + int64_t(k) * ROWB;
        if (whole)
          xr[i] = load_raw<TYPE == LIN_BF16, true>(row, c * R::N, BK);
        else
          xr[i] = load_raw<TYPE == LIN_BF16>(row, c * R::N, last_k);
      }
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        if constexpr (ACROSS) {
          const int kr = w_at(i) / WPR, c = w_at(i) % WPR;
          const char* row = w + (int64_t(k) * BK + kr) * p.ldw;
          if (!whole && kr >= last_k)
            wr[i] = u32x4_t{0, 0, 0, 0};
          else if (rows_w == BN)
            wr[i] = load_raw<TYPE == LIN_BF16, true>(row, c * R::N, BN);
          else
            wr[i] = load_raw<TYPE == LIN_BF16>(row, c * R::N, rows_w);
        } else {
          const int r = w_at(i) / 8, c = w_at(i) % 8;
          const char* row = w + int64_t(r < rows_w ? r : rows_w - 1) * p.ldw + int64_t(k) * ROWB;
          if (whole)
            wr[i] = load_raw<TYPE == LIN_BF16, true>(row, c * R::N, BK);
          else
            wr[i] = load_raw<TYPE == LIN_BF16>(row, c * R::N, last_k);
        }
      }
    }
  };
  auto write = [&](int buf) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
      LDS_AS char* s = smem + buf * STAGE;
#pragma unroll
      for (int i = 0; i < XI; ++i) {
        const int r = x_at(i) / 8, c = x_at(i) % 8;
        *reinterpret_cast<LDS_AS u32x4_t*>(s + r * ROWB + (c ^ swz(r)) * 16) = xr[i];
      }
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        const int per = ACROSS ? WPR : 8, r = w_at(i) / per, c = w_at(i) % per;
        *reinterpret_cast<LDS_AS u32x4_t*>(s + X_BYTES + r * per * 16 +
                                           (c ^ (ACROSS ? w_swz(r) : swz(r))) * 16) = wr[i];
      }
    }
  };

  // ---- fragments and products of a step
  auto frag = [&](const LDS_AS char* tile, int row0, int s) {
    const int r = row0 + (lane & 31), c = 2 * s + (lane >> 5);
    return *reinterpret_cast<const LDS_AS u32x4_t*>(tile + r * ROWB + (c ^ swz(r)) * 16);
  };
  auto frag_w = [&](const LDS_AS char* tile, int row0, int s) -> u32x4_t {
    if constexpr (!ACROSS) {
      return frag(tile, row0, s);
    } else if constexpr (TYPE == LIN_BF16) {
      return __builtin_bit_cast(u32x4_t, lds_frag_xT<BN>(tile, 16 * s, row0, lane));
    } else {
      const int n = row0 + (lane & 31), k = 4 * (2 * s + (lane >> 5));
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const LDS_AS uint32_t*>(tile + (k + i) * (BN * 4) +
                                                         (((n >> 2) ^ w_swz(k + i)) << 4) + (n & 3) * 4);
      return v;
    }
  };
  auto multiply = [&](int buf, int k) __attribute__((always_inline)) {
    const LDS_AS char* s = smem + buf * STAGE;
    const LDS_AS char* sw = s + X_BYTES;
    const int xr0 = wm * MT * 32, wr0 = wn * NT * 32;
    if constexpr (E4M3) {
      uint32_t sx[MT];
#pragma unroll
      for (int a = 0; a < MT; ++a)
        sx[a] = *reinterpret_cast<const LDS_AS uint32_t*>(s + X_BYTES + W_BYTES + (xr0 + a * 32 + (lane & 31)) * 4);
      const uint32_t wsc = *reinterpret_cast<const LDS_AS uint8_t*>(smem + WS_AT + wr0 / SIDE * (MUON_MAX_DIM / SIDE) + k);
      static_assert(SIDE % (NT * 32) == 0, "a wave's outputs share a scale");
      if constexpr (TYPE == LIN_E4M3_EXACT) {
        // a chunk of 16 as two of bf16, exact: the conversion multiplies by 2^e
        // (255, a marked block, by NaN)
        auto wide = [&](u32x4_t q, uint32_t byte, bf16x8_t (&o)[2]) {
          const float up = __uint_as_float(byte << 23);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t v = {
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h], up, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h], up, true)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h + 1], up, false)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * h + 1], up, true))};
            o[h] = __builtin_bit_cast(bf16x8_t, v);
          }
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          bf16x8_t xf[MT][2], wf[NT][2];
          // both chunks of a fragment (one per half of the lanes) are of block c
#pragma unroll
          for (int a = 0; a < MT; ++a) wide(frag(s, xr0 + a * 32, c), sx[a] >> (8 * c) & 0xff, xf[a]);
#pragma unroll
          for (int b = 0; b < NT; ++b) wide(frag(sw, wr0 + b * 32, c), wsc, wf[b]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
              for (int b = 0; b < NT; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wf[b][h], xf[a][h], acc[a][b], 0, 0, 0);
        }
        return;
      }
#pragma unroll
      for (int a = 0; a < MT; ++a) sx[a] >>= 8 * (lane >> 5);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x8_t xf[MT], wf[NT];
        auto two = [&](const LDS_AS char* tile, int row0) {
          const u32x4_t lo = frag(tile, row0, 2 * h), hi = frag(tile, row0, 2 * h + 1);
          return i32x8_t{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                         int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
        };
#pragma unroll
        for (int a = 0; a < MT; ++a) xf[a] = two(s, xr0 + a * 32);
#pragma unroll
        for (int b = 0; b < NT; ++b) wf[b] = two(sw, wr0 + b * 32);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < NT; ++b) {
            if (h == 0)
              acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[b], xf[a], acc[a][b], 0, 0, 0, int(wsc),
                                                                          0, int(sx[a]));
            else
              acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[b], xf[a], acc[a][b], 0, 0, 0, int(wsc),
                                                                          2, int(sx[a]));
          }
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        u32x4_t xf[MT], wf[NT];
#pragma unroll
        for (int a = 0; a < MT; ++a) xf[a] = frag(s, xr0 + a * 32, c);
#pragma unroll
        for (int b = 0; b < NT; ++b) wf[b] = frag_w(sw, wr0 + b * 32, c);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < NT; ++b) {
            if constexpr (TYPE == LIN_BF16) {
              acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, wf[b]),
                                                                  __builtin_bit_cast(bf16x8_t, xf[a]),
                                                                  acc[a][b], 0, 0, 0);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wf[b][i]),
                                                                 __uint_as_float(xf[a][i]), acc[a][b], 0, 0, 0);
            }
          }
      }
    }
  };

  if (steps > 0) {
    if constexpr (E4M3) {      // the weight's scales, all of k
      const uint8_t* ws = p.w_scale + at.e * p.ws_stride + int64_t(n0 / SIDE) * p.ws_row;
#pragma unroll
      for (int b = 0; b < BN / SIDE; ++b)
        if (n0 + b * SIDE < p.n)
          for (int k = t; k < steps; k += THREADS)
            *reinterpret_cast<LDS_AS uint8_t*>(smem + WS_AT + b * (MUON_MAX_DIM / SIDE) + k) =
                ws[b * p.ws_row + k * p.ws_col];
    }
    if constexpr (DIRECT) {
      issue(std::true_type{}, 0, 0);
      for (int k = 0; k < steps; ++k) {
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        if (!E4M3 && k == steps - 1 && last_chunks < 8) clear_tail(k & 1);
        block_barrier();
        if (k + 1 < steps) issue(std::true_type{}, (k + 1) & 1, k + 1);
        multiply(k & 1, k);
      }
    } else {
      load(0);
      write(0);
      for (int k = 0; k < steps; ++k) {
        block_barrier();
        if (k + 1 < steps) load(k + 1);
        multiply(k & 1, k);
        if (k + 1 < steps) write((k + 1) & 1);
      }
    }
    block_barrier();
  }
  store_tile<MT, NT>(p, t0 + wm * MT * 32, at.end, n0 + wn * NT * 32, acc,
                     smem + wave * window_bytes<NT>(), lane);
}

template <LinearType TYPE, bool ACROSS, bool DIRECT, class S>
hipError_t launch_tiles(const Linear& p, hipStream_t s) {
  const int64_t tiles_n = cdiv(p.n, S::BN);
  const int64_t tiles_m = p.offsets ? p.tokens / S::BM + p.count + 2 : cdiv(p.tokens, S::BM);
  hipLaunchKernelGGL((linear_kernel<TYPE, ACROSS, DIRECT, S>), dim3(unsigned(cdiv(tiles_m * tiles_n, 8) * 8)),
                     dim3(S::THREADS), 0, s, p, int(tiles_n));
  return hipGetLastError();
}

}  // namespace

LinearPlan linear_plan(LinearType type, bool across, int64_t count, int64_t tokens, int64_t k, int64_t n) {
  if ((tokens / 128 + count + 10) * cdiv(n, 128) >= (int64_t(1) << 24) - 8) return LIN_NONE;
  if (type == LIN_F32) return LIN_128;
  return cdiv(tokens, count) >= 512 ? LIN_256 : LIN_128;
}

hipError_t launch_linear(const Linear& p, LinearType type, bool across, LinearPlan plan, hipStream_t s) {
  const int es = type == LIN_BF16 ? 2 : 4;
  // whole chunks in both operands' rows, and offsets within a tile in 32 bits
  const bool direct = type >= LIN_E4M3 ||
                      (reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.W) % 16 == 0 &&
                       p.ldx % 16 == 0 && p.ldw % 16 == 0 && p.k * es % 16 == 0 && (!across || p.n * es % 16 == 0) &&
                       p.ldx <= (1 << 23));
  if (type == LIN_E4M3_EXACT) return launch_tiles<LIN_E4M3_EXACT, false, true, Tile128>(p, s);
  if (type == LIN_E4M3)
    return plan == LIN_256 ? launch_tiles<LIN_E4M3, false, true, Tile256>(p, s)
                           : launch_tiles<LIN_E4M3, false, true, Tile128>(p, s);
  if (type == LIN_BF16) {
    if (plan == LIN_256 && direct)
      return across ? launch_tiles<LIN_BF16, true, true, Tile256>(p, s)
                    : launch_tiles<LIN_BF16, false, true, Tile256>(p, s);
    if (direct)
      return across ? launch_tiles<LIN_BF16, true, true, Tile128>(p, s)
                    : launch_tiles<LIN_BF16, false, true, Tile128>(p, s);
    return across ? launch_tiles<LIN_BF16, true, false, Tile128>(p, s)
                  : launch_tiles<LIN_BF16, false, false, Tile128>(p, s);
  }
  if (direct)
    return across ? launch_tiles<LIN_F32, true, true, Tile128>(p, s)
                  : launch_tiles<LIN_F32, false, true, Tile128>(p, s);
  return across ? launch_tiles<LIN_F32, true, false, Tile128>(p, s)
                : launch_tiles<LIN_F32, false, false, Tile128>(p, s);
}

}  // namespace muon
