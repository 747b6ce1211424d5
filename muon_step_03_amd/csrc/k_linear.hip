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
//
// Tiles of 64 x 64 (four steps on their way to LDS) while those of 128 x 128 (two
// blocks per CU, a step ahead) would not fill the chip: bound by latency there,
// then by the loads from the L2.  Measured on one MI355X, calls between others: bf16
// input gradient of 49152 tokens, 64 x 1408 x 512, uneven, 128 x 128: 110 us (650
// TFLOP/s), over the same operands again and again, which the caches hold then, 83 to
// 92; 1023 tokens of 7 x 777 x 1001, no row on 16 bytes, 64 x 64: 15.9 us; 1024 tokens
// of 1024 x 1024 10.3 us.  float32: 16384 tokens of 1024 x 1024 248 us forward, 245
// back, 140 TFLOP/s as the library's product; 2049 tokens of 7 x 1001 x 777 46 us
// forward, 47 back; 16384 of 64 x 1408 x 512 233 and 257 (102 and 92 TFLOP/s).  8 bits
// to float32, 16384 tokens of 4096 x 1024: 142 us forward, 119 back (970 and 1155).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "lds_tiles.h"
#include "linear_device.h"

namespace muon {
namespace {

// ---------------------------------------------------------------- the epilogue
// Writes a wave's 32 MT tokens (from t0) x 32 NT outputs (from n0) through a
// window of LDS of its own, 32 tokens at a time, so that lanes store whole runs
// of a row.  Lane l, register 4 g + i of a 32 x 32 block holds token l % 32,
// output 8 g + 4 (l / 32) + i.  STREAM: the L2 need not keep them, as for calls that
// fill the chip with the larger tiles (49152 tokens of 64 x 1408 x 512, input
// gradient, over the same operands again: 110 -> 94 us).
template <int NT>
constexpr int window_bytes() { return 32 * (32 * NT + 4) * 4; }
template <int MT, int NT, bool STREAM>
__device__ __forceinline__ void store_tile(const Linear& p, int t0, int end, int n0,
                                           const f32x16_t (&acc)[MT][NT], LDS_AS char* window,
                                           int lane) {
  constexpr int PITCH = 32 * NT + 4;
  LDS_AS float* w = (LDS_AS float*)window;
  const bool lines = whole_lines(p);
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
          T* y = static_cast<T*>(p.y) + int64_t(t) * p.n + n;
          if (STREAM && lines)
            store_vec<decltype(bf16)::value, true>(y, 0, p.n - n, v);
          else
            store_vec<decltype(bf16)::value, false>(y, 0, p.n - n, v);
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
template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;   // tokens, outputs, waves
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int MT = BM / WM / 32, NT = BN / WN / 32;     // 32 x 32 blocks per wave
  static constexpr int STAGES = STAGES_;   // steps in LDS, loaded straight there
  static constexpr int AHEAD = BM == 64 ? 4 : 2;                 // steps in registers otherwise
};
using Tile64 = Shape<64, 64, 2, 2, 4>;
using Tile128 = Shape<128, 128, 2, 2, 2>;

template <LinearType TYPE>
constexpr int elem_bytes() { return TYPE == LIN_BF16 ? 2 : TYPE == LIN_F32 ? 4 : 1; }

// ACROSS: the weight's rows are k (dx = dy W).  How operands reach LDS: straight,
// where the rows of both start on 16 bytes and hold whole chunks; otherwise
// through registers, where what follows a row's end becomes zero; rows shorter
// than a chunk by elements.
enum LinearPath { DIRECTLY, BY_VECTORS, BY_ELEMENTS };
template <LinearType TYPE, bool ACROSS, LinearPath PATH, class S>
__global__ __launch_bounds__(S::THREADS, 2) void linear_kernel(const Linear p, int tiles_n) {
  constexpr int ES = elem_bytes<TYPE>(), BK = ROWB / ES;
  constexpr int BM = S::BM, BN = S::BN, MT = S::MT, NT = S::NT, THREADS = S::THREADS;
  constexpr bool E4M3 = TYPE >= LIN_E4M3, DIRECT = PATH == DIRECTLY, TINY = PATH == BY_ELEMENTS;
  static_assert(!(E4M3 && ACROSS), "8-bit weights are kept both ways");
  constexpr int X_BYTES = BM * ROWB, W_BYTES = BN * ROWB;
  constexpr int XS_BYTES = E4M3 ? S::NW * 256 : 0;        // x scales of a step
  constexpr int STAGE = X_BYTES + W_BYTES + XS_BYTES;
  constexpr int STAGES = DIRECT ? S::STAGES : 2;
  static_assert(SIDE % BN == 0, "a tile's outputs share the scales of a weight");
  constexpr int WS_AT = STAGES * STAGE, WS_BYTES = E4M3 ? MUON_MAX_DIM / SIDE : 0;
  constexpr int LDS_BYTES = WS_AT + WS_BYTES;
  static_assert(LDS_BYTES <= 80 * 1024, "LDS");
  static_assert(S::NW * window_bytes<NT>() <= LDS_BYTES, "the epilogue's windows");
  __shared__ __attribute__((aligned(1024))) char smem_raw[LDS_BYTES];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;
  const uint32_t smem_base = uint32_t(reinterpret_cast<uintptr_t>(smem));

  Bounds bounds{};
  bounds.tiles = cdiv_d(int(p.tokens), BM);
  if (p.offsets) bounds = find_bounds<THREADS, true>(p, BM, (LDS_AS int*)smem);
  const int64_t id = xcd_order(blockIdx.x, uint32_t(bounds.tiles) * tiles_n);
  if (id < 0) return;
  const Place at = place_of(p, bounds, BM, tiles_n, int(id));
  __syncthreads();      // the tiles overwrite what was read here
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
  auto w_swz = [](int k) { return TYPE == LIN_BF16 ? swz_across<BN>(k) : (k >> 2 & 1) << 3; };

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
  constexpr int LOADS = XI + WI + (E4M3 ? 1 : 0);   // per wave and step
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

  // ---- loads through registers (float32 and bf16).  A vector that crosses a row's
  // end, or lies behind it, is loaded from the row's last elements and shifted down
  // when it is written, with zeros behind them: a load that no branch guards, which
  // nothing has to wait for before (elements loaded one by one in the last step
  // took half of the time of 1000 tokens).
  constexpr int AHEAD = DIRECT ? 1 : S::AHEAD;
  using R = RowVec<TYPE == LIN_BF16>;
  constexpr int N = R::N;
  u32x4_t xq[AHEAD][DIRECT ? 1 : XI], wq[AHEAD][DIRECT ? 1 : WI];
  auto load = [&](auto slot, int k) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
      constexpr bool BF16 = TYPE == LIN_BF16;
      using T = typename R::T;
      auto& xr = xq[decltype(slot)::value];
      auto& wr = wq[decltype(slot)::value];
      auto along = [&](const char* rows, int64_t ld, int r, int c) __attribute__((always_inline)) {
        const T* row = reinterpret_cast<const T*>(rows + r * ld);
        const int at = k * BK + c * N;
        if constexpr (TINY) {
          return load_raw<BF16>(row, at, p.k);
        } else {
          const typename R::Raw v = *reinterpret_cast<const typename R::Raw*>(row + min(at, p.k - N));
          return u32x4_t{v[0], v[1], v[2], v[3]};
        }
      };
#pragma unroll
      for (int i = 0; i < XI; ++i)
        xr[i] = along(x, p.ldx, min(x_at(i) / 8, rows_x - 1), x_at(i) % 8);
#pragma unroll
      for (int i = 0; i < WI; ++i) {
        if constexpr (ACROSS) {
          const T* row = reinterpret_cast<const T*>(static_cast<const char*>(p.W) + at.e * p.w_stride +
                                                    min(k * BK + w_at(i) / WPR, p.k - 1) * p.ldw);
          const int col = n0 + w_at(i) % WPR * N;
          if constexpr (TINY) {
            wr[i] = load_raw<BF16>(row, col, p.n);
          } else {
            const typename R::Raw v = *reinterpret_cast<const typename R::Raw*>(row + min(col, p.n - N));
            wr[i] = u32x4_t{v[0], v[1], v[2], v[3]};
          }
        } else {
          wr[i] = along(w, p.ldw, min(w_at(i) / 8, rows_w - 1), w_at(i) % 8);
        }
      }
    }
  };
  auto write = [&](auto slot, int buf, int k) __attribute__((always_inline)) {
    if constexpr (!DIRECT) {
      constexpr bool BF16 = TYPE == LIN_BF16;
      auto& xr = xq[decltype(slot)::value];
      auto& wr = wq[decltype(slot)::value];
      if (k == steps - 1 && last_k < BK) {
#pragma unroll
        for (int i = 0; i < XI; ++i)
          if (!TINY) shift_down<BF16>(xr[i], max(x_at(i) % 8 * N + N - last_k, 0));
#pragma unroll
        for (int i = 0; i < WI; ++i) {
          if (!ACROSS && !TINY) shift_down<BF16>(wr[i], max(w_at(i) % 8 * N + N - last_k, 0));
          if (ACROSS && w_at(i) / WPR >= last_k) wr[i] = u32x4_t{0, 0, 0, 0};
        }
      }
      if (ACROSS && rows_w < BN && !TINY) {
#pragma unroll
        for (int i = 0; i < WI; ++i) shift_down<BF16>(wr[i], max(n0 + w_at(i) % WPR * N - (p.n - N), 0));
      }
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
      return __builtin_bit_cast(u32x4_t, frag_across<BN>(tile, 16 * s, row0, lane));
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
      const uint32_t wsc = *reinterpret_cast<const LDS_AS uint8_t*>(smem + WS_AT + k);
      if constexpr (TYPE == LIN_E4M3_EXACT) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          bf16x8_t xf[MT][2], wf[NT][2];
          // both chunks of a fragment (one per half of the lanes) are of block c
#pragma unroll
          for (int a = 0; a < MT; ++a) widen(frag(s, xr0 + a * 32, c), sx[a] >> (8 * c) & 0xff, xf[a]);
#pragma unroll
          for (int b = 0; b < NT; ++b) widen(frag(sw, wr0 + b * 32, c), wsc, wf[b]);
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
      // small bf16 tiles read a whole step first, for a wave has too few products in
      // a chunk to wait for the next one's reads behind them (1023 tokens of 777 x
      // 1001: 17.3 -> 16.4 us)
      constexpr int FIRST = MT * NT == 1 && TYPE == LIN_BF16 ? 4 : 1;
#pragma unroll
      for (int c0 = 0; c0 < 4; c0 += FIRST) {
        u32x4_t xf[FIRST][MT], wf[FIRST][NT];
#pragma unroll
        for (int c = 0; c < FIRST; ++c) {
#pragma unroll
          for (int a = 0; a < MT; ++a) xf[c][a] = frag(s, xr0 + a * 32, c0 + c);
#pragma unroll
          for (int b = 0; b < NT; ++b) wf[c][b] = frag_w(sw, wr0 + b * 32, c0 + c);
        }
        if constexpr (FIRST > 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < FIRST; ++c)
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) {
              if constexpr (TYPE == LIN_BF16) {
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, wf[c][b]),
                                                                    __builtin_bit_cast(bf16x8_t, xf[c][a]),
                                                                    acc[a][b], 0, 0, 0);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(wf[c][b][i]),
                                                                   __uint_as_float(xf[c][a][i]), acc[a][b], 0, 0, 0);
              }
            }
      }
    }
  };

  if (steps > 0) {
    if constexpr (E4M3) {      // the weight's scales, all of k
      const uint8_t* ws = p.w_scale + at.e * p.ws_stride + int64_t(n0 / SIDE) * p.ws_row;
      for (int k = t; k < steps; k += THREADS)
        *reinterpret_cast<LDS_AS uint8_t*>(smem + WS_AT + k) = ws[k * p.ws_col];
    }
    if constexpr (DIRECT) {
      std::true_type end;
#pragma unroll
      for (int k = 0; k < STAGES - 1; ++k)
        if (k < steps) issue(end, k, k);
      int buf = 0;
      for (int k = 0; k < steps; ++k) {
        // step k has come: only the loads of the steps behind it may be on their way
        const int behind = min(steps - 1 - k, STAGES - 2);
        if (STAGES == 2 || behind == 0)
          wait_vmcnt<0>();
        else if (behind == 1)
          wait_vmcnt<LOADS>();
        else
          wait_vmcnt<2 * LOADS>();
        static_assert(STAGES == 2 || STAGES == 4, "the waits above");
        asm volatile("" ::: "memory");
        if (!E4M3 && k == steps - 1 && last_chunks < 8) clear_tail(buf);
        block_barrier();
        if (k + STAGES - 1 < steps) issue(end, (buf + STAGES - 1) % STAGES, k + STAGES - 1);
        multiply(buf, k);
        buf = (buf + 1) % STAGES;
      }
    } else {
      // Steps k + 1 .. k + AHEAD are on their way to registers while step k is
      // multiplied.  Behind the last step that one is loaded again: loads behind a
      // branch would all be waited for at the next write.
      auto step = [&](auto slot, int k) __attribute__((always_inline)) {
        constexpr int I = decltype(slot)::value;
        block_barrier();
        load(slot, min(k + AHEAD, steps - 1));
        multiply(k & 1, k);
        write(std::integral_constant<int, (I + 1) % AHEAD>{}, (k + 1) & 1, k + 1);
      };
      std::integral_constant<int, 0> c0;
      std::integral_constant<int, 1 % AHEAD> c1;
      std::integral_constant<int, 2 % AHEAD> c2;
      std::integral_constant<int, 3 % AHEAD> c3;
      load(c0, 0);
      load(c1, min(1, steps - 1));
      if constexpr (AHEAD == 4) {
        load(c2, min(2, steps - 1));
        load(c3, min(3, steps - 1));
      }
      write(c0, 0, 0);
      int k = 0;
      for (; k + AHEAD <= steps; k += AHEAD) {
        step(c0, k);
        step(c1, k + 1);
        if constexpr (AHEAD == 4) {
          step(c2, k + 2);
          step(c3, k + 3);
        }
      }
      if (k < steps) step(c0, k);
      if (k + 1 < steps) step(c1, k + 1);
      if (AHEAD == 4 && k + 2 < steps) step(c2, k + 2);
    }
    block_barrier();
  }
  store_tile<MT, NT, BM == 128>(p, t0 + wm * MT * 32, at.end, n0 + wn * NT * 32, acc,
                     smem + wave * window_bytes<NT>(), lane);
}

template <LinearType TYPE, bool ACROSS, LinearPath PATH, class S>
hipError_t launch_tiles(const Linear& p, hipStream_t s) {
  const int64_t tiles_n = cdiv(p.n, S::BN);
  // of the matrices, only those with tokens have tiles, and the tokens of none
  const int64_t tiles_m = p.offsets ? p.tokens / S::BM + std::min<int64_t>(p.count + 2, p.tokens)
                                    : cdiv(p.tokens, S::BM);
  hipLaunchKernelGGL((linear_kernel<TYPE, ACROSS, PATH, S>), dim3(unsigned(cdiv(tiles_m * tiles_n, 8) * 8)),
                     dim3(S::THREADS), 0, s, p, int(tiles_n));
  return hipGetLastError();
}
template <LinearType TYPE, bool ACROSS, LinearPath PATH>
hipError_t launch_shape(const Linear& p, LinearPlan plan, hipStream_t s) {
  return plan == LIN_64 ? launch_tiles<TYPE, ACROSS, PATH, Tile64>(p, s)
                        : launch_tiles<TYPE, ACROSS, PATH, Tile128>(p, s);
}
template <LinearType TYPE, bool ACROSS>
hipError_t launch_path(const Linear& p, LinearPath path, LinearPlan plan, hipStream_t s) {
  if (path == DIRECTLY) return launch_shape<TYPE, ACROSS, DIRECTLY>(p, plan, s);
  if (path == BY_VECTORS) return launch_shape<TYPE, ACROSS, BY_VECTORS>(p, plan, s);
  return launch_tiles<TYPE, ACROSS, BY_ELEMENTS, Tile64>(p, s);
}

}  // namespace

// Estimates of the tiles of `bm` tokens that a call has: matrices share the tokens
// evenly, and half of a tile of each lies behind its last token.
static double tiles_of(int64_t count, int64_t tokens, int64_t n, int bm, int bn) {
  const double hit = double(std::min(count, std::max<int64_t>(tokens, 1))), each = double(tokens) / hit;
  return hit * std::max(1.0, each / bm + (count > 1 ? 0.5 : 0.0)) * double(cdiv(n, bn));
}

// Which kernel, by times measured on one MI355X for 1, 8 and 64 matrices of 1408 x
// 512 to 5632 x 2048 and 1 to 16384 tokens (microseconds, bf16 unless said).
static LinearPlan choose(LinearType type, bool across, int64_t count, int64_t tokens, int64_t k, int64_t n) {
  const double few = tiles_of(count, tokens, n, 16, 16), n64 = tiles_of(count, tokens, n, 64, 64),
               n128 = tiles_of(count, tokens, n, 128, 128), n256 = tiles_of(count, tokens, n, 256, 256);
  // Few tokens, while the blocks are all there at once (1 token of 4096 x 1024: 6.0,
  // tiles of 64 9.5; 64 tokens 12.9 and 9.7).  float32, whose tiles are slow, where
  // the tokens of a matrix are few (64 matrices of 1408 x 512, 1024 tokens: 57, 65).
  if (!across && (few <= 768 || (type == LIN_F32 && tokens <= 16 * count))) return LIN_FEW;
  if (type == LIN_F32) {
    // bound by the matrix instructions: the fewer products with nothing, a tile of
    // 128 taking 3.3 times one of 64 (4096 tokens of 64 x 1408 x 512: 102 against 68;
    // of one 1024 x 1024: 78 against 89)
    return n128 >= 200 && 3.3 * n128 <= n64 ? LIN_128 : LIN_64;
  }
  // Tiles of 64 until those of 128 fill the chip (1024 tokens of 1024 x 1024: 10.3
  // against 14.9; 4096: 22.7 against 17.7).
  if (n64 <= 640) return LIN_64;
  if (type == LIN_E4M3_EXACT) return LIN_128;
  // Blocks that stay, from two per CU on (16384 tokens of 64 x 1408 x 512: 40 against
  // 47), and not across the rows, where they gained nothing before they stored whole
  // lines (tried since, between other calls: 16384 tokens of 64 x 1408 x 512 53 us
  // against 56 in the tiles here, 49152 109 against 111, of 64 x 512 x 1408 110 against
  // 128, 32768 of 16 x 2048 x 1024 165 against 179: not built); and their tiles of
  // 256 x 256, which read half as much, where whole rounds of them do not lose it again
  // (16384 tokens of 4096 x 2048: 227, of 128 x 128 255; of 1408 x 512: 36 against 30).
  const double steps = double(k) * (type == LIN_E4M3 ? 1 : 2) / ROWB;
  const double step256 = type == LIN_E4M3 ? 1.22 : across ? 1.62 : 1.34, step128 = across ? 0.88 : 0.93;
  const double us256 = std::ceil(n256 / 256) * (step256 * steps + 10),
               us128 = std::max(1.0, n128 / 512) * (step128 * steps + 3);
  // (whole steps of k, and rows of outputs of whole 16 bytes)
  const bool whole = k % (type == LIN_E4M3 ? 128 : 64) == 0 && n % 8 == 0;
  if (whole && us256 < us128) return LIN_STREAM_256;
  return whole && n128 >= 512 && !across ? LIN_STREAM_128 : LIN_128;
}

LinearPlan linear_plan(LinearType type, bool across, int64_t count, int64_t tokens, int64_t k, int64_t n) {
  LinearPlan plan = choose(type, across, count, tokens, k, n);
  // operands' rows of less than 16 bytes are loaded by the element, in tiles of 64
  const int64_t vec = type == LIN_BF16 ? 8 : 4;
  if (type <= LIN_F32 && plan != LIN_FEW && (k < vec || (across && n < vec))) plan = LIN_64;
  // the largest grid, with whole turns of the 8 XCDs (rows that do not start on 16
  // bytes may take tiles of 128 instead of 256)
  const int64_t side = plan == LIN_FEW ? 16 : plan == LIN_64 ? 64 : 128;
  return (tokens / side + count + 2) * cdiv(n, side) >= (int64_t(1) << 24) - 8 ? LIN_NONE : plan;
}

hipError_t launch_linear(const Linear& p, LinearType type, bool across, LinearPlan plan, hipStream_t s) {
  const int es = type == LIN_BF16 ? 2 : 4, vec = 16 / es;
  // whole chunks in both operands' rows, and offsets within a tile in 32 bits
  const bool direct = type >= LIN_E4M3 ||
                      (reinterpret_cast<uintptr_t>(p.x) % 16 == 0 && reinterpret_cast<uintptr_t>(p.W) % 16 == 0 &&
                       p.ldx % 16 == 0 && p.ldw % 16 == 0 && p.k % vec == 0 && (!across || p.n % vec == 0) &&
                       p.ldx <= (1 << 23));
  const LinearPath path = direct                                       ? DIRECTLY
                          : p.k >= vec && (!across || p.n >= vec) ? BY_VECTORS
                                                                       : BY_ELEMENTS;
  if (plan == LIN_FEW) return launch_linear_few(p, type, s);
  if ((plan == LIN_STREAM_128 || plan == LIN_STREAM_256) && direct)
    return launch_linear_stream(p, type, across, plan == LIN_STREAM_256 ? 256 : 128, s);
  switch (type) {
    case LIN_E4M3_EXACT: return launch_shape<LIN_E4M3_EXACT, false, DIRECTLY>(p, plan, s);
    case LIN_E4M3: return launch_shape<LIN_E4M3, false, DIRECTLY>(p, plan, s);
    case LIN_BF16:
      return across ? launch_path<LIN_BF16, true>(p, path, plan, s) : launch_path<LIN_BF16, false>(p, path, plan, s);
    default:
      return across ? launch_path<LIN_F32, true>(p, path, plan, s) : launch_path<LIN_F32, false>(p, path, plan, s);
  }
}

}  // namespace muon
