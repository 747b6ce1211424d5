// Weight gradients from 8-bit activation checkpoints:
//
//   G[e] (+)= sum_t dy[t]^T x[t]     (rows x cols, t over the tokens of e)
//
// The contraction runs over tokens, the slow axis of both operands, so both
// are staged as token rows in LDS and read as MFMA fragments with transposing
// LDS reads.  x is brought back from 8 bits when it is written to LDS: a
// checkpoint's values are exact in bf16, so bf16 matrix cores see exactly what
// it holds.  float32 dy is split into three bf16 parts of 8 bits each
// (remainders exact, see split3), whose three products per element replace the sixteen
// times slower float32 matrix instruction.
//
// Bound by the matrix cores for many tokens (an element of G takes 2 flops per
// token, of dy and x 2 cols and 2 rows).  Measured on one MI355X, 4096 x 1024 over
// 16384 tokens: bf16 dy 123 us with e4m3 x in a row of the same call, 131 among
// others (1050 TFLOP/s; 98.6 us at the rate of a large library product), 127 with
// int8; float32 dy 426 with e4m3, 441 with int8.  For few tokens it is bound by the latency of a launch and one tile (768 x 768 over
// 96: 5.4 us), in between by the partial sums' traffic.
//
// The tokens of a matrix are cut into pieces of at most `chunk`; every block
// computes one tile over one piece.  A matrix of one piece is written at once,
// one of several leaves float32 tiles that the join kernel adds in order: no
// atomics, the same bits on every run.
#include <algorithm>
#include <type_traits>

#include "lds_tiles.h"
#include "layer_internal.h"

namespace muon {
namespace {

constexpr int BM = 128, BN = 128, BK = 32;   // rows of G, columns of G, tokens
constexpr int kThreads = 256;                // 2 x 2 waves of 64 x 64

// A piece: tokens [begin, end) of matrix e; slot: its place among the partial
// sums (parts > 1).  In the table of a ragged call, e < 0 marks no piece.
struct Piece {
  int e, begin, end, parts;
  int64_t slot;
  int64_t pad_;
};
static_assert(sizeof(Piece) == kWeightGradPieceBytes, "size of the table");
// A matrix of several pieces, for the join.
struct Split {
  int e, parts;
  int64_t slot;
};
static_assert(sizeof(Split) == kWeightGradSplitBytes, "size of the table");

// Ragged calls: the pieces of all matrices and the list of the split ones,
// from the offsets on the device.  One block; a thread takes a matrix.  The
// offsets are clamped to [0, tokens] and read as the largest so far, so that
// no piece leaves the buffers and their number is bounded whatever the offsets
// hold.  A matrix's tokens are shared evenly between its pieces, in whole
// steps.  Up to 128 matrices, pieces are put in order of their length,
// longest first: blocks start in this order, so that all end together.  Up to
// 64 matrices need one wave (NT = 64), up to 128 are compared by all threads, a
// share of them each.  Ordered against as they come, uneven, bf16, int8 x: 96 of
// 1408 x 512 over 49152 tokens 108 and 136 us, 128 of 768 x 512 70.5 and 79, 128 of
// 128 x 128 over 16384 20.0 and 18.7; ordering 256 of 1408 x 512 gains nothing (176)
// and of 128 x 128 costs 6 of 18.  The plan takes 6 to 7 us ordered, 5 unordered.
constexpr int kPlanThreads = 1024, kPlanOrdered = 128;
template <int NT>
__global__ __launch_bounds__(NT) void plan_kernel(const WeightGrad p) {
  constexpr int WAVES = NT / 64, SHARES = NT / kPlanOrdered;
  __shared__ int wave_top[WAVES], wave_n[WAVES], wave_m[WAVES], wave_s[WAVES];
  __shared__ int keys[NT], counts[NT], ranks[NT];
  Piece* table = static_cast<Piece*>(p.table);
  Split* splits = reinterpret_cast<Split*>(table + p.pieces);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int T = int(p.tokens);
  auto clamp = [&](int64_t v) { return int(v < 0 ? 0 : v > T ? T : v); };
  int top = clamp(p.offsets[0]);
  int pieces = 0, slots = 0, split = 0;   // of the matrices before this group
  for (int base = 0; base < p.count; base += NT) {
    const int e = base + t;
    const bool in = e < p.count;
    // end of every matrix: the largest offset up to it
    int hi = in ? clamp(p.offsets[e + 1]) : 0;
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
    for (int w = 0; w < WAVES; ++w) top = top > wave_top[w] ? top : wave_top[w];
    // pieces, slots and split matrices before this one
    const int len = hi - lo, chunk = int(p.chunk);
    const int n = !in ? 0 : len <= chunk ? 1 : (len - 1) / chunk + 1;
    const int m = n > 1 ? n : 0, d = n > 1 ? 1 : 0;
    int sn = n, sm = m, sd = d;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(sn, off, 64), y = __shfl_up(sm, off, 64), z = __shfl_up(sd, off, 64);
      if (lane >= off) {
        sn += x;
        sm += y;
        sd += z;
      }
    }
    if (lane == 63) {
      wave_n[wave] = sn;
      wave_m[wave] = sm;
      wave_s[wave] = sd;
    }
    const int share = n > 1 ? ((len + n - 1) / n + BK - 1) / BK * BK : len;
    keys[t] = share;
    counts[t] = n;
    __syncthreads();
    int first = pieces + sn - n, slot = slots + sm - m, at = split + sd - d;
    for (int w = 0; w < wave; ++w) {
      first += wave_n[w];
      slot += wave_m[w];
      at += wave_s[w];
    }
    if (p.count <= (NT == 64 ? 64 : kPlanOrdered)) {
      first = 0;
      if constexpr (NT == 64) {
#pragma unroll
        for (int j = 0; j < 64; ++j) {   // lanes past the last matrix have no pieces
          const int kj = __builtin_amdgcn_readlane(share, j), nj = __builtin_amdgcn_readlane(n, j);
          first += kj > share || (kj == share && j < t) ? nj : 0;
        }
      } else {
        const int me = t % kPlanOrdered, key = keys[me];
        int s = 0;
        for (int j = t / kPlanOrdered; j < p.count; j += SHARES)
          s += keys[j] > key || (keys[j] == key && j < me) ? counts[j] : 0;
        ranks[t] = s;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < SHARES; ++i) first += ranks[i * kPlanOrdered + me];
      }
    }
    for (int j = 0; j < n; ++j) {
      Piece pc{};
      pc.e = e;
      pc.begin = j * share < len ? lo + j * share : hi;
      pc.end = hi - pc.begin > share ? pc.begin + share : hi;
      pc.parts = n;
      pc.slot = slot + j;
      table[first + j] = pc;
    }
    if (d) splits[at] = Split{e, n, slot};
    for (int w = 0; w < WAVES; ++w) {
      pieces += wave_n[w];
      slots += wave_m[w];
      split += wave_s[w];
    }
    __syncthreads();
  }
  for (int64_t i = pieces + t; i < p.pieces; i += NT) table[i].e = -1;
  if (t == 0) splits[p.count] = Split{split, 0, 0};   // their number
}

// The piece and tile of block `b`.  The hardware deals blocks to the 8 XCDs in
// turn; tiles that share operands are put on one XCD, which has an L2 of its
// own: without offsets XCD x takes a contiguous eighth of all tiles, with
// them the tiles of a piece (at most 32 at a time, an XCD's compute units) go
// to the XCDs in turn.
__device__ __forceinline__ bool find_piece(const WeightGrad& p, uint32_t b, uint32_t tiles,
                                           Piece& out, int& tile) {
  const uint32_t turn = b >> 3, pieces = uint32_t(p.pieces);
  if (!p.offsets) {
    const uint32_t per = (pieces * tiles + 7) / 8, id = (b & 7) * per + turn;
    if (turn >= per || id >= pieces * tiles) return false;
    const uint32_t want = id / tiles;
    tile = int(id - want * tiles);
    out.e = 0;
    out.begin = int(want * p.chunk);
    out.end = int(out.begin + p.chunk < p.tokens ? out.begin + p.chunk : p.tokens);
    out.parts = int(pieces);
    out.slot = want;
    return true;
  }
  const uint32_t deal = tiles < 32 ? tiles : 32;
  const uint32_t id = (turn / deal * 8 + (b & 7)) * deal + turn % deal;
  const uint32_t want = id / tiles;
  tile = int(id - want * tiles);
  if (want >= pieces) return false;
  const Piece pc = static_cast<const Piece*>(p.table)[want];
  out.e = __builtin_amdgcn_readfirstlane(pc.e);
  out.begin = __builtin_amdgcn_readfirstlane(pc.begin);
  out.end = __builtin_amdgcn_readfirstlane(pc.end);
  out.parts = __builtin_amdgcn_readfirstlane(pc.parts);
  out.slot = __builtin_amdgcn_readfirstlane(int(pc.slot));
  return out.e >= 0;
}

// Tile number -> tile row and column: groups of 8 tile rows, columns first
// within a group, so that 32 consecutive tiles (an XCD's compute units) read
// 8 column strips of dy and 4 of x.
__device__ __forceinline__ void place_tile(int tile, int tiles_m, int tiles_n, int& ti, int& tj) {
  const int group = tile / (8 * tiles_n), r = tile - group * 8 * tiles_n;
  const int rows = tiles_m - group * 8 < 8 ? tiles_m - group * 8 : 8;
  tj = r / rows;
  ti = group * 8 + r - tj * rows;
}

// Eight consecutive columns of one row into a bf16 gradient.  The L2 need not
// keep what is stored (64 even experts of 1408 x 512 over 49152 tokens: 89 -> 82
// us; float32 over 16384: 117 -> 113): the join's reads of partial sums come from
// the Infinity Cache all the same (1001 x 777 over 2049: 29.9 -> 28.5).
__device__ __forceinline__ void store_bf16(const WeightGrad& p, int64_t base, int row, int col,
                                           f32x4_t lo, f32x4_t hi) {
  if (row >= p.rows || col >= p.cols) return;
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = lo[i];
    v[4 + i] = hi[i];
  }
  const int left = p.cols - col;
  uint16_t* g = static_cast<uint16_t*>(p.G) + base + int64_t(row) * p.cols + col;
  if (p.accumulate) {
    float old[8];
    load_vec<true>(g, 0, left, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += old[i];
  }
  store_vec<true, true>(g, 0, left, v);
}
// Four into a float32 matrix: the gradient, or a piece's partial sums.
__device__ __forceinline__ void store_f32(const WeightGrad& p, float* to, bool add, int row, int col,
                                          f32x4_t x) {
  if (row >= p.rows || col >= p.cols) return;
  float v[4] = {x[0], x[1], x[2], x[3]};
  const int left = p.cols - col;
  to += int64_t(row) * p.cols + col;
  if (add) {
    float old[4];
    load_vec<false>(to, 0, left, old);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += old[i];
  }
  store_vec<false, true>(to, 0, left, v);
}

// Writes a wave's 32 MI x 64 accumulators (rows from i0, columns from j0)
// through a window of LDS of its own, 32 rows at a time, so that lanes store
// whole runs of a row.  Lane l, register 4 g + i of a 32 x 32 block holds row
// l % 32, column 8 g + 4 (l / 32) + i.  A pitch of 68 floats spreads the
// 16-byte writes of 16 rows over all banks.
constexpr int kWindow = 32 * 68 * 4;   // bytes per wave
template <int MI>
__device__ __forceinline__ void store_tile(const WeightGrad& p, const Piece& pc, int i0, int j0,
                                           const f32x16_t (&acc)[MI][2], LDS_AS char* window,
                                           int lane) {
  const int64_t size = int64_t(p.rows) * p.cols;
  const bool whole = pc.parts == 1, f32 = !whole || !p.g_bf16;
  float* to = whole ? static_cast<float*>(p.G) + pc.e * size : p.partial + pc.slot * size;   // f32
  LDS_AS float* w = (LDS_AS float*)window;
#pragma unroll
  for (int a = 0; a < MI; ++a) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(LDS_AS f32x4_t*)(w + (lane & 31) * 68 + b * 32 + 8 * g + 4 * (lane >> 5)) =
            f32x4_t{acc[a][b][4 * g], acc[a][b][4 * g + 1], acc[a][b][4 * g + 2],
                    acc[a][b][4 * g + 3]};
    wave_lds_sync();
    if (f32) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int row = r * 4 + (lane >> 4), col = (lane & 15) * 4;
        store_f32(p, to, whole && p.accumulate, i0 + a * 32 + row, j0 + col,
                  *(const LDS_AS f32x4_t*)(w + row * 68 + col));
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = r * 8 + (lane >> 3), col = (lane & 7) * 8;
        store_bf16(p, pc.e * size, i0 + a * 32 + row, j0 + col,
                   *(const LDS_AS f32x4_t*)(w + row * 68 + col),
                   *(const LDS_AS f32x4_t*)(w + row * 68 + col + 4));
      }
    }
    wave_lds_sync();
  }
}

// Four checkpoint bytes -> four bf16, exact; a marked block gives NaN.
template <int FMT>
__device__ __forceinline__ void unpack4(uint32_t q, int byte, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == MUON_CKPT_E4M3) {
    // the conversion scales by the exponent of `up`, 255 giving NaN
    const float up = __uint_as_float(uint32_t(byte) << 23);
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, up, false));
    hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, up, true));
  } else {
    // each byte is converted with its sign before it is scaled: at the largest
    // scales an offset times 2^e would be infinite where the values are not
    float v[4];
    ckpt_unpack4(q, ckpt_up(byte), FMT, v);
    lo = f2bf2(v[0], v[1]);
    hi = f2bf2(v[2], v[3]);
  }
}

// Two float32 values as three bf16 pairs that add up to them exactly, down to
// bf16's smallest step of 2^-133 (the 24 bits of a value below 2^-109 reach further
// down: at most 2^-134 of it is rounded off).  The first is cut off, for a value
// near the largest must not become an infinity (which itself leaves no
// remainder); 16 bits remain, whose half is rounded off and leaves 8.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&o)[3]) {
  const uint32_t a = __float_as_uint(x) & 0xffff0000u, b = __float_as_uint(y) & 0xffff0000u;
  o[0] = (a >> 16) | b;
  const float fa = __uint_as_float(a), fb = __uint_as_float(b);
  x = x == fa ? 0.f : x - fa;
  y = y == fb ? 0.f : y - fb;
  o[1] = f2bf2(x, y);
  o[2] = f2bf2(x - __uint_as_float(o[1] << 16), y - __uint_as_float(o[1] & 0xffff0000u));
}

// Byte address of the 8 columns `chunk` of token row k in a [BK][128] tile.
__device__ __forceinline__ int tile_at(int k, int chunk) {
  return k * (BN * 2) + ((chunk ^ gswz(k)) << 4);
}

template <bool BF16, int FMT>
__global__ __launch_bounds__(kThreads, 2) void weight_grad_kernel(const WeightGrad p, int tiles_m,
                                                            int tiles_n) {
  constexpr int P = BF16 ? 1 : 3;            // bf16 parts of dy
  constexpr int PLANE = BK * BM * 2;         // bytes
  constexpr int STAGE = (P + 1) * PLANE;
  static_assert(BM == BN, "one tile layout");
  constexpr int WINDOWS = kThreads / 64 * kWindow;   // of the epilogue
  __shared__ __attribute__((aligned(1024))) char smem_raw[2 * STAGE > WINDOWS ? 2 * STAGE : WINDOWS];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;

  Piece pc;
  int tile, ti, tj;
  if (!find_piece(p, blockIdx.x, tiles_m * tiles_n, pc, tile)) return;
  place_tile(tile, tiles_m, tiles_n, ti, tj);
  const int i0 = ti * BM, j0 = tj * BN;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // This thread's part of a step: 8 columns of dy of two tokens, 16 of x of one.
  // D steps are in flight, each in registers of its own.
  constexpr int D = BF16 ? 4 : 2;
  const int yk = t >> 4, yc = t & 15;
  const int xk = t >> 3, xc = t & 7;
  using T = typename RowVec<BF16>::T;
  constexpr int N = RowVec<BF16>::N, W = 8 / N;   // vectors per 8 columns
  u32x4_t y[D][2][W], q[D];
  int scale[D];
  // Every lane loads: tokens past the end the last one (their dy is zeroed when
  // it is written), vectors past a row's end its last (columns past the end
  // reach nothing that is stored; one that crosses it is shifted when written).
  // Loads that no branch guards can be waited for one step at a time.
  auto load = [&](auto end, auto slot, int k0) __attribute__((always_inline)) {
    constexpr int I = decltype(slot)::value;
    constexpr RowEnd HOW = decltype(end)::value == END_SHORT ? END_SHORT : END_INSIDE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + yk + 16 * h;
      const T* row = static_cast<const T*>(p.dy) + int64_t(k < pc.end ? k : pc.end - 1) * p.lddy;
#pragma unroll
      for (int i = 0; i < W; ++i)
        y[I][h][i] = load_ahead<BF16, HOW>(row, i0 + yc * 8 + i * N, p.rows);
    }
    const int k = k0 + xk, col = j0 + xc * 16;
    const int64_t token = k < pc.end ? k : pc.end - 1;
    const int at = col < p.x.q_pitch ? col : int(p.x.q_pitch) - 16;
    q[I] = *reinterpret_cast<const u32x4_t*>(p.x.q + token * p.x.q_pitch + at);
    scale[I] = p.x.scale[token * p.x.s_pitch + at / MUON_CKPT_BLOCK];
  };
  int by[W];   // elements by which a vector at the row's end was loaded too early
#pragma unroll
  for (int i = 0; i < W; ++i) by[i] = max(0, i0 + yc * 8 + i * N - (p.rows - N));
  auto write = [&](auto end, auto slot, int buf, int k0) __attribute__((always_inline)) {
    constexpr int I = decltype(slot)::value;
    LDS_AS char* s = smem + buf * STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if constexpr (decltype(end)::value == END_INSIDE) shift_down<BF16>(y[I][h][i], by[i]);
      if (k0 + yk + 16 * h >= pc.end) {
#pragma unroll
        for (int i = 0; i < W; ++i) y[I][h][i] = u32x4_t{0, 0, 0, 0};
      }
      if constexpr (BF16) {
        *reinterpret_cast<LDS_AS u32x4_t*>(s + tile_at(yk + 16 * h, yc)) = y[I][h][0];
      } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < W; ++i) unpack_raw<false>(y[I][h][i], v + i * N);
        uint32_t o[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3(v[2 * i], v[2 * i + 1], o[i]);
#pragma unroll
        for (int part = 0; part < P; ++part)
          *reinterpret_cast<LDS_AS u32x4_t*>(s + part * PLANE + tile_at(yk + 16 * h, yc)) =
              u32x4_t{o[0][part], o[1][part], o[2][part], o[3][part]};
      }
    }
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack4<FMT>(q[I][i], scale[I], o[2 * i], o[2 * i + 1]);
    LDS_AS char* sx = s + P * PLANE;
    *reinterpret_cast<LDS_AS u32x4_t*>(sx + tile_at(xk, 2 * xc)) = u32x4_t{o[0], o[1], o[2], o[3]};
    *reinterpret_cast<LDS_AS u32x4_t*>(sx + tile_at(xk, 2 * xc + 1)) = u32x4_t{o[4], o[5], o[6], o[7]};
  };

  f32x16_t acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  const int steps = (pc.end - pc.begin + BK - 1) / BK;
  // Step k, in slot I = k % D: its loads are in LDS; its slot takes those of step
  // k + D, and the next slot's go to the other buffer.  LAST: there may be no such
  // steps.  (Loads behind a branch would all be waited for at the next write.)
  auto step = [&](auto end, auto slot, auto last, int k) __attribute__((always_inline)) {
    constexpr int I = decltype(slot)::value;
    constexpr bool LAST = decltype(last)::value;
    const LDS_AS char* s = smem + (I & 1) * STAGE;
    bf16x8_t xf[BK / 16][2], yf[BK / 16][P][2];
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        xf[ks][b] = lds_frag_xT<BN>(s + P * PLANE, ks * 16, wn * 64 + b * 32, lane);
#pragma unroll
      for (int part = 0; part < P; ++part)
#pragma unroll
        for (int a = 0; a < 2; ++a)
          yf[ks][part][a] = lds_frag_xT<BM>(s + part * PLANE, ks * 16, wm * 64 + a * 32, lane);
    }
    if (!LAST || k + D < steps) load(end, slot, pc.begin + (k + D) * BK);
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
#pragma unroll
      for (int part = P - 1; part >= 0; --part)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf[ks][b], yf[ks][part][a], acc[a][b],
                                                                0, 0, 0);
      if (ks == 0 && (!LAST || k + 1 < steps))
        write(end, std::integral_constant<int, (I + 1) % D>{}, (I + 1) & 1, pc.begin + (k + 1) * BK);
    }
    block_barrier();
  };
  static_assert(D % 2 == 0, "the buffer of a step follows from its slot");
  std::integral_constant<int, 0> c0;
  std::integral_constant<int, 1> c1;
  std::integral_constant<int, 2 % D> c2;
  std::integral_constant<int, 3 % D> c3;
  auto run = [&](auto end) __attribute__((always_inline)) {
    load(end, c0, pc.begin);
    if (steps > 1) load(end, c1, pc.begin + BK);
    if constexpr (D > 2) {
      if (steps > 2) load(end, c2, pc.begin + 2 * BK);
      if (steps > 3) load(end, c3, pc.begin + 3 * BK);
    }
    write(end, c0, 0, pc.begin);
    block_barrier();
    int k = 0;
    for (; k + 2 * D <= steps; k += D) {
      step(end, c0, std::false_type{}, k);
      step(end, c1, std::false_type{}, k + 1);
      if constexpr (D > 2) {
        step(end, c2, std::false_type{}, k + 2);
        step(end, c3, std::false_type{}, k + 3);
      }
    }
    std::true_type last;
    for (; k < steps; k += D) {
      step(end, c0, last, k);
      if (k + 1 < steps) step(end, c1, last, k + 1);
      if constexpr (D > 2) {
        if (k + 2 < steps) step(end, c2, last, k + 2);
        if (k + 3 < steps) step(end, c3, last, k + 3);
      }
    }
  };
  if (steps > 0) {
    if (p.rows % N == 0 || i0 + BM <= p.rows)
      run(std::integral_constant<RowEnd, END_WHOLE>{});
    else if (p.rows >= N)
      run(std::integral_constant<RowEnd, END_INSIDE>{});
    else
      run(std::integral_constant<RowEnd, END_SHORT>{});
  }

  if (pc.parts == 1 && steps == 0 && p.accumulate) return;
  store_tile<2>(p, pc, i0 + wm * 64, j0 + wn * 64, acc, smem + wave * kWindow, lane);
}

// ------------------------------------------------------ bf16 dy in aligned rows
// Tiles of 256 x 256, one block of 8 waves per CU, waves of 128 x 64.  Steps of
// 32 tokens: dy, the 8-bit x and its scales go straight to LDS; each wave turns
// the x bytes that it loaded itself into its part of the bf16 tile two steps
// ahead.
struct Wide {
  static constexpr int NW = 8, BM = 256, BN = 256, WGN = 4, MI = 4, NI = 2;
  static constexpr int YS = 4, XS = 4, QS = 2;   // buffers of dy, bf16 x, x bytes with scales
  static constexpr int Y_BYTES = BK * BM * 2, X_BYTES = BK * BN * 2;
  static constexpr int Q_BYTES = BK * BN, QW_BYTES = Q_BYTES + NW * 256;
  static constexpr int Y_INSTR = Y_BYTES / NW / WAVE_BYTES;
  static constexpr int X_AT = YS * Y_BYTES, Q_AT = X_AT + XS * X_BYTES;
  static constexpr int LDS = Q_AT + QS * QW_BYTES;
  static_assert(Q_BYTES == NW * WAVE_BYTES, "one x load per wave");
  static_assert(QW_BYTES <= X_BYTES, "x bytes of the first steps in unused x tiles");
  static_assert(LDS >= NW * kWindow && LDS <= 160 * 1024, "LDS");
};

// Byte address of the 8 columns `chunk` of token row k in a [BK][W] tile of
// bf16 x.  On top of the swizzle that the fragment reads need, the upper half
// of a 512-byte row is shifted by a chunk: lanes that write every other chunk
// of a row then use all banks once.
template <int W>
__device__ __forceinline__ int x_at(int k, int chunk) {
  return k * (W * 2) + ((chunk ^ gswz(k) ^ ((chunk >> 4) & 1)) << 4);
}
// Fragment of a tile laid out so: lane l gets column nb + l % 32, tokens
// kb + 8 (l / 32) .. + 7 (lds_frag_xT with the shift).
template <int W>
__device__ __forceinline__ bf16x8_t frag_x(const LDS_AS char* tile, int kb, int nb, int lane) {
  const int s = lane & 15;
  const int n = nb + 16 * ((lane >> 4) & 1) + 4 * (s & 3);
  const int k = kb + 8 * (lane >> 5) + (s >> 2);
  const LDS_AS char* p0 = tile + x_at<W>(k, n >> 3) + (n & 7) * 2;
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)p0);
  const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(p0 + 4 * W * 2));
  const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

template <int FMT>
__global__ __launch_bounds__(64 * Wide::NW, 1) void weight_grad_wide_kernel(
    const WeightGrad p, int tiles_m, int tiles_n) {
  using C = Wide;
  constexpr int BM = C::BM, BN = C::BN, MI = C::MI, NI = C::NI;
  __shared__ __attribute__((aligned(1024))) char smem_raw[C::LDS];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;
  const uint32_t smem_base = uint32_t(reinterpret_cast<uintptr_t>(smem));

  Piece pc;
  int tile, ti, tj;
  if (!find_piece(p, blockIdx.x, tiles_m * tiles_n, pc, tile)) return;
  place_tile(tile, tiles_m, tiles_n, ti, tj);
  const int i0 = ti * BM, j0 = tj * BN;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  const int len = pc.end - pc.begin;
  const int steps = (len + BK - 1) / BK;
  const int last = len - (steps - 1) * BK;   // tokens of the last step

  // Addresses of this lane's loads within a step.  Columns past a row's end
  // read its last ones instead (they only reach elements of G that are not
  // stored), tokens past the end the last token (their dy is zeroed below).
  int y_k[C::Y_INSTR];
  uint32_t y_off[C::Y_INSTR];
  const uint32_t y_ld = uint32_t(p.y_ld) * 2;
#pragma unroll
  for (int i = 0; i < C::Y_INSTR; ++i) {
    constexpr int CPR = BM / 8;   // chunks per token row
    const int at = (wave * C::Y_INSTR + i) * 64 + lane;
    y_k[i] = at / CPR;
    const int col = i0 + ((at % CPR) ^ gswz(y_k[i])) * 8;
    y_off[i] = uint32_t(y_k[i]) * y_ld + uint32_t(col < p.y_cols ? col : p.y_cols - 8) * 2;
  }
  constexpr int XL = BN / 16;     // lanes per token row of x
  const int x_k = wave * (64 / XL) + lane / XL, x_c = lane % XL;
  const int x_col = j0 + x_c * 16, s_col = (j0 / MUON_CKPT_BLOCK) + (x_c / 2 & ~3);
  const uint32_t q_ld = uint32_t(p.x.q_pitch), s_ld = uint32_t(p.x.s_pitch);
  const uint32_t q_off = uint32_t(x_k) * q_ld + (x_col < int(q_ld) ? x_col : int(q_ld) - 16);
  const uint32_t s_off = uint32_t(x_k) * s_ld + (s_col < int(s_ld) ? s_col : int(s_ld) - 4);
  const char* y_base = reinterpret_cast<const char*>(p.y) + int64_t(pc.begin) * y_ld;
  const char* q_base = reinterpret_cast<const char*>(p.x.q) + int64_t(pc.begin) * q_ld;
  const char* s_base = reinterpret_cast<const char*>(p.x.scale) + int64_t(pc.begin) * s_ld;

  // Loads of step k: dy into buffer J; the bytes and scales of x to byte `at` of
  // LDS.  END: k may be of
  // the last tokens.
  auto issue_y = [&](auto buf, auto end, int i, int k) {
    constexpr int J = decltype(buf)::value;
    uint32_t off = y_off[i];
    if (decltype(end)::value && k >= steps - 1 && y_k[i] >= last)
      off -= uint32_t(y_k[i] - (last - 1)) * y_ld;
    dma16(off, y_base + int64_t(k) * BK * y_ld,
          smem_base + J * C::Y_BYTES + (wave * C::Y_INSTR + i) * WAVE_BYTES);
  };
  auto issue_q = [&](auto end, int at, int k) {
    uint32_t off = q_off;
    if (decltype(end)::value && k >= steps - 1 && x_k >= last) off -= uint32_t(x_k - (last - 1)) * q_ld;
    dma16(off, q_base + int64_t(k) * BK * q_ld, smem_base + at + wave * WAVE_BYTES);
  };
  auto issue_s = [&](auto end, int at, int k) {
    uint32_t off = s_off;
    if (decltype(end)::value && k >= steps - 1 && x_k >= last) off -= uint32_t(x_k - (last - 1)) * s_ld;
    dma4(off, s_base + int64_t(k) * BK * s_ld, smem_base + at + C::Q_BYTES + wave * 256);
  };
  // This wave's x bytes of a step, and its part of their bf16 tile X.
  u32x4_t q;
  uint32_t sw;
  auto read_q = [&](int at) {
    q = *reinterpret_cast<const LDS_AS u32x4_t*>(smem + at + wave * WAVE_BYTES + lane * 16);
    sw = *reinterpret_cast<const LDS_AS uint32_t*>(smem + at + C::Q_BYTES + wave * 256 + lane * 4);
  };
  uint32_t o[8];
  auto unpack = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      unpack4<FMT>(q[i], (sw >> (8 * ((x_c / 2) & 3))) & 0xff, o[2 * i], o[2 * i + 1]);
  };
  auto write_x = [&](auto tile_x) {
    LDS_AS char* x = smem + C::X_AT + decltype(tile_x)::value * C::X_BYTES;
    *reinterpret_cast<LDS_AS u32x4_t*>(x + x_at<BN>(x_k, 2 * x_c)) = u32x4_t{o[0], o[1], o[2], o[3]};
    *reinterpret_cast<LDS_AS u32x4_t*>(x + x_at<BN>(x_k, 2 * x_c + 1)) = u32x4_t{o[4], o[5], o[6], o[7]};
  };
  // dy of the tokens past the end, in buffer J of the last step: zero.
  auto zero_tail = [&](auto buf) {
#pragma unroll
    for (int i = 0; i < C::Y_INSTR; ++i)
      if (y_k[i] >= last)
        *reinterpret_cast<LDS_AS u32x4_t*>(smem + decltype(buf)::value * C::Y_BYTES +
                                           (wave * C::Y_INSTR + i) * WAVE_BYTES + lane * 16) =
            u32x4_t{0, 0, 0, 0};
  };

  f32x16_t acc[MI][NI];
#pragma unroll
  for (int a = 0; a < MI; ++a)
#pragma unroll
    for (int b = 0; b < NI; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  bf16x8_t yf[2][MI], xf[2][NI];
  auto frags = [&](auto buf, auto tile_x, int ks) {
    constexpr int J = decltype(buf)::value, X = decltype(tile_x)::value;
#pragma unroll
    for (int a = 0; a < MI; ++a)
      yf[ks][a] = lds_frag_xT<BM>(smem + J * C::Y_BYTES, ks * 16, wm * 128 + a * 32, lane);
#pragma unroll
    for (int b = 0; b < NI; ++b)
      xf[ks][b] = frag_x<BN>(smem + C::X_AT + X * C::X_BYTES, ks * 16, wn * 64 + b * 32, lane);
  };
  // Two of a step's 16 matrix instructions; nothing is moved across.
  auto multiply = [&](int ks, int a) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < NI; ++b)
      acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf[ks][b], yf[ks][a], acc[a][b], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  using std::false_type;
  using std::integral_constant;
  using std::true_type;
  // The waves 0-3 and 4-7 (a wave of each on every SIMD) run half a step apart.
  // Step k is a memory phase, in which a wave reads its fragments of the step
  // and its x bytes of step k + 2, which it turns into bf16 while the fragments
  // arrive, and a compute phase, in which it multiplies, issues the loads of dy
  // for step k + 3 and of x for step k + 4 and writes its bf16 x of step k + 2.
  // (Turning the int8 bytes in the compute phase instead cost 143 us against
  // 132 over 16384 tokens of 4096 x 1024; e4m3 bytes, 126 in both.)  A barrier closes each; the second group enters the
  // loop one barrier late and the first leaves it one late, so while one group
  // multiplies the other reads.  With phases numbered by barriers, the first
  // group reads step k in phase 2k and writes in 2k + 1, the second in 2k + 1 and
  // 2k + 2: x of step k + 2 is complete before phase 2k + 4 reads it, and its
  // tile, as the dy buffer of step k + 3, was last read in phases 2k - 3 and
  // 2k - 1.
  auto step = [&](auto n, auto end, int k) {
    constexpr int I = decltype(n)::value;
    constexpr bool END = decltype(end)::value;
    constexpr int SLOT = C::Q_AT + I % C::QS * C::QW_BYTES;
    integral_constant<int, (I + 1) % C::YS> buf_1;
    integral_constant<int, (I + 3) % C::YS> buf_3;
    integral_constant<int, (I + 2) % C::XS> tile_2;
    // dy of step k + 1 and x of step k + 2 are there: only what the last compute
    // phase issued may be in flight
    if (!END || k + 3 < steps)
      wait_vmcnt<C::Y_INSTR + 2>();
    else if (k + 2 < steps)
      wait_vmcnt<C::Y_INSTR>();
    else
      wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    const bool more_x = !END || k + 2 < steps, more_y = !END || k + 3 < steps,
               more_q = !END || k + 4 < steps;
    if (more_x) read_q(SLOT);
    frags(n, n, 0);
    frags(n, n, 1);
    if (more_x) unpack();
    if (END && k + 1 == steps - 1 && last < BK) zero_tail(buf_1);
    block_barrier();
    multiply(0, 0);
    if (more_y) issue_y(buf_3, end, 0, k + 3);
    multiply(0, 1);
    if (more_y) issue_y(buf_3, end, 1, k + 3);
    multiply(0, 2);
    if (more_q) issue_q(end, SLOT, k + 4);
    multiply(0, 3);
    if (more_q) issue_s(end, SLOT, k + 4);
    multiply(1, 0);
    multiply(1, 1);
    if (more_x) write_x(tile_2);
    multiply(1, 2);
    multiply(1, 3);
    block_barrier();
  };
  if (steps > 0) {
    static_assert(C::YS == 4 && C::XS == 4 && C::QS == 2, "the loop is unrolled by 4");
    integral_constant<int, 0> c0;
    integral_constant<int, 1> c1;
    integral_constant<int, 2> c2;
    integral_constant<int, 3> c3;
    true_type end;
    // the x bytes of steps 0 and 1 wait in the x tiles of steps 2 and 3
    constexpr int Q0 = C::X_AT + 2 * C::X_BYTES, Q1 = C::X_AT + 3 * C::X_BYTES;
    auto issue_x = [&](int at, int k) {
      issue_q(end, at, k);
      issue_s(end, at, k);
    };
    issue_x(Q0, 0);
    if (1 < steps) issue_x(Q1, 1);
    for (int i = 0; i < C::Y_INSTR; ++i) issue_y(c0, end, i, 0);
    if (1 < steps)
      for (int i = 0; i < C::Y_INSTR; ++i) issue_y(c1, end, i, 1);
    if (2 < steps) {
      issue_x(C::Q_AT, 2);
      for (int i = 0; i < C::Y_INSTR; ++i) issue_y(c2, end, i, 2);
    }
    if (3 < steps) issue_x(C::Q_AT + C::QW_BYTES, 3);
    // steps 0 and 1 of x, and step 0 of dy: all but the loads behind it
    if (3 < steps)
      wait_vmcnt<2 * C::Y_INSTR + 4>();
    else if (2 < steps)
      wait_vmcnt<2 * C::Y_INSTR + 2>();
    else if (1 < steps)
      wait_vmcnt<C::Y_INSTR>();
    else
      wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    read_q(Q0);
    unpack();
    write_x(c0);
    if (1 < steps) {
      read_q(Q1);
      unpack();
      write_x(c1);
    }
    if (steps == 1 && last < BK) zero_tail(c0);
    block_barrier();
    if (wave >= 4) block_barrier();
    int k = 0;
    for (; k + 8 < steps; k += 4) {   // every load of whole steps
      step(c0, false_type{}, k);
      step(c1, false_type{}, k + 1);
      step(c2, false_type{}, k + 2);
      step(c3, false_type{}, k + 3);
    }
    for (; k < steps; k += 4) {
      step(c0, end, k);
      if (k + 1 < steps) step(c1, end, k + 1);
      if (k + 2 < steps) step(c2, end, k + 2);
      if (k + 3 < steps) step(c3, end, k + 3);
    }
    if (wave < 4) block_barrier();
  }
  if (pc.parts == 1 && steps == 0 && p.accumulate) return;
  store_tile<MI>(p, pc, i0 + wm * 128, j0 + wn * 64, acc, smem + wave * kWindow, lane);
}

// dy as the wide tiles read it: rows padded with zeros to whole 16-byte vectors.
__global__ __launch_bounds__(kThreads) void repack_kernel(const uint16_t* dy, int64_t lddy,
                                                          int64_t tokens, int rows, uint16_t* out,
                                                          int64_t out_ld) {
  const uint32_t vecs = uint32_t(out_ld / 8);
  const int64_t total = tokens * vecs;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t t = i / vecs;
    const int col = int(i - t * vecs) * 8;
    *reinterpret_cast<u32x4_t*>(out + t * out_ld + col) = load_raw<true>(dy + t * lddy, col, rows);
  }
}

// Adds the partial sums of the matrices with several pieces, in their order:
// kJoin elements at a time, four per thread, the loads of eight pieces in
// flight.
constexpr int kJoin = 4 * kThreads;
__global__ __launch_bounds__(kThreads) void join_kernel(const WeightGrad p, int64_t blocks) {
  const int64_t size = int64_t(p.rows) * p.cols;
  const Split* splits = reinterpret_cast<const Split*>(static_cast<const Piece*>(p.table) + p.pieces);
  const int64_t work = p.offsets ? splits[p.count].e * blocks : blocks;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t which = i / blocks, at = (i - which * blocks) * kJoin + threadIdx.x * 4;
    const Split sp = p.offsets ? splits[which] : Split{0, int(p.pieces), 0};
    if (at >= size) continue;
    const int left = size - at < 4 ? int(size - at) : 4;
    const float* part = p.partial + sp.slot * size + at;
    float v[4] = {};
    if (left == 4) {
#pragma unroll 8
      for (int j = 0; j < sp.parts; ++j) {
        const u32x4_a4 w = *reinterpret_cast<const u32x4_a4*>(part + j * size);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += __uint_as_float(w[c]);
      }
    } else {
      for (int j = 0; j < sp.parts; ++j)
        for (int c = 0; c < 4; ++c) v[c] += c < left ? part[j * size + c] : 0.f;
    }
    const int64_t to = sp.e * size + at;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c >= left) break;
      if (p.g_bf16) {
        const uint16_t* g = static_cast<const uint16_t*>(p.G) + to + c;
        if (p.accumulate) v[c] += bf2f(*g);
      } else {
        if (p.accumulate) v[c] += static_cast<const float*>(p.G)[to + c];
      }
    }
    if (p.g_bf16) {
      uint16_t* g = static_cast<uint16_t*>(p.G) + to;
      typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
      if (left == 4)
        *reinterpret_cast<u32x2_a2*>(g) = u32x2_a2{f2bf2(v[0], v[1]), f2bf2(v[2], v[3])};
      else
        for (int c = 0; c < left; ++c) g[c] = f2bf(v[c]);
    } else {
      store_vec<false>(static_cast<float*>(p.G) + to, 0, left, v);
    }
  }
}

int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

// How a call is cut: its tiles, and the parts of the tokens.
struct Cut {
  double us;
  int64_t parts;
};
// The parts that take least, by estimates in microseconds fitted to one MI355X,
// `count` even matrices at once.  The tiles of 256 x 256 run one to a CU, those
// of 128 x 128 two; a round of them takes 11 (7) for its start and its stores
// and, per step of 32 tokens, 0.53 on few CUs to 0.76 on all, where the chip's
// power and its caches are shared (128 x 128: 0.34 where each has a CU to itself,
// 0.59 where some have not, a fifth more on rows whose vectors straddle cache
// lines; float32 0.87 and 1.6).  Partial sums cost 3 for the launch that joins
// them, 0.25 per part, a read that waits for memory, and 0.8 per 2^20 elements
// and part to write and read.
// Estimated against measured: 4096 x 1024 over 16384 tokens, 256 x 256, in 2
// parts 166 and 167, in 4 127 and 127, in 8 150 and 152; 128 x 128, in 1 part 181
// and 183, in 4 171 and 175; 256 x 256 over 16384, 128 x 128, in 1 part 182 and
// 180, in 16 25 and 23.
Cut cut_of(int64_t count, int64_t tokens, int64_t rows, int64_t cols, bool wide, bool bf16) {
  const int64_t tiles = wide ? cdiv(rows, Wide::BM) * cdiv(cols, Wide::BN) : cdiv(rows, BM) * cdiv(cols, BN);
  const int64_t at_once = wide ? 256 : 512;
  const double g = double(count) * double(rows) * double(cols);
  auto step = [&](int64_t blocks) {
    const double u = double(blocks) / 256;
    if (wide) return 0.53 + 0.23 * u * u * u;
    if (!bf16) return u > 1 ? 1.6 : 0.87;
    return (u > 1 ? 0.59 : 0.34) * (rows % 8 == 0 ? 1 : 1.2);
  };
  Cut best{0, 0};
  for (int64_t n = 1; n <= 64 && n <= cdiv(tokens, 4 * BK); ++n) {
    const int64_t blocks = count * tiles * n, rounds = blocks / at_once, rest = blocks % at_once;
    const double start = wide ? 11 : 7, steps = double(cdiv(cdiv(tokens, n), BK));
    double us = double(rounds) * (start + step(at_once) * steps);
    if (rest > 0) us += start + step(rest) * steps;
    if (n > 1) us += 3 + 0.25 * double(n) + g * double(n) * 0.8e-6;
    if (n == 1 || us < best.us) best = {us, n};
  }
  if (best.parts == 0) best.parts = 1;   // no tokens
  return best;
}

}  // namespace

// Ragged matrices are taken as even for the cut; the uneven ones get pieces
// of at most that length or, where it is more, of an even share of the whole
// call per CU (64 experts of 1408 x 512 over 49152 tokens, a spread of 3:1: an
// eighth slower in pieces of 1024 than of 2048 to 4096, 3 % of 8192).
WeightGradPlan weight_grad_plan(int64_t count, int64_t tokens, int64_t rows, int64_t cols,
                                bool ragged, bool bf16) {
  constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;
  WeightGradPlan w{};
  const int64_t even = cdiv(tokens, count);
  Cut cut = cut_of(count, even, rows, cols, false, bf16);
  // The 256 x 256 tiles are ahead where they fill the chip for many steps
  // (1024 x 1024: 12.6 against 21.8 us over 700 tokens; 4096 x 1024: 51 against 53
  // over 4096, 168 against 127 over 16384).  They read rows of whole 16-byte
  // vectors of bf16; others are repacked first, at 5 TB/s (4095 x 1024 over
  // 16384: 178 us, 211 with the small tiles).  float32 is bound by its three
  // products on either, and turned into them in the small tiles.
  if (bf16) {
    const Cut c = cut_of(count, even, rows, cols, true, bf16);
    const bool repack = rows % 8 != 0;
    w.wide = c.us + (repack ? 3 + double(tokens) * double(rows) * 4 / 5e6 : 0) < cut.us;
    if (w.wide) {
      cut = c;
      if (repack) w.repack_bytes = size_t(tokens) * size_t(cdiv(rows, 8) * 8) * 2;
    }
  }
  int64_t chunk = cdiv(even, cut.parts);
  if (ragged) {
    const int64_t tiles = w.wide ? cdiv(rows, Wide::BM) * cdiv(cols, Wide::BN) : cdiv(rows, BM) * cdiv(cols, BN);
    chunk = std::max(chunk, tokens / (w.wide ? 256 : 512) * tiles);
  }
  chunk = std::max<int64_t>(4 * BK, cdiv(std::min(chunk, MUON_MAX_TOKENS), BK) * BK);
  w.chunk = uint32_t(chunk);
  if (!ragged) {
    w.pieces = std::max<int64_t>(1, cdiv(tokens, chunk));
    w.slots = w.pieces > 1 ? w.pieces : 0;
  } else {
    // a matrix of n > 1 pieces has more than (n - 1) chunk tokens
    w.pieces = tokens / chunk + count;
    w.slots = tokens > chunk ? std::min(2 * (tokens / chunk) + 1, w.pieces) : 0;
    w.table_bytes = w.pieces * kWeightGradPieceBytes + (count + 1) * kWeightGradSplitBytes;
  }
  // the largest grid: the smallest tiles, and whole turns of the 8 XCDs
  if ((w.pieces + 64) * (cdiv(rows, BM) * cdiv(cols, BN)) > kMaxBlocks) {
    w.pieces = 0;
    return w;
  }
  w.partial_bytes = size_t(w.slots) * size_t(rows) * size_t(cols) * 4;
  return w;
}

template <bool BF16>
hipError_t launch_small(const WeightGrad& p, dim3 grid, int tm, int tn, hipStream_t s) {
  if (p.x.fmt == MUON_CKPT_E4M3)
    hipLaunchKernelGGL((weight_grad_kernel<BF16, MUON_CKPT_E4M3>), grid, dim3(kThreads), 0, s, p, tm, tn);
  else
    hipLaunchKernelGGL((weight_grad_kernel<BF16, MUON_CKPT_INT8>), grid, dim3(kThreads), 0, s, p, tm, tn);
  return hipGetLastError();
}
hipError_t launch_wide(const WeightGrad& p, dim3 grid, int tm, int tn, hipStream_t s) {
  if (p.x.fmt == MUON_CKPT_E4M3)
    hipLaunchKernelGGL(weight_grad_wide_kernel<MUON_CKPT_E4M3>, grid, dim3(64 * Wide::NW), 0, s, p, tm, tn);
  else
    hipLaunchKernelGGL(weight_grad_wide_kernel<MUON_CKPT_INT8>, grid, dim3(64 * Wide::NW), 0, s, p, tm, tn);
  return hipGetLastError();
}

hipError_t launch_weight_grad(const WeightGrad& call, const WeightGradPlan& plan, bool bf16,
                              hipStream_t s) {
  WeightGrad p = call;
  // a multiple of 8 blocks; with offsets, whole turns of `deal` tiles per XCD
  auto grid = [&](int tm, int tn) {
    const int64_t tiles = int64_t(tm) * tn, deal = p.offsets ? std::min<int64_t>(tiles, 32) : 1;
    return dim3(unsigned(cdiv(plan.pieces * tiles, 8 * deal) * 8 * deal));
  };
  if (p.offsets) {
    if (p.count <= 64)
      hipLaunchKernelGGL(plan_kernel<64>, dim3(1), dim3(64), 0, s, p);
    else
      hipLaunchKernelGGL(plan_kernel<kPlanThreads>, dim3(1), dim3(kPlanThreads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool rows16 = p.lddy % 8 == 0 && reinterpret_cast<uintptr_t>(p.dy) % 16 == 0;
  if (plan.wide && (plan.repack_bytes > 0 || rows16)) {
    p.y = static_cast<const uint16_t*>(p.dy);
    p.y_ld = p.lddy;
    p.y_cols = p.rows;
    if (plan.repack_bytes > 0) {
      p.y = p.repack;
      p.y_ld = p.y_cols = int(cdiv(p.rows, 8) * 8);
      const int64_t blocks = cdiv(p.tokens * (p.y_ld / 8), kThreads);
      hipLaunchKernelGGL(repack_kernel, dim3(unsigned(std::min<int64_t>(blocks, 16384))), dim3(kThreads), 0,
                         s, static_cast<const uint16_t*>(p.dy), p.lddy, p.tokens, p.rows, p.repack, p.y_ld);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const int tm = int(cdiv(p.rows, Wide::BM)), tn = int(cdiv(p.cols, Wide::BN));
    return launch_wide(p, grid(tm, tn), tm, tn, s);
  }
  const int tm = int(cdiv(p.rows, BM)), tn = int(cdiv(p.cols, BN));
  return bf16 ? launch_small<true>(p, grid(tm, tn), tm, tn, s) : launch_small<false>(p, grid(tm, tn), tm, tn, s);
}

hipError_t launch_weight_grad_join(const WeightGrad& p, const WeightGradPlan& plan, hipStream_t s) {
  const int64_t blocks = cdiv(int64_t(p.rows) * p.cols, kJoin);
  const int64_t most = p.offsets ? std::max<int64_t>(1, plan.slots / 2) : 1;   // split matrices
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(std::min<int64_t>(most * blocks, 4096))), dim3(kThreads), 0,
                     s, p, blocks);
  return hipGetLastError();
}

}  // namespace muon
