// The linear products where there is work for the whole chip: blocks that stay,
// each computing tile after tile in one unbroken stream of steps, so that the
// loads of the next tile's first steps are under way while the last steps of
// this one are multiplied and its outputs are stored.
//
// Tiles of 256 x 256, one block of 4 waves of 128 x 128 per CU (a wave on each
// SIMD, with half of its registers as accumulators: the fewest reads of LDS, and
// of the L2, per product), or of 128 x 128, two blocks of 4 waves of 64 x 64, one
// of which multiplies while the other stores.  A step is 128 bytes of k (64 bf16
// or 128 e4m3), multiplied in units of one chunk (two of e4m3) per lane.  While a
// wave multiplies one unit, it reads the next, between the matrix instructions;
// the last unit of a step reads the first one of the next step:
//
//   read units 1 .. of step s          multiply 0 .. of step s
//   step s + 1 has come: barrier       (all have read step s: its place is free)
//   read unit 0 of step s + 1, issue   multiply the last unit
//   the loads of step s + 2
//
// Outputs are stored in whole lines of 128 bytes past the L2 (16384 tokens of 4096 x
// 1024, e4m3, k = 1024: 86 us with 32 bytes of a row at a time, 78 so; 49152 of 64 x
// 1408 x 512, bf16: 118, 105).
//
// Measured on one MI355X: e4m3, 256 x 256, 16384 tokens of 4096 x 1024 across
// (k = 4096) 64 us, 2150 TFLOP/s; of 8 x 5632 x 2048, uneven, 191 (1980); k = 1024 78
// (1760), of which 30 are stores: loads behind them wait for them, so that they do
// not overlap with the next tile.  bf16, 16384 tokens of 4096 x 1024 131 (1050;
// PyTorch's library product of these widths reaches 900 to 1050).  128 x 128: 49152
// tokens of 64 x 1408 x 512, uneven, 105 us in a row, of which the instructions alone
// take 58 and the loads 75 (every step waits for the L2, one step ahead being all
// that LDS holds).
#include <algorithm>
#include <type_traits>

#include "lds_tiles.h"
#include "linear_device.h"

namespace muon {
namespace {

// 1 byte per lane straight to LDS, zero-extended to a word each.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma1(uint32_t off, const char* base, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// The places of a block's tiles, kTable at a time in a ring, refilled by halves.
constexpr int kTable = 96;

template <LinearType TYPE, bool ACROSS, int BM, int BN, int PER_CU>
__global__ __launch_bounds__(256, PER_CU) void linear_stream_kernel(const Linear p, int tiles_n) {
  constexpr int NW = 4, THREADS = 64 * NW, WN = 2, NT = BN / WN / 32, MT = BM / 64;
  constexpr bool E4M3 = TYPE == LIN_E4M3;
  static_assert(E4M3 || TYPE == LIN_BF16, "types of this kernel");
  static_assert(!(E4M3 && ACROSS), "8-bit weights are kept both ways");
  constexpr int ES = E4M3 ? 1 : 2, BK = ROWB / ES;
  constexpr int STAGES = 2;
  constexpr int X_BYTES = BM * ROWB, W_BYTES = BN * ROWB;
  // scales: words of x, 64 per wave, then of w: loaded by the waves that x leaves,
  // or by all
  constexpr int XSW = BM / 64;
  constexpr bool SHARE = NW > XSW;
  constexpr int S_BYTES = E4M3 ? (SHARE ? NW : 2 * NW) * 256 : 0;
  constexpr int STAGE = X_BYTES + W_BYTES + S_BYTES;
  constexpr int XI = X_BYTES / WAVE_BYTES / NW, WI = W_BYTES / WAVE_BYTES / NW;
  constexpr int LOADS = XI + WI + (!E4M3 ? 0 : SHARE ? 1 : 2);   // per wave and step
  constexpr int UNITS = E4M3 ? 2 : 4, CHUNKS = 4 / UNITS;
  constexpr int TABLE_AT = STAGES * STAGE, BOUNDS_AT = TABLE_AT + kTable * 16;
  __shared__ __attribute__((aligned(1024))) char smem_raw[BOUNDS_AT + kBoundsWords * 4];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;
  const uint32_t smem_base = uint32_t(reinterpret_cast<uintptr_t>(smem));
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;

  Bounds bounds{};
  bounds.tiles = cdiv_d(int(p.tokens), BM);
  if (p.offsets) {
    bounds = find_bounds<THREADS, false>(p, BM, (LDS_AS int*)(smem + BOUNDS_AT));
    // the outputs of tokens of no matrix
    const int before = bounds.ends[0], behind = bounds.ends[p.count];
    const int none = before + int(p.tokens) - behind;
    for (int i = blockIdx.x; i < none; i += gridDim.x) {
      const int64_t row = i < before ? i : behind + i - before;
      const u32x4_t zero = {0, 0, 0, 0};
      for (int c = t * 8; c < p.n; c += THREADS * 8)
        store_raw<true>(static_cast<uint16_t*>(p.y) + row * p.n, c, p.n, zero);
    }
  }
  // This block's tiles: XCD x takes a contiguous eighth of all, its blocks by
  // turns, so that its compute units work on neighbouring tiles.
  const int total = bounds.tiles * tiles_n, per = (total + 7) / 8, stride = int(gridDim.x) / 8;
  const int first_id = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
  const int end_id = min(int(blockIdx.x & 7) * per + per, total);
  if (first_id >= end_id) return;
  const int steps = p.k / BK;                              // of a tile

  // Each thread finds the place of one tile: first token, end of its matrix's
  // tokens, first output, matrix.  (The search and the divisions by a whole wave
  // at each tile's beginning and end took a fifth of the time of short tiles.)
  typedef int i32x4_t __attribute__((ext_vector_type(4)));
  LDS_AS i32x4_t* table = (LDS_AS i32x4_t*)(smem + TABLE_AT);
  const int tiles = (end_id - first_id + stride - 1) / stride;
  auto fill_table = [&](int from, int count) __attribute__((always_inline)) {
    const int i = from + t;
    if (t < count && i < tiles) {
      const int id = first_id + i * stride;
      int e = 0, begin = 0, end = int(p.tokens), first = 0, next = bounds.tiles;
      if (p.offsets) {
        // the last segment whose first tile is not behind this one
        const int row = id / tiles_n;
        int lo = 0, hi = p.count + 2;
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (bounds.firsts[mid] <= row)
            lo = mid;
          else
            hi = mid;
        }
        e = lo - 1;
        begin = bounds.ends[lo - 1];
        end = bounds.ends[lo];
        first = bounds.firsts[lo];
        next = bounds.firsts[lo + 1];
      }
      int tm, tn;
      place_tile(id - first * tiles_n, next - first, tiles_n, tm, tn);
      table[i % kTable] = i32x4_t{begin + tm * BM, end, tn * BN, e};
    }
    block_barrier();
  };
  fill_table(0, kTable);
  struct Tile {
    int t0, end, n0, e;
  };
  auto tile_at = [&](int i) __attribute__((always_inline)) {
    const i32x4_t v = table[i % kTable];
    return Tile{__builtin_amdgcn_readfirstlane(v[0]), __builtin_amdgcn_readfirstlane(v[1]),
                __builtin_amdgcn_readfirstlane(v[2]), __builtin_amdgcn_readfirstlane(v[3])};
  };

  // What only a tile's beginning or end needs is computed there, from a lane
  // number that the compiler cannot follow: hoisted out of the loop, it would
  // take the registers that the accumulators leave.
  auto fresh = [](int v) __attribute__((always_inline)) {
    asm volatile("" : "+v"(v));
    return v;
  };

  // ---- loads: the tile that they have reached
  constexpr int WPR = BN * ES / 16;              // chunks per k row of a w across
  uint32_t x_off[XI], w_off[WI], xs_off = 0, ws_off = 0;
  const char *x = nullptr, *w = nullptr, *xs = nullptr, *ws = nullptr;
  int load_tile_number = 0, load_k = 0, load_buf = 0;
  auto load_tile = [&]() __attribute__((always_inline)) {
    const Tile at = tile_at(load_tile_number);
    const int t0 = at.t0, n0 = at.n0;
    const int rows_x = min(at.end - t0, BM), rows_w = min(p.n - n0, BN);
    const int ln = fresh(lane);
    x = static_cast<const char*>(p.x) + int64_t(t0) * p.ldx;
    w = static_cast<const char*>(p.W) + at.e * p.w_stride + (ACROSS ? int64_t(n0) * ES : int64_t(n0) * p.ldw);
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int to = (wave * XI + i) * 64 + ln, r = to / 8;
      x_off[i] = uint32_t(min(r, rows_x - 1)) * uint32_t(p.ldx) + ((to % 8) ^ swz(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < WI; ++i) {
      const int to = (wave * WI + i) * 64 + ln;
      if constexpr (ACROSS) {
        const int k = to / WPR, c = (to % WPR) ^ gswz(k);
        w_off[i] = uint32_t(k) * uint32_t(p.ldw) + min(c * 16, rows_w * ES - 16);
      } else {
        const int r = to / 8;
        w_off[i] = uint32_t(min(r, rows_w - 1)) * uint32_t(p.ldw) + ((to % 8) ^ swz(r)) * 16;
      }
    }
    if constexpr (E4M3) {
      // a word of scales per token; the bytes of the tile's two blocks of outputs
      xs = reinterpret_cast<const char*>(p.x_scale) + int64_t(t0) * p.xs_pitch;
      xs_off = uint32_t(min((wave * 64 + ln) % BM, rows_x - 1)) * uint32_t(p.xs_pitch);
      ws = reinterpret_cast<const char*>(p.w_scale) + at.e * p.ws_stride + int64_t(n0 / SIDE) * p.ws_row;
      ws_off = (ln & 1) * SIDE < rows_w ? uint32_t(ln & 1) * uint32_t(p.ws_row) : 0;
    }
  };
  auto issue_one = [&](int i) __attribute__((always_inline)) {
    const uint32_t base = smem_base + load_buf * STAGE;
    if (i < XI)
      dma16(x_off[i], x, base + (wave * XI + i) * WAVE_BYTES);
    else
      dma16(w_off[i - XI], w, base + X_BYTES + (wave * WI + i - XI) * WAVE_BYTES);
  };
  auto issue_scales = [&]() __attribute__((always_inline)) {
    const uint32_t base = smem_base + load_buf * STAGE + X_BYTES + W_BYTES + wave * 256;
    if (!SHARE || wave < XSW) dma4(xs_off, xs, base);
    if (!SHARE || wave >= XSW) dma1(ws_off, ws, base + (SHARE ? 0 : NW * 256));
  };
  // The next step's loads; behind the last one of the block's tiles that one
  // again, which nothing reads.
  const int64_t w_step = ACROSS ? BK * p.ldw : ROWB;
  auto issue_end = [&]() __attribute__((always_inline)) {
    load_buf ^= 1;
    if (load_k + 1 < steps) {
      ++load_k;
      x += ROWB;
      w += w_step;
      if constexpr (E4M3) {
        xs += 4;
        ws += p.ws_col;
      }
    } else if (load_tile_number + 1 < tiles) {
      ++load_tile_number;
      load_k = 0;
      if (load_tile_number >= kTable && load_tile_number % (kTable / 2) == 0)
        fill_table(load_tile_number, kTable / 2);
      load_tile();
    }
  };

  // ---- fragments
  struct Unit {
    u32x4_t x[MT][CHUNKS], w[NT][CHUNKS];
  };
  constexpr int READS = (MT + NT) * CHUNKS, PRODUCTS = MT * NT;   // of a unit
  int frag_at[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    frag_at[c] = (lane & 31) * ROWB + (((2 * c + (lane >> 5)) ^ swz(lane & 31)) << 4);
  // Read number i of a unit: those that the first products need come first.
  auto read_one = [&](Unit& f, int buf, int unit, int i) __attribute__((always_inline)) {
    const LDS_AS char* s = smem + buf * STAGE;
    const int c = i % CHUNKS, j = i / CHUNKS;
    const int at = frag_at[unit * CHUNKS + c];
    if (j == 0 || j > NT) {
      const int a = j == 0 ? 0 : j - NT;
      f.x[a][c] = *reinterpret_cast<const LDS_AS u32x4_t*>(s + (wm * MT + a) * 32 * ROWB + at);
    } else {
      const int b = j - 1;
      if constexpr (ACROSS)
        f.w[b][c] = __builtin_bit_cast(u32x4_t, frag_across<BN>(s + X_BYTES, 16 * unit, (wn * NT + b) * 32, lane));
      else
        f.w[b][c] = *reinterpret_cast<const LDS_AS u32x4_t*>(s + X_BYTES + (wn * NT + b) * 32 * ROWB + at);
    }
  };
  uint32_t sx[MT] = {}, sw = 0, sx_next[MT] = {}, sw_next = 0;   // scales of a step
  auto read_scales = [&](int buf) __attribute__((always_inline)) {
    const LDS_AS char* q = smem + buf * STAGE + X_BYTES + W_BYTES;
#pragma unroll
    for (int a = 0; a < MT; ++a)
      sx_next[a] = *reinterpret_cast<const LDS_AS uint32_t*>(q + ((wm * MT + a) * 32 + (lane & 31)) * 4);
    sw_next = *reinterpret_cast<const LDS_AS uint32_t*>(q + (SHARE ? XSW : NW + wave) * 256 + wn * NT * 32 / SIDE * 4);
  };
  f32x16_t acc[MT][NT];
  // Keeps the products before it there, and the sums in the accumulation
  // registers (no instruction).
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < NT; ++b) asm volatile("" : "+a"(acc[a][b]));
  };
  // Zeros by products of zeros: an instruction for 16 registers.
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        u32x4_t zero = {0, 0, 0, 0};
        asm volatile("" : "+v"(zero));       // one product is not copied to all
        const bf16x8_t z = __builtin_bit_cast(bf16x8_t, zero);
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(z, z, f32x16_t{}, 0, 0, 0);
      }
    pin();
  };
  // FIRST: of a tile, whose sums begin with it.
  auto product = [&](const Unit& f, auto unit, auto first, int i) __attribute__((always_inline)) {
    const int a = i / NT, b = i % NT;
    constexpr bool FIRST = decltype(first)::value;
    const f32x16_t sum = FIRST ? f32x16_t{} : acc[a][b];
    if constexpr (E4M3) {
      auto both = [](const u32x4_t& lo, const u32x4_t& hi) {
        return i32x8_t{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                       int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
      };
      acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          both(f.w[b][0], f.w[b][1]), both(f.x[a][0], f.x[a][1]), sum, 0, 0, 0, int(sw),
          2 * decltype(unit)::value, int(sx[a]));
    } else {
      acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f.w[b][0]),
                                                          __builtin_bit_cast(bf16x8_t, f.x[a][0]),
                                                          sum, 0, 0, 0);
    }
  };
  // The products of unit f, and between them the reads of `g` and the loads.
  auto run_unit = [&](const Unit& f, auto unit, Unit& g, int buf, int next_unit, auto loads, auto first)
      __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PRODUCTS; ++i) {
      product(f, unit, first, i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = i * READS / PRODUCTS; j < (i + 1) * READS / PRODUCTS; ++j) read_one(g, buf, next_unit, j);
      if constexpr (decltype(loads)::value) {
#pragma unroll
        for (int j = i * (XI + WI) / PRODUCTS; j < (i + 1) * (XI + WI) / PRODUCTS; ++j) issue_one(j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
  };

  // ---- a tile's outputs, from the registers, in whole lines of 128 bytes.  Lane
  // l, register 4 g + i of a 32 x 32 block holds token l % 32, output 8 g + 4 (l /
  // 32) + i.  The halves of the wave exchange parts of two blocks, so that a lane
  // has all 32 outputs of a token in one of them, four chunks of 16 bytes; then
  // four neighbouring lanes exchange chunks, so that they hold the four of one
  // token, and of the next one, .., which they store side by side.  Returns whether
  // every lane took part in all the stores, which then count as loads in flight do.
  constexpr int STORES = MT * NT * 2;
  auto store = [&](int number) __attribute__((always_inline)) {
    const Tile at = tile_at(number);
    const int t0 = at.t0 + wm * MT * 32, n0 = at.n0 + wn * NT * 32;
    const bool whole = at.t0 + BM <= at.end && at.n0 + BN <= p.n;
    const int ln = fresh(lane), row = ln & 28, col = 32 * (ln >> 5) + 8 * (ln & 3);
    const int rows = at.end - t0 - row, cols = p.n - n0 - col;   // that are left
    char* y = static_cast<char*>(p.y) + (int64_t(t0 + row) * p.n + n0 + col) * 2;
    const int64_t pitch = int64_t(p.n) * 2;
    const bool lines = whole_lines(p);
    const bool odd1 = ln & 1, odd2 = ln & 2;
    // chunk `lo` of the lanes with the bit and `hi` of those without change places
    auto exchange = [](u32x4_t& lo, u32x4_t& hi, bool bit, auto perm) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t out = bit ? lo[i] : hi[i];
        const uint32_t in = __builtin_amdgcn_mov_dpp(out, decltype(perm)::value, 0xf, 0xf, true);
        lo[i] = bit ? in : lo[i];
        hi[i] = bit ? hi[i] : in;
      }
    };
    const std::integral_constant<int, 0xb1> next1;   // lanes 1 0 3 2
    const std::integral_constant<int, 0x4e> next2;   // lanes 2 3 0 1
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < NT; b += 2) {
        u32x4_t c[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const auto r = __builtin_amdgcn_permlane32_swap(
                f2bf2(acc[a][b][4 * g + 2 * i], acc[a][b][4 * g + 2 * i + 1]),
                f2bf2(acc[a][b + 1][4 * g + 2 * i], acc[a][b + 1][4 * g + 2 * i + 1]), false, false);
            c[g][i] = r[0];
            c[g][2 + i] = r[1];
          }
        exchange(c[0], c[1], odd1, next1);
        exchange(c[2], c[3], odd1, next1);
        exchange(c[0], c[2], odd2, next2);
        exchange(c[1], c[3], odd2, next2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (whole || (a * 32 + i < rows && b * 32 < cols)) {
            const RowVec<true>::Raw v = {c[i][0], c[i][1], c[i][2], c[i][3]};
            auto to = reinterpret_cast<RowVec<true>::Raw*>(y + (a * 32 + i) * pitch + b * 64);
            if (lines)
              __builtin_nontemporal_store(v, to);
            else
              *to = v;
          }
      }
    return whole;
  };

  load_tile();
  for (int i = 0; i < STAGES; ++i) {
#pragma unroll
    for (int j = 0; j < XI + WI; ++j) issue_one(j);
    if constexpr (E4M3) issue_scales();
    issue_end();
  }
  wait_vmcnt<(STAGES - 1) * LOADS>();
  asm volatile("" ::: "memory");
  block_barrier();
  Unit f0, f1;
#pragma unroll
  for (int i = 0; i < READS; ++i) read_one(f0, 0, 0, i);
  if constexpr (E4M3) read_scales(0);
  int buf = 0;
  bool stored = false;       // whether a tile's stores ended the step before
  std::integral_constant<int, 0> u0;
  std::integral_constant<int, 1> u1;
  std::integral_constant<int, 2> u2;
  std::integral_constant<int, 3> u3;
  std::false_type only_reads;
  std::true_type with_loads;
  // A tile's first products begin its sums; with 256 accumulation registers, all
  // there are, another copy of that unit would spill, so they are set to zero.
  constexpr bool FIRST = MT * NT < 16;
  for (int number = 0; number < tiles; ++number) {
    if constexpr (!FIRST) clear();
    for (int k = 0; k < steps; ++k) {
      const int next = buf ^ 1;
      if constexpr (E4M3) {
#pragma unroll
        for (int a = 0; a < MT; ++a) sx[a] = sx_next[a] >> (8 * (lane >> 5));
        sw = sw_next;
      }
      if (FIRST && k == 0)
        run_unit(f0, u0, f1, buf, 1, only_reads, std::integral_constant<bool, FIRST>{});
      else
        run_unit(f0, u0, f1, buf, 1, only_reads, std::false_type{});
      if constexpr (UNITS == 4) {
        run_unit(f1, u1, f0, buf, 2, only_reads, std::false_type{});
        run_unit(f0, u2, f1, buf, 3, only_reads, std::false_type{});
      }
      // the next step has come: behind it, the stores of a tile that ended since may
      // be on their way
      if (stored)
        wait_vmcnt<STORES>();
      else
        wait_vmcnt<0>();
      stored = false;
      asm volatile("" ::: "memory");
      block_barrier();
      if constexpr (E4M3) {
        read_scales(next);
        issue_scales();
      }
      if constexpr (UNITS == 4)
        run_unit(f1, u3, f0, next, 0, with_loads, std::false_type{});
      else
        run_unit(f1, u1, f0, next, 0, with_loads, std::false_type{});
      issue_end();
      buf = next;
    }
    stored = store(number);
  }
  wait_vmcnt<0>();      // loads to LDS that nothing waited for
}

template <LinearType TYPE, bool ACROSS, int SIDE_, int PER_CU>
hipError_t launch_stream(const Linear& p, hipStream_t s) {
  const int64_t tiles_n = (p.n + SIDE_ - 1) / SIDE_;
  const int64_t tiles = (p.offsets ? p.tokens / SIDE_ + p.count : (p.tokens + SIDE_ - 1) / SIDE_) * tiles_n;
  const dim3 grid(unsigned(std::min<int64_t>(256 * PER_CU, (tiles + 8) / 8 * 8)));
  hipLaunchKernelGGL((linear_stream_kernel<TYPE, ACROSS, SIDE_, SIDE_, PER_CU>), grid, dim3(256), 0, s, p, int(tiles_n));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_stream(const Linear& p, LinearType type, bool across, int side, hipStream_t s) {
  if (side == 256)
    return type == LIN_E4M3 ? launch_stream<LIN_E4M3, false, 256, 1>(p, s)
           : across         ? launch_stream<LIN_BF16, true, 256, 1>(p, s)
                            : launch_stream<LIN_BF16, false, 256, 1>(p, s);
  return type == LIN_E4M3 ? launch_stream<LIN_E4M3, false, 128, 2>(p, s)
                          : launch_stream<LIN_BF16, false, 128, 2>(p, s);
}

}  // namespace muon
