// Device helpers of the kernels of the linear products.
#pragma once

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

// Chunk swizzle of a tile of bf16 rows of k with BN outputs each (a weight that
// is read across its rows), and its fragment: lane l gets output nb + l % 32, k
// kb + 8 (l / 32) .. + 7.  The 4 rows x 64 bytes that 32 lanes of a transposing
// read take cover the 64 banks once: rows of 128 bytes share banks with every
// other one, longer ones with all.
template <int BN>
__device__ __forceinline__ int swz_across(int k) { return BN == 64 ? (k & 2) << 1 : gswz(k); }
template <int BN>
__device__ __forceinline__ bf16x8_t frag_across(const LDS_AS char* tile, int kb, int nb, int lane) {
  const int s = lane & 15;
  const int n = nb + 16 * ((lane >> 4) & 1) + 4 * (s & 3);
  const int k = kb + 8 * (lane >> 5) + (s >> 2);
  const LDS_AS char* p0 = tile + k * (BN * 2) + (((n >> 3) ^ swz_across<BN>(k)) << 4) + (n & 7) * 2;
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)p0);
  const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(p0 + 4 * BN * 2));
  const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// 16 e4m3 numbers as bf16, exact: the conversion multiplies by 2^e (255, a
// marked block, by NaN).
__device__ __forceinline__ void widen(u32x4_t q, uint32_t byte, bf16x8_t (&o)[2]) {
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
}

// Whether the outputs' rows begin with lines of 128 bytes: a wave's stores then fill
// whole lines and go past the L2, parts of lines through it (16384 tokens of 4104 x
// 2048, bf16: past it 290 us, through it 276).
__device__ __forceinline__ bool whole_lines(const Linear& p) {
  return p.n % (p.y_bf16 ? 64 : 32) == 0 && reinterpret_cast<uintptr_t>(p.y) % 128 == 0;
}

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
// turn; XCD x takes a contiguous eighth.  -1: none.
__device__ __forceinline__ int64_t xcd_order(uint32_t b, uint32_t total) {
  const uint32_t per = (total + 7) / 8, turn = b >> 3, id = (b & 7) * per + turn;
  return turn < per && id < total ? int64_t(id) : -1;
}

// The segments of a call with offsets, in LDS: segment 0 lies before the first
// offset, segment s holds matrix s - 1, the last one the tokens behind the last
// offset.  Offsets are clamped to [0, tokens] and read as the largest so far, so
// that no place leaves the buffers.
struct Bounds {
  LDS_AS int *ends, *firsts;   // of each segment: its end, the first of its tiles of `bm` tokens
  int tiles;                   // of all segments, along the tokens
};
constexpr int kBoundsWords = 2 * kLinearMaxSegs + 32;

// Every block of threads finds the bounds itself (a launch for them alone would
// take longer).  NONE: the tokens of no matrix have tiles too.
template <int THREADS, bool NONE>
__device__ __forceinline__ Bounds find_bounds(const Linear& p, int bm, LDS_AS int* lds) {
  constexpr int WAVES = THREADS / 64;
  const int t = threadIdx.x, T = int(p.tokens);
  const int lane = t & 63, wave = t >> 6, segs = p.count + 2;
  LDS_AS int *ends = lds, *firsts = lds + kLinearMaxSegs, *wave_top = firsts + kLinearMaxSegs,
             *wave_sum = wave_top + 16;
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
    const bool counts = s < segs && (NONE || (s > 0 && s <= p.count));
    const int n = counts ? cdiv_d(hi - lo, bm) : 0;
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
  return Bounds{ends, firsts, tiles};
}

// The place of tile `id` of a call (a whole wave takes part).
__device__ __forceinline__ Place place_of(const Linear& p, const Bounds& b, int bm, int tiles_n, int id) {
  Place out;
  if (!p.offsets) {
    out.e = out.begin = 0;
    out.end = int(p.tokens);
    place_tile(id, cdiv_d(out.end, bm), tiles_n, out.tm, out.tn);
    return out;
  }
  // the last segment whose first tile is not behind this one
  const int lane = threadIdx.x & 63, segs = p.count + 2, row = id / tiles_n;
  int s = -1;
  for (int base = 0; base < segs; base += 64) {
    const uint64_t m = __ballot(base + lane < segs && b.firsts[base + lane < segs ? base + lane : 0] <= row);
    s += __builtin_popcountll(m);
    if (m != ~uint64_t(0)) break;
  }
  const int first = __builtin_amdgcn_readfirstlane(b.firsts[s]);
  const int next = __builtin_amdgcn_readfirstlane(s + 1 < segs ? b.firsts[s + 1] : b.tiles);
  out.e = s > p.count ? -1 : s - 1;
  out.begin = __builtin_amdgcn_readfirstlane(s > 0 ? b.ends[s - 1] : 0);
  out.end = __builtin_amdgcn_readfirstlane(b.ends[s]);
  place_tile(id - first * tiles_n, next - first, tiles_n, out.tm, out.tn);
  return out;
}

}  // namespace
}  // namespace muon
