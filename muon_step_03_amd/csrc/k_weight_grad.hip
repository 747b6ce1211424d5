// Weight gradients from 8-bit activation checkpoints:
//
//   G[e] (+)= sum_t dy[t]^T x[t]     (rows x cols, t over the tokens of e)
//
// The contraction runs over tokens, the slow axis of both operands, so both
// are staged as token rows in LDS and read as MFMA fragments with transposing
// LDS reads.  x is brought back from 8 bits when it is written to LDS: a
// checkpoint's values are exact in bf16, so bf16 matrix cores see exactly what
// it holds.  float32 dy is split into three bf16 parts of 8 bits each
// (truncation, remainders exact), whose three products per element replace
// the sixteen times slower float32 matrix instruction.
//
// The tokens of a matrix are cut into pieces of at most `chunk`; every block
// computes one tile over one piece.  A matrix of one piece is written at once,
// one of several leaves float32 tiles that the join kernel adds in order: no
// atomics, the same bits on every run.
#include <algorithm>

#include "lds_tiles.h"
#include "layer_internal.h"

namespace muon {
namespace {

constexpr int BM = 128, BN = 128, BK = 32;   // rows of G, columns of G, tokens
constexpr int NT = 256;                      // 2 x 2 waves of 64 x 64
constexpr int kTile = BM * BN;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct Piece {
  int e;             // matrix
  int begin, end;    // tokens
  int parts;         // pieces of its matrix
  int64_t slot;      // its place among the partial sums (parts > 1)
};

// Piece number `want`, or the matrix number `want` when BY_MATRIX (begin and
// end are then those of its first piece).  False past the last.  Every wave
// scans the offsets 64 at a time; begin offsets are read as the largest
// offset so far, clamped to [0, tokens], so that no piece leaves the buffers
// and their number is bounded whatever the offsets hold.
template <bool BY_MATRIX>
__device__ __forceinline__ bool find_piece(const WeightGrad& p, int64_t want, Piece& out) {
  const int64_t C = p.chunk;
  if (!p.offsets) {
    const int64_t parts = p.tokens > C ? (p.tokens + C - 1) / C : 1;
    if (want >= (BY_MATRIX ? 1 : parts)) return false;
    out.e = 0;
    out.begin = int(BY_MATRIX ? 0 : want * C);
    out.end = int(out.begin + C < p.tokens ? out.begin + C : p.tokens);
    out.parts = int(parts);
    out.slot = BY_MATRIX ? 0 : want;
    return true;
  }
  const int lane = threadIdx.x & 63;
  const int T = int(p.tokens);
  auto clamp = [&](int64_t v) { return int(v < 0 ? 0 : v > T ? T : v); };
  int top = clamp(p.offsets[0]);   // largest offset before this group of 64
  int64_t pieces = 0, slots = 0;
  for (int base = 0; base < p.count; base += 64) {
    const bool in = base + lane < p.count;
    int hi = in ? clamp(p.offsets[base + lane + 1]) : 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(hi, off, 64);
      if (lane >= off && o > hi) hi = o;
    }
    hi = hi > top ? hi : top;
    int lo = __shfl_up(hi, 1, 64);
    if (lane == 0) lo = top;
    const uint32_t len = uint32_t(hi - lo);
    const int n = !in ? 0 : len <= p.chunk ? 1 : int((len + p.chunk - 1) / p.chunk);
    const int m = n > 1 ? n : 0;
    int sn = n, sm = m;   // inclusive sums
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int a = __shfl_up(sn, off, 64), b = __shfl_up(sm, off, 64);
      if (lane >= off) {
        sn += a;
        sm += b;
      }
    }
    const bool hit = BY_MATRIX ? in && base + lane == want
                               : want >= pieces + sn - n && want < pieces + sn;
    const uint64_t mask = __ballot(hit);
    if (mask) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)mask) - 1);
      const int first = __builtin_amdgcn_readlane(lo, src);
      const int last = __builtin_amdgcn_readlane(hi, src);
      const int before = __builtin_amdgcn_readlane(sn - n, src);
      const int j = BY_MATRIX ? 0 : int(want - pieces) - before;
      out.e = base + src;
      out.begin = first + j * int(p.chunk);
      out.end = last - out.begin > int(p.chunk) ? out.begin + int(p.chunk) : last;
      out.parts = __builtin_amdgcn_readlane(n, src);
      out.slot = slots + __builtin_amdgcn_readlane(sm - m, src) + j;
      return true;
    }
    pieces += __builtin_amdgcn_readlane(sn, 63);
    slots += __builtin_amdgcn_readlane(sm, 63);
    top = __builtin_amdgcn_readlane(hi, 63);
  }
  return false;
}

// Four consecutive columns of one row of a matrix's gradient.
__device__ __forceinline__ void store_g(const WeightGrad& p, int64_t base, int row, int col,
                                        f32x4_t v) {
  if (row >= p.rows) return;
  const int64_t at = base + int64_t(row) * p.cols + col;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col + i >= p.cols) break;
    if (p.g_bf16) {
      uint16_t* g = static_cast<uint16_t*>(p.G) + at + i;
      *g = f2bf(p.accumulate ? bf2f(*g) + v[i] : v[i]);
    } else {
      float* g = static_cast<float*>(p.G) + at + i;
      *g = p.accumulate ? *g + v[i] : v[i];
    }
  }
}

// bf16 pairs of four checkpoint bytes (exact).
__device__ __forceinline__ void unpack_bf16(uint32_t w, float up, int fmt, uint32_t* o) {
  float v[4];
  ckpt_unpack4(w, up, fmt, v);
  o[0] = f2bf2(v[0], v[1]);
  o[1] = f2bf2(v[2], v[3]);
}

// Byte address of the 8 columns `chunk` of token row k in a [BK][128] tile.
__device__ __forceinline__ int tile_at(int k, int chunk) {
  return k * (BN * 2) + ((chunk ^ gswz(k)) << 4);
}

template <bool BF16>
__global__ __launch_bounds__(NT, 2) void weight_grad_kernel(const WeightGrad p, int tiles_n,
                                                            int tiles) {
  constexpr int P = BF16 ? 1 : 3;            // bf16 parts of dy
  constexpr int PLANE = BK * BM * 2;         // bytes
  constexpr int STAGE = (P + 1) * PLANE;
  static_assert(BM == BN, "one tile layout");
  __shared__ __attribute__((aligned(1024))) char smem_raw[2 * STAGE];
  LDS_AS char* smem = (LDS_AS char*)smem_raw;

  const int64_t number = blockIdx.x / unsigned(tiles);
  const int tile = int(blockIdx.x - number * tiles);
  Piece pc;
  if (!find_piece<false>(p, number, pc)) return;
  const int i0 = tile / tiles_n * BM, j0 = tile % tiles_n * BN;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // This thread's part of a step: 8 columns of dy of two tokens, 16 of x of one.
  const int yk = t >> 4, yc = t & 15;
  const int xk = t >> 3, xc = t & 7;
  using T = typename RowVec<BF16>::T;
  constexpr int N = RowVec<BF16>::N;
  float y[2][8];
  uint32_t xr[4];
  int xs;
  auto load = [&](int k0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + yk + 16 * h;
      const T* row = static_cast<const T*>(p.dy) + int64_t(k) * p.lddy;
#pragma unroll
      for (int i = 0; i < 8; i += N) {
        if (k < pc.end) {
          load_vec<BF16>(row, i0 + yc * 8 + i, p.rows, y[h] + i);
        } else {
#pragma unroll
          for (int c = 0; c < N; ++c) y[h][i + c] = 0.f;
        }
      }
    }
    const int k = k0 + xk, col = j0 + xc * 16;
    xr[0] = xr[1] = xr[2] = xr[3] = 0;
    xs = 0;
    if (k < pc.end && col < p.x.q_pitch) {
      const uint4 w = *reinterpret_cast<const uint4*>(p.x.q + int64_t(k) * p.x.q_pitch + col);
      xr[0] = w.x;
      xr[1] = w.y;
      xr[2] = w.z;
      xr[3] = w.w;
      xs = p.x.scale[int64_t(k) * p.x.s_pitch + col / MUON_CKPT_BLOCK];
    }
  };
  auto write = [&](int buf) {
    LDS_AS char* s = smem + buf * STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = y[h][i];
#pragma unroll
      for (int part = 0; part < P; ++part) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the leading 8 bits of each value; an infinity leaves no remainder
          const uint32_t a = __float_as_uint(v[2 * i]) & 0xffff0000u;
          const uint32_t b = __float_as_uint(v[2 * i + 1]) & 0xffff0000u;
          w[i] = (a >> 16) | b;
          if (part + 1 < P) {
            const float fa = __uint_as_float(a), fb = __uint_as_float(b);
            v[2 * i] = v[2 * i] == fa ? 0.f : v[2 * i] - fa;
            v[2 * i + 1] = v[2 * i + 1] == fb ? 0.f : v[2 * i + 1] - fb;
          }
        }
        *reinterpret_cast<LDS_AS u32x4_t*>(s + part * PLANE + tile_at(yk + 16 * h, yc)) =
            u32x4_t{w[0], w[1], w[2], w[3]};
      }
    }
    const float up = ckpt_up(xs);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack_bf16(xr[i], up, p.x.fmt, o + 2 * i);
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
  if (steps > 0) {
    load(pc.begin);
    write(0);
  }
  __syncthreads();
  for (int k = 0; k < steps; ++k) {
    if (k + 1 < steps) load(pc.begin + (k + 1) * BK);
    const LDS_AS char* s = smem + (k & 1) * STAGE;
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks) {
      bf16x8_t xf[2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
        xf[b] = lds_frag_xT<BN>(s + P * PLANE, ks * 16, wn * 64 + b * 32, lane);
#pragma unroll
      for (int part = P - 1; part >= 0; --part)
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const bf16x8_t yf = lds_frag_xT<BM>(s + part * PLANE, ks * 16, wm * 64 + a * 32, lane);
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xf[b], yf, acc[a][b], 0, 0, 0);
        }
    }
    if (k + 1 < steps) write((k + 1) & 1);
    __syncthreads();
  }

  // Lane l, register 4 g + i of a 32 x 32 block: row l % 32, column 8 g + 4 (l / 32) + i.
  const bool direct = pc.parts == 1;
  if (direct && steps == 0 && p.accumulate) return;
  const int64_t base = int64_t(pc.e) * p.rows * p.cols;
  float* part = p.partial + (pc.slot * tiles + tile) * int64_t(kTile);
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4_t v = {acc[a][b][4 * g], acc[a][b][4 * g + 1], acc[a][b][4 * g + 2],
                           acc[a][b][4 * g + 3]};
        if (direct)
          store_g(p, base, i0 + wm * 64 + a * 32 + (lane & 31),
                  j0 + wn * 64 + b * 32 + 8 * g + 4 * (lane >> 5), v);
        else
          *reinterpret_cast<f32x4_t*>(part + ((((a * 2 + b) * 4 + g) * 4 + wave) * 64 + lane) * 4) = v;
      }
}

// Adds the partial tiles of matrices with several pieces, one 32 x 32 block
// of each wave's tile per block.
__global__ __launch_bounds__(NT) void join_kernel(const WeightGrad p, int tiles_n, int tiles) {
  const int64_t id = blockIdx.x;
  const int ab = int(id & 3);
  const int tile = int((id >> 2) % tiles);
  Piece pc;
  if (!find_piece<true>(p, (id >> 2) / tiles, pc) || pc.parts == 1) return;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int wm = wave >> 1, wn = wave & 1, a = ab >> 1, b = ab & 1;
  const int64_t base = int64_t(pc.e) * p.rows * p.cols;
  f32x4_t sum[4] = {};
  for (int j = 0; j < pc.parts; ++j) {
    const float* part = p.partial + ((pc.slot + j) * tiles + tile) * int64_t(kTile);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      sum[g] += *reinterpret_cast<const f32x4_t*>(part + (((ab * 4 + g) * 4 + wave) * 64 + lane) * 4);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g)
    store_g(p, base, tile / tiles_n * BM + wm * 64 + a * 32 + (lane & 31),
            tile % tiles_n * BN + wn * 64 + b * 32 + 8 * g + 4 * (lane >> 5), sum[g]);
}

int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }

}  // namespace

// Pieces: enough blocks for two per CU, of at least 128 tokens each.
WeightGradPlan weight_grad_plan(int64_t count, int64_t tokens, int64_t rows, int64_t cols) {
  constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;
  WeightGradPlan w{};
  w.bm = BM;
  w.bn = BN;
  w.tiles = cdiv(rows, BM) * cdiv(cols, BN);
  const int64_t want = std::max<int64_t>(count, 512 / w.tiles);
  const int64_t chunk = std::max<int64_t>(128, cdiv(cdiv(tokens, want), BK) * BK);
  w.chunk = uint32_t(chunk);
  if (count == 1) {
    w.pieces = std::max<int64_t>(1, cdiv(tokens, chunk));
    w.slots = w.pieces > 1 ? w.pieces : 0;
  } else {
    w.pieces = tokens / chunk + count;
    w.slots = tokens > chunk ? std::min(2 * tokens / chunk, w.pieces) : 0;
  }
  if (w.pieces * w.tiles > kMaxBlocks || 4 * count * w.tiles > kMaxBlocks) {
    w.pieces = 0;
    return w;
  }
  w.partial_bytes = size_t(w.slots) * size_t(w.tiles) * kTile * 4;
  return w;
}

hipError_t launch_weight_grad(const WeightGrad& p, const WeightGradPlan& plan, bool bf16,
                              hipStream_t s) {
  const int tiles_n = int(cdiv(p.cols, BN));
  const dim3 grid(unsigned(plan.pieces * plan.tiles));
  if (bf16)
    hipLaunchKernelGGL(weight_grad_kernel<true>, grid, dim3(NT), 0, s, p, tiles_n, int(plan.tiles));
  else
    hipLaunchKernelGGL(weight_grad_kernel<false>, grid, dim3(NT), 0, s, p, tiles_n, int(plan.tiles));
  return hipGetLastError();
}

hipError_t launch_weight_grad_join(const WeightGrad& p, const WeightGradPlan& plan, hipStream_t s) {
  const int tiles_n = int(cdiv(p.cols, BN));
  hipLaunchKernelGGL(join_kernel, dim3(unsigned(4 * p.count * plan.tiles)), dim3(NT), 0, s, p,
                     tiles_n, int(plan.tiles));
  return hipGetLastError();
}

}  // namespace muon
