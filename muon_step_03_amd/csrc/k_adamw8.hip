// AdamW with both moments in 8 bits (include/muon.h, "State format").  The
// state holds m as e4m3 and r = sqrt(v) with 4 bits of exponent and 4 of
// mantissa, each with a power-of-two scale per 32 elements; the arithmetic is
// float32 throughout, and the kept values are rounded stochastically by bits
// hashed from the element's index.
//
// 10.1 bytes per element move with bf16 p and g (p r/w, g r, m r/w, r r/w),
// 16.1 with float32, against 22 and 28 of float32 states.  A thread takes
// vectors of 8 consecutive elements, so 4 neighbouring lanes hold a block and
// find its largest magnitude with two lane exchanges; all loads of a thread
// are issued before its arithmetic.  HBM-bound, with the vector units close
// behind: 77 M elements of bf16 (GPT-160M's embedding and head) take 148 us on
// one MI355X, 5.3 TB/s where a 1 GiB copy moves 5.45; reading both moments
// back 76 us (6.1).
#include <type_traits>

#include "adamw8_internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int V = kAdam8Vec;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Scale exponents of r: its smallest step, 2^-10 * 2^e, is a normal number.
constexpr int kRootEMin = -116, kRootEMax = 118;

// Scale byte of a block of r whose largest value has the bit pattern `a`:
// e + 127, e the smallest exponent with a <= 496 * 2^e = 1.9375 * 2^(8+e).
__device__ __forceinline__ int root_scale_byte(uint32_t a) {
  int e = int(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x780000u ? 1 : 0);
  e = e < kRootEMin ? kRootEMin : e > kRootEMax ? kRootEMax : e;
  return a >= kInfBits ? 255 : e + 127;
}

// 32 random bits of element i.
__device__ __forceinline__ uint32_t random_bits(uint64_t i, uint32_t seed) {
  uint32_t x = uint32_t(i) * 0x9e3779b1u + uint32_t(i >> 32) * 0x85ebca77u + seed;
  x = (x ^ x >> 16) * 0x7feb352du;
  x = (x ^ x >> 15) * 0x846ca68bu;
  return x ^ x >> 16;
}

// Multiplied by 2^-120, a magnitude whose exponent has bias 7 becomes the
// float32 with the same exponent field, and one below the format's normal
// numbers a subnormal float32: the format's bits are the ones behind the sign,
// those to be rounded off follow.  `exp` brings the block into range and does
// that at once (2^-120 2^(127 - scale)).
__device__ __forceinline__ uint32_t keep_m(float m, int exp, uint32_t random) {
  const uint32_t b = __float_as_uint(__builtin_amdgcn_ldexpf(__builtin_fabsf(m), exp)) +
                     ((random >> 12 & 0xffff0u) | 8u);
  return min(b, 0x7efffffu) >> 20;   // without its sign
}
__device__ __forceinline__ uint32_t keep_r(float r, int exp, uint32_t random) {
  const uint32_t b = __float_as_uint(__builtin_amdgcn_ldexpf(r, exp)) + ((random & 0xffffu) * 8 + 4);
  return r > 0.f ? min(max(b, 0x80000u), 0x7ffffffu) >> 19 : 0u;
}
// The sign bits of four floats, one per byte.
__device__ __forceinline__ uint32_t signs4(const float* v) {
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(v[1]), __float_as_uint(v[0]), 0x0c0c0703u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(v[3]), __float_as_uint(v[2]), 0x07030c0cu);
  return (lo | hi) & 0x80808080u;
}

struct Coef {
  float b1, omb1, b2, omb2, eps, inv_sqrt_bc2, decay, step_size;
};

// Every rounding is spelled out: m' and v' are the float32 operations of the
// formula one by one.  The root and the quotient of most elements take the
// hardware's estimates and one correction by the exact remainder, which leaves
// them within 0.51 units of the last place: for a root between 2^-40 and 2^40
// (or zero), where no intermediate value leaves the normal numbers.  Vectors
// with others take the library's root and division, which are twice as long
// (all of them: 176 us for 77 M elements of bf16, bound by the vector units).
__device__ __forceinline__ void adam_vec(float* p, const float* g, float* m, float* r, const Coef& c) {
#pragma clang fp contract(off)
  float v[V], u[V];
  float least = 1.f, most = 1.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m[i] = c.b1 * m[i] + c.omb1 * g[i];
    v[i] = c.b2 * (r[i] * r[i]) + c.omb2 * (g[i] * g[i]);
    u[i] = v[i] == 0.f ? 1.f : v[i];
    least = __builtin_fminf(least, u[i]);
    most = __builtin_fmaxf(most, u[i]);
  }
  // (a NaN fails neither test, and passes through the estimates)
  if (least >= 0x1p-80f && most <= 0x1p80f && c.eps >= 0x1p-80f) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float y = __builtin_amdgcn_rsqf(u[i]), root = u[i] * y;
      const float fixed = __builtin_fmaf(__builtin_fmaf(-root, root, u[i]), 0.5f * y, root);
      r[i] = v[i] == 0.f ? 0.f : fixed;
      const float denom = r[i] * c.inv_sqrt_bc2 + c.eps;
      const float inv = __builtin_amdgcn_rcpf(denom), q = m[i] * inv;
      const float ratio = __builtin_fmaf(__builtin_fmaf(-denom, q, m[i]), inv, q);
      p[i] = __builtin_fmaf(c.decay, p[i], -(c.step_size * ratio));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      r[i] = __builtin_sqrtf(v[i]);
      const float denom = r[i] * c.inv_sqrt_bc2 + c.eps;
      p[i] = __builtin_fmaf(c.decay, p[i], -(c.step_size * (m[i] / denom)));
    }
  }
}

// Eight elements from `col` on of `left`, those past the end as zero: as they
// are loaded (16 bytes of bf16, 32 of float32), and as numbers.
template <bool BF16>
struct Eight {
  u32x4_t w[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Eight<BF16> load8(const void* base, int col, int left) {
  using R = RowVec<BF16>;
  Eight<BF16> o;
#pragma unroll
  for (int h = 0; h < V / R::N; ++h) {
    const int at = col + h * R::N;
    if (at + R::N <= left) {
      const typename R::Raw r = __builtin_nontemporal_load(reinterpret_cast<const typename R::Raw*>(
          static_cast<const typename R::T*>(base) + at));
      o.w[h] = u32x4_t{r[0], r[1], r[2], r[3]};
    } else {
      o.w[h] = load_raw<BF16>(base, at, left);
    }
  }
  return o;
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const Eight<BF16>& o, float* v) {
#pragma unroll
  for (int h = 0; h < V / RowVec<BF16>::N; ++h) unpack_raw<BF16>(o.w[h], v + h * RowVec<BF16>::N);
}
template <bool BF16>
__device__ __forceinline__ void store8(void* base, int col, int left, const float* v) {
#pragma unroll
  for (int h = 0; h < V; h += RowVec<BF16>::N)
    store_vec<BF16, true>(base, col + h, left, v + h);
}

// Eight bytes of a state and their scale, of the blocks that begin before `left`.
struct Kept {
  u32x2_t q;
  int scale;
};
__device__ __forceinline__ Kept load_kept(const uint8_t* q, const uint8_t* scale, int col, int left) {
  Kept k{{0, 0}, 0};
  if ((col & ~(MUON_CKPT_BLOCK - 1)) < left) {
    k.q = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(q + col));
    k.scale = scale[col / MUON_CKPT_BLOCK];
  }
  return k;
}
__device__ __forceinline__ void values_m(const Kept& k, float* v) {
  const float up = ckpt_up(k.scale);
  ckpt_unpack4(k.q[0], up, MUON_CKPT_E4M3, v);
  ckpt_unpack4(k.q[1], up, MUON_CKPT_E4M3, v + 4);
}
__device__ __forceinline__ void values_r(const Kept& k, float* v) {
  const int exp = k.scale - 127 + 120;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t c = k.q[i / 4] >> (8 * (i & 3)) & 0xffu;
    v[i] = __builtin_amdgcn_ldexpf(__uint_as_float(c << 19), exp);
  }
  if (k.scale == 255) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __builtin_nanf("");
  }
}

// The largest magnitude of a block, as a bit pattern, from its four lanes.
__device__ __forceinline__ uint32_t block_max(const float* v) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) a = max(a, __float_as_uint(v[i]) & 0x7fffffffu);
  a = max(a, dpp<kXor1>(a));
  return max(a, dpp<kXor2>(a));
}

// The tensor of a block and its first element: the lanes look at a tensor each
// (looking one by one, 48 loads that wait for each other, cost 16 us).
__device__ __forceinline__ const Adam8Seg& find_seg(const Adam8Batch& bt, int64_t& base) {
  static_assert(kAdam8Segs <= 64, "a lane per tensor");
  const int lane = threadIdx.x & 63;
  const bool from = lane < bt.nseg && blockIdx.x >= bt.seg[lane < bt.nseg ? lane : 0].begin;
  const int s = __builtin_popcountll(__ballot(from)) - 1;
  base = int64_t(blockIdx.x - bt.seg[s].begin) * kAdam8Chunk;
  return bt.seg[s];
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void adamw8_kernel(const Adam8Batch bt) {
  using T = typename RowVec<BF16>::T;
  int64_t base;
  const Adam8Seg& sg = find_seg(bt, base);
  const Coef c{bt.beta1, bt.one_minus_beta1, bt.beta2, bt.one_minus_beta2, bt.eps, bt.inv_sqrt_bc2,
               sg.decay, sg.step_size};
  const int left = int(sg.n - base < kAdam8Chunk ? sg.n - base : kAdam8Chunk);
  T* P = static_cast<T*>(sg.P) + base;
  const T* G = static_cast<const T*>(sg.G) + base;
  uint8_t *mq = sg.m_q + base, *rq = sg.r_q + base;
  uint8_t *ms = sg.m_scale + base / MUON_CKPT_BLOCK, *rs = sg.r_scale + base / MUON_CKPT_BLOCK;

  Eight<BF16> p8[kAdam8PerThread], g8[kAdam8PerThread];
  Kept m8[kAdam8PerThread], r8[kAdam8PerThread];
  // WHOLE: no element of the chunk lies past the tensor's end
  auto run = [&](auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int n = WHOLE ? kAdam8Chunk : left;
#pragma unroll
    for (int j = 0; j < kAdam8PerThread; ++j) {
      const int col = (j * kThreads + int(threadIdx.x)) * V;
      p8[j] = load8<BF16>(P, col, n);
      g8[j] = load8<BF16>(G, col, n);
      m8[j] = load_kept(mq, ms, col, n);
      r8[j] = load_kept(rq, rs, col, n);
    }
#pragma unroll
    for (int j = 0; j < kAdam8PerThread; ++j) {
      const int col = (j * kThreads + int(threadIdx.x)) * V;
      // the four lanes of a block pass together
      if (!WHOLE && (col & ~(MUON_CKPT_BLOCK - 1)) >= n) continue;
      float p[V], g[V], m[V], r[V];
      unpack8<BF16>(p8[j], p);
      unpack8<BF16>(g8[j], g);
      values_m(m8[j], m);
      values_r(r8[j], r);
      adam_vec(p, g, m, r, c);
      if constexpr (!WHOLE) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (col + i >= n) m[i] = r[i] = 0.f;
      }
      store8<BF16>(P, col, n, p);
      const int mb = ckpt_scale_byte(block_max(m), MUON_CKPT_E4M3), rb = root_scale_byte(block_max(r));
      u32x2_t mw = {0, 0}, rw = {0, 0};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t random = random_bits(uint64_t(base + col + i), sg.seed);
        uint32_t mk = keep_m(m[i], 7 - mb, random);
        // what follows the end stays zero (no random bits lift a zero r)
        if (!WHOLE && col + i >= n) mk = 0;
        mw[i / 4] |= mk << (8 * (i & 3));
        rw[i / 4] |= keep_r(r[i], 7 - rb, random) << (8 * (i & 3));
      }
      mw[0] |= signs4(m);
      mw[1] |= signs4(m + 4);
      if (mb == 255) mw = u32x2_t{0, 0};
      if (rb == 255) rw = u32x2_t{0, 0};
      __builtin_nontemporal_store(mw, reinterpret_cast<u32x2_t*>(mq + col));
      __builtin_nontemporal_store(rw, reinterpret_cast<u32x2_t*>(rq + col));
      if (col % MUON_CKPT_BLOCK == 0) {
        ms[col / MUON_CKPT_BLOCK] = uint8_t(mb);
        rs[col / MUON_CKPT_BLOCK] = uint8_t(rb);
      }
    }
  };
  if (left == kAdam8Chunk)
    run(std::true_type{});
  else
    run(std::false_type{});
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void moments_kernel(const Adam8Batch bt) {
  using T = typename RowVec<BF16>::T;
  int64_t base;
  const Adam8Seg& sg = find_seg(bt, base);
  const int left = int(sg.n - base < kAdam8Chunk ? sg.n - base : kAdam8Chunk);
  T* m_out = static_cast<T*>(sg.P) + base;
  T* r_out = static_cast<T*>(const_cast<void*>(sg.G)) + base;
  const int64_t block = base / MUON_CKPT_BLOCK;
  Kept m8[kAdam8PerThread], r8[kAdam8PerThread];
#pragma unroll
  for (int j = 0; j < kAdam8PerThread; ++j) {
    const int col = (j * kThreads + int(threadIdx.x)) * V;
    m8[j] = load_kept(sg.m_q + base, sg.m_scale + block, col, left);
    r8[j] = load_kept(sg.r_q + base, sg.r_scale + block, col, left);
  }
#pragma unroll
  for (int j = 0; j < kAdam8PerThread; ++j) {
    const int col = (j * kThreads + int(threadIdx.x)) * V;
    float m[V], r[V];
    values_m(m8[j], m);
    values_r(r8[j], r);
    store8<BF16>(m_out, col, left, m);
    store8<BF16>(r_out, col, left, r);
  }
}

}  // namespace

hipError_t launch_adamw8(const Adam8Batch& bt, bool bf16, hipStream_t s) {
  if (bf16)
    hipLaunchKernelGGL(adamw8_kernel<true>, dim3(bt.blocks), dim3(kThreads), 0, s, bt);
  else
    hipLaunchKernelGGL(adamw8_kernel<false>, dim3(bt.blocks), dim3(kThreads), 0, s, bt);
  return hipGetLastError();
}

hipError_t launch_adamw8_moments(const Adam8Batch& bt, bool bf16, hipStream_t s) {
  if (bf16)
    hipLaunchKernelGGL(moments_kernel<true>, dim3(bt.blocks), dim3(kThreads), 0, s, bt);
  else
    hipLaunchKernelGGL(moments_kernel<false>, dim3(bt.blocks), dim3(kThreads), 0, s, bt);
  return hipGetLastError();
}

}  // namespace muon
