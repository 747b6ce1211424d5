// LDS tiles and direct-to-LDS loads of the bf16 matrix kernels
// (k_ns_bf16.hip, k_weight_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
#define LDS_AS __attribute__((address_space(3)))

constexpr int WAVE_BYTES = 1024;    // bytes one direct-to-LDS instruction moves
// LDS banking measured on gfx950 (bank-conflict counters over single-pattern
// probes): 64 banks of 4 bytes; a 16-byte read serves 16 lanes per clock
// (lanes 0-31 and 32-63 each in two sets of four quads, split by the parity
// of the quad index), an 8-byte read (plain or transposing) 32 lanes.
//
// Chunk swizzle of the update's N-contiguous X tile (K-rows of 256 bytes, all
// on the same banks): chunk c of K-row k is stored at c ^ {0, 6, 12, 10}[k & 3],
// so the 4 K-rows x 64 bytes that 32 lanes of a transposing read take cover
// the 64 banks once.
__device__ __forceinline__ int gswz(int k) { return (0xAC60 >> ((k & 3) * 4)) & 15; }

// vmcnt-only wait (expcnt and lgkmcnt left at their maxima).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// 16-byte direct-to-LDS load: lane L's 16 bytes from `base + off` land at
// LDS address lds_base + 16 L (lds_base wave-uniform, passed in m0; base a
// 64-bit scalar address, off the lane's 32-bit byte offset).  Written as asm
// so that the compiler does not treat every later LDS read as possibly
// aliasing it (which would make it wait for all loads in flight, prefetches
// included); completion is tracked explicitly with wait_vmcnt before the
// barrier that publishes a K step.  The instruction has no result register.
// It reads m0 one wait state after a scalar write at the earliest, which only the
// compiler's own instructions are spaced for: s_nop.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(uint32_t off, const char* base, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_base)
               : "memory", "m0");
}
// The same for 4 bytes per lane.
__device__ __forceinline__ void dma4(uint32_t off, const char* base, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Workgroup barrier that publishes this wave's LDS traffic (lgkmcnt(0): its
// LDS reads and writes are complete) but leaves global loads in flight (no
// vmcnt wait, unlike a fence); the empty asm statements keep the compiler
// from moving LDS accesses across it in either direction.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((7 << 4) | (0 << 8) | 15 | (3 << 14));  // lgkmcnt(0) only
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Completes this wave's LDS writes before its following LDS reads of other
// lanes' data (a wave-private exchange: no other wave takes part), and keeps
// the compiler from moving LDS accesses across it.
__device__ __forceinline__ void wave_lds_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((7 << 4) | (0 << 8) | 15 | (3 << 14));  // lgkmcnt(0) only
  asm volatile("" ::: "memory");
}

template <int BN>
__device__ __forceinline__ bf16x8_t lds_frag_xT(const LDS_AS char* tile, int kb, int nb, int lane) {
  const int s = lane & 15;
  const int n = nb + 16 * ((lane >> 4) & 1) + 4 * (s & 3);
  const int k = kb + 8 * (lane >> 5) + (s >> 2);
  const LDS_AS char* p0 = tile + k * (BN * 2) + (((n >> 3) ^ gswz(k)) << 4) + (n & 7) * 2;
  const LDS_AS char* p1 = tile + (k + 4) * (BN * 2) + (((n >> 3) ^ gswz(k + 4)) << 4) + (n & 7) * 2;
  const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)p0);
  const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)p1);
  const i16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

}  // namespace
}  // namespace muon
