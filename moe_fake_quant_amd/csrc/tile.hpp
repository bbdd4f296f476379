// Pieces that the tiled MFMA kernels share (gfx950): the fragment types, the
// swizzled LDS layout of a contraction-contiguous stage, global -> LDS loads with
// their waits, and the tile list of a segmented call.
#pragma once

#include "common.hpp"

namespace fq {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8v;
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
constexpr int NT = 512;   // threads per block (8 waves, 2 per SIMD)

// Contraction-contiguous layout: row idx (0..255) of 8 16-byte chunks (8
// contraction elements each); chunk kc sits at kc ^ sw(idx). The swizzle
// (rows in pairs share one) was chosen by measuring the LDS bank-conflict
// counter for the fragment read pattern (32 consecutive rows, one chunk).
__device__ __forceinline__ uint32_t nrm_sw(uint32_t idx) { return (idx >> 1) & 7u; }
__device__ __forceinline__ uint32_t nrm_off(uint32_t idx, uint32_t kc) {
  return idx * 128u + ((kc ^ nrm_sw(idx)) << 4);
}

// 16 bytes per lane from global memory into LDS at lds_wave_base + 16 * lane:
// the lane reads base + off (base uniform, held in scalar registers).
// Issued as inline asm: the compiler then does not model the LDS write and
// inserts no wait before reads of the other stages; the ring's own
// vmcnt waits and barriers order the accesses. The compiler's hazard pass
// does not look inside the asm, so it starts with the wait states the
// hardware needs when the instruction just before wrote M0 (one) or, as a
// vector instruction (v_readfirstlane), one of the base registers (five).
__device__ __forceinline__ void dma16(const char *base, uint32_t off, char *lds_wave_base) {
  const uint32_t m0v = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds_wave_base);
  // readfirstlane returns a signed int: widen through uint32_t (no sign extension)
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint64_t sb = ((uint64_t)hi << 32) | (uint64_t)lo;
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(sb), "{m0}"(m0v)
               : "memory");
}

// One barrier for the whole block without a memory fence (a fence would wait
// for every outstanding load, draining the ring).
__device__ __forceinline__ void block_barrier() { asm volatile("s_barrier" ::: "memory"); }

// s_waitcnt lgkmcnt(0) leaving the other counters alone (gfx9 encoding): this
// wave's LDS reads have returned
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// s_waitcnt vmcnt(n) leaving the other counters alone (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

constexpr int kMaxExperts = 1024;

// tile_start[e] = number of work units of experts 0..e-1 (e = 0..E), from
// seg_offsets on the device: a block-wide exclusive scan in LDS. Units per
// expert: ceil(rows / rows_per_unit), at least min_units.
template <int THREADS = NT>
__device__ inline void build_tile_prefix(const int32_t *seg, int E, int rows_per_unit, int min_units,
                                         int *tile_start) {
  __shared__ int s_wsum[THREADS / 64];
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    const int nt =
        e < E ? max((seg[e + 1] - seg[e] + rows_per_unit - 1) / rows_per_unit, min_units) : 0;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int x = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (lane == 63) s_wsum[w] = x;
    __syncthreads();
    int before = base, total = base;
#pragma unroll
    for (int k = 0; k < THREADS / 64; ++k) {
      if (k < w) before += s_wsum[k];
      total += s_wsum[k];
    }
    if (e < E) tile_start[e] = before + x - nt;
    __syncthreads();
    base = total;
  }
  if (threadIdx.x == 0) tile_start[E] = base;
  __syncthreads();
}

// expert of row tile `tile`: the last e with tile_start[e] <= tile
__device__ __forceinline__ int expert_of_tile(const int *tile_start, int E, int tile) {
  int lo = 0, hi = E;  // tile_start[lo] <= tile < tile_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace fq
