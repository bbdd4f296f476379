// Device helpers of the passes that hold whole rows in registers (gfx950): sums
// and maxima over the lanes of a row, and the int8 codes of a row with one scale.
#pragma once

#include "actq.hpp"

namespace fq {

// A row of nv 8-element vectors lies over WPR waves: lane `lane` of the row's
// WPR * 64 lanes holds the vectors lane + i * WPR * 64. A block is four rows of one
// wave each (no barrier), or one row.
template <int WPR>
constexpr int kRowThreads = WPR == 1 ? 256 : WPR * 64;
template <int WPR>
constexpr int kBlockRows = WPR == 1 ? 4 : 1;

// the row of this thread's group; the grid's last blocks may lie behind the last row
template <int WPR>
__device__ __forceinline__ uint32_t grid_row() {
  return block_of_grid() * (uint32_t)kBlockRows<WPR> + threadIdx.x / (uint32_t)(WPR * 64);
}

// Sums of N values over the row's lanes, the same in each of them and in a fixed
// order. WPR > 1: every thread of the block takes part; `red` has room for WPR * N
// floats and is free again at the next barrier.
template <int WPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], o, 64);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[w * N + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = red[k];
#pragma unroll
      for (int j = 1; j < WPR; ++j) v[k] += red[j * N + k];
    }
  }
}

// the largest of the magnitude bits `m` over the row's lanes
template <int WPR>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t m, uint32_t *red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int j = 1; j < WPR; ++j) m = max(m, red[j]);
  }
  return m;
}

// A token's int8 scale from its largest magnitude (the bits of an fp32): as one
// group of the 8-bit checkpoints, s = max(amax * fp32(1/127), 2^-126), 1 for a
// row of zeros, NaN with codes 0 for a row that is not finite.
struct TokenScale {
  float s, r;
  bool finite;
};
__device__ __forceinline__ TokenScale token_scale(uint32_t top) {
  TokenScale t;
  t.finite = top < 0x7F800000u;
  t.s = fmaxf(__uint_as_float(top) * (1.0f / 127.0f), 0x1p-126f);
  if (top == 0) t.s = 1.0f;
  if (!t.finite) t.s = __uint_as_float(0x7FC00000u);
  t.r = t.finite ? 1.0f / t.s : 0.0f;
  return t;
}

// the 8 codes of rne(clamp(x / s)), element j in byte j
__device__ __forceinline__ uint2 token_codes8(const float *x, const TokenScale &t) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // z + 1.5 * 2^23 rounds z to an integer (ties to even); its two's complement
    // is the sum's low byte
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b[j] = __float_as_uint(fminf(fmaxf(x[4 * h + j] * t.r, -128.0f), 127.0f) + 12582912.0f);
    w[h] = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u) |
           __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    if (!t.finite) w[h] = 0u;
  }
  return make_uint2(w[0], w[1]);
}

// magnitude bits of the largest of 8 bf16 values, as an fp32
__device__ __forceinline__ uint32_t max_bits8(const bf16x8_t &v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max((v.w[i] << 16) & 0x7FFFFFFFu, v.w[i] & 0x7FFF0000u));
  return m;
}

}  // namespace fq
