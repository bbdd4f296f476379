// Arguments of the int8 and gated products, shared by the kernels for few rows
// (product.hip), a middling number (mid_product.hip) and many (tile_product.hip).
#pragma once

#include "actq.hpp"
#include "internal.hpp"
#include "tile.hpp"

namespace fq {

typedef int i32x4 __attribute__((ext_vector_type(4)));

enum Kind { PLAIN = 0, GATED = 1, GATED_BWD = 2 };

struct ProdArgs {
  const char *w, *x;       // weights [E, N, KB], x rows of KB bytes
  const int32_t *perm;     // x row of routed row r is perm[r] / topk; NULL: r
  FastDiv topk;
  const int32_t *seg;      // [E + 1]
  int E, N;                // weight rows of an expert (gated: 2F)
  int C;                   // output columns (N, gated: F)
  uint32_t KB;             // bytes of a row
  const float *sx, *sw;    // int8: token scales, channel scales
  int sw_rows;             // 1: sw [E, N], 0: sw [E]
  const uint16_t *daq;     // bwd [R, F]
  int afmt;
  const float *ascale;
  uint16_t *out;           // y, aq or dh
  uint16_t *aq;            // bwd: FQ_a(a), or NULL
};

__device__ __forceinline__ int x_row(const ProdArgs &a, int r) {
  return a.perm ? (int)a.topk.div((uint32_t)a.perm[r]) : r;
}

// dh of one element: dg = da u s (1 + g (1 - s)), du = da g s, s = sigmoid(g)
__device__ __forceinline__ void swiglu_grad(float da, float g, float u, float s, float &dg, float &du) {
  dg = ((da * u) * s) * (1.0f + g * (1.0f - s));
  du = (da * g) * s;
}

// 8 sums of row r and weight rows n0 .. n0+7 of expert e, from their place in LDS
// (16-byte aligned): fp32, or int32 with the scales of the row and the channels
template <bool I8>
__device__ __forceinline__ void sums8(const ProdArgs &a, int e, int r, int n0, const int *src, float *v) {
  int w[8];
  *reinterpret_cast<i32x4 *>(w) = *reinterpret_cast<const i32x4 *>(src);
  *reinterpret_cast<i32x4 *>(w + 4) = *reinterpret_cast<const i32x4 *>(src + 4);
  if constexpr (I8) {
    const float sx = a.sx[x_row(a, r)];
    const float *sw = a.sw + (a.sw_rows ? (size_t)e * a.N + n0 : (size_t)e);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = ((float)w[k] * sx) * sw[a.sw_rows ? k : 0];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __int_as_float(w[k]);
  }
}

// The outputs of 8 columns c0 .. c0+7 of row r from their sums (g, and u for the
// gated kinds). Lane ^ 1 holds the other half of the 16-block and runs the same
// call; `store` says whether this lane's row exists.
template <int KIND>
__device__ __forceinline__ void finish8(const ProdArgs &a, const ActQ &q, int r, int c0, float *g,
                                        const float *u, bool store) {
  if constexpr (KIND == PLAIN) {
    if (store) *reinterpret_cast<bf16x8_t *>(a.out + (size_t)r * a.C + c0) = pack8(g);
  } else {
    float v[8], sig[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sig[j] = sigmoid_hw(g[j]);
      v[j] = bf16_to_f32(f32_to_bf16((g[j] * sig[j]) * u[j]));
    }
    const uint32_t m = act_fq8_pair(q, v);
    if constexpr (KIND == GATED) {
      if (store) *reinterpret_cast<bf16x8_t *>(a.out + (size_t)r * a.C + c0) = pack8(v);
    } else if (store) {
      if (a.aq) *reinterpret_cast<bf16x8_t *>(a.aq + (size_t)r * a.C + c0) = pack8(v);
      float d[8], dg[8], du[8];
      unpack8(*reinterpret_cast<const bf16x8_t *>(a.daq + (size_t)r * a.C + c0), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float da = (m >> j) & 1u ? d[j] : 0.0f;
        swiglu_grad(da, g[j], u[j], sig[j], dg[j], du[j]);
      }
      uint16_t *o = a.out + (size_t)r * 2 * a.C + c0;
      *reinterpret_cast<bf16x8_t *>(o) = pack8(dg);
      *reinterpret_cast<bf16x8_t *>(o + a.C) = pack8(du);
    }
  }
}

// Tile order: groups of gm row tiles, a group's tiles column by column with the row
// tile fastest, so that the tiles in flight on an XCD form a block that shares both
// operands' panels in its L2 (gm = 1: columns fastest).
__device__ __forceinline__ void tile_of(int w, int n_it, int gm, int n_rows, int &row, int &it) {
  const int g = w / (gm * n_it), r0 = g * gm, gs = min(gm, n_rows - r0);
  const int in = w - g * gm * n_it;
  // divisions come out of vector registers: the same in every lane, taken back
  it = __builtin_amdgcn_readfirstlane(in / gs);
  row = __builtin_amdgcn_readfirstlane(r0 + (in - it * gs));
}
// gm for `flight` tiles in flight on an XCD and about `rows` row tiles an expert: the
// side of a square block, unless a row of tiles is too short to fill more than one
inline int tile_group(int flight, int n_it, int rows) {
  int g = 1;
  while ((g + 1) * (g + 1) <= flight) ++g;
  if (g > rows) g = rows;
  return n_it >= 2 * g && g > 1 ? g : 1;
}

// 16-byte chunk of a 128-byte stage row that a lane carries in the DMA instructions
// of parity ii & 1 (the swizzle of tile.hpp over 8-row pieces)
__device__ __forceinline__ uint32_t lane_chunk(int lane, int ii) {
  return (uint32_t)(lane & 7) ^ (uint32_t)((4 * (ii & 1) + (lane >> 4)) & 7);
}

// one 32x32 MFMA tile over 16 bytes a lane: 16 bf16 or 32 int8 of the contraction
typedef __attribute__((__vector_size__(16 * sizeof(int)))) int i32x16v;
template <bool I8>
struct Acc32 {
  typedef f32x16 type;
};
template <>
struct Acc32<true> {
  typedef i32x16v type;
};
template <bool I8>
__device__ __forceinline__ void mfma32(const i32x4 &p, const i32x4 &q, typename Acc32<I8>::type &acc) {
  if constexpr (I8)
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(p, q, acc, 0, 0, 0);
  else
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, p),
                                                  __builtin_bit_cast(bf16x8v, q), acc, 0, 0, 0);
}

// tiles of 64 or 128 weight rows and routed rows (mid_product.hip)
void launch_mid_product(const ProdArgs &a, int kind, bool i8, int tile, int R_max, hipStream_t st);
// the tiled kernels (tile_product.hip): 256 routed rows x 256 weight rows a tile
void launch_tile_product(const ProdArgs &a, int kind, bool i8, int R_max, hipStream_t st);

}  // namespace fq
