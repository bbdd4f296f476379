// Arguments of the int8 and gated products, shared by the kernels for few rows
// (product.hip) and the tiled ones (tile_product.hip).
#pragma once

#include "internal.hpp"

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

// the tiled kernels (tile_product.hip): 256 routed rows x 256 weight rows a tile
void launch_tile_product(const ProdArgs &a, int kind, bool i8, int R_max, hipStream_t st);

}  // namespace fq
