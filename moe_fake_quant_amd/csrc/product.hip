// Products of routed rows with weight stacks on gfx950: int8 operands with a scale
// for each token and channel, and the gated feed-forward block (gate and up
// projections, SwiGLU and the activation fake-quant in one kernel) with its
// recomputing backward.
//
//   int8   y[r, n] = (sum_k cx[r, k] cw[e, n, k]) * sx[r] * sw[e, n], the sum exact in int32
//   gated  g = x W[f], u = x W[F + f], a = bf16(silu(g) u), aq = FQ_a(a); h = [g, u]
//          stays in registers (fp32)
//   bwd    the same g, u again; da = m_a daq, dh = [da u s (1 + g (1 - s)), da g s]
//          with s = sigmoid(g)
//
// A weight row and an x row are KB bytes with the contraction contiguous, and an
// MFMA operand is 16 bytes a lane for bf16 (16x16x32) and int8 (16x16x64) alike,
// so both types share the loads.
#include "internal.hpp"
#include "product.hpp"
#include "rowq.hpp"
#include "tile.hpp"

namespace fq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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

template <bool I8>
__device__ __forceinline__ void mfma16(const i32x4 &w, const i32x4 &x, i32x4 &acc) {
  if constexpr (I8) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, acc, 0, 0, 0);
  } else {
    acc = __builtin_bit_cast(
        i32x4, __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                   __builtin_bit_cast(bf16x8v, w), __builtin_bit_cast(bf16x8v, x),
                   __builtin_bit_cast(f32x4, acc), 0, 0, 0));
  }
}

// Few rows: the weights' stream bounds it. A block takes 16 output columns of one
// expert and MT * 16 rows; its NW waves share out the contraction in pieces of 256
// bytes, read both operands from global memory straight into MFMA fragments, and
// leave their sums in LDS, where they are added in wave order.
// Grid: (columns / 16, E, row chunks, strided).
constexpr int NW = 8;
template <int KIND, bool I8, int MT>
__global__ __launch_bounds__(NW * 64) void k_rows_product(ProdArgs a) {
  constexpr int NP = KIND == PLAIN ? 1 : 2;   // gate and up
  constexpr int S = NP * MT * 256;            // sums of a block
  __shared__ __attribute__((aligned(16))) int part[NW * S];
  const int e = blockIdx.y, c0 = blockIdx.x * 16;
  const int r_end = a.seg[e + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = (lane >> 4) * 16;
  const ActQ q = load_actq(KIND == PLAIN ? FQ_FMT_NONE : a.afmt, a.ascale);
  const char *wrow[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    wrow[p] = a.w + ((size_t)e * a.N + (size_t)p * a.C + c0 + l16) * a.KB;
  for (int r0 = a.seg[e] + blockIdx.z * (16 * MT); r0 < r_end; r0 += gridDim.z * (16 * MT)) {
    const char *xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      xrow[m] = a.x + (size_t)x_row(a, min(r0 + 16 * m + l16, r_end - 1)) * a.KB;
    i32x4 acc[NP][MT];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[p][m] = i32x4{0, 0, 0, 0};
    // a piece of 256 bytes; the last one may end inside: chunks past the row's end
    // are zero in both operands
    auto piece = [&](uint32_t k0, auto tail_tag) {
      constexpr bool TAIL = decltype(tail_tag)::value;
      i32x4 w[NP][4], x[MT][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t k = k0 + 64 * s + kq;
        const bool in = !TAIL || k < a.KB;
        const uint32_t at = in ? k : 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          w[p][s] = *reinterpret_cast<const i32x4 *>(wrow[p] + at);
          if (!in) w[p][s] = i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          x[m][s] = *reinterpret_cast<const i32x4 *>(xrow[m] + at);
          if (!in) x[m][s] = i32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int m = 0; m < MT; ++m) mfma16<I8>(w[p][s], x[m][s], acc[p][m]);
    };
    uint32_t k0 = 256 * wave;
    for (; k0 + 256 <= a.KB; k0 += 256 * NW) piece(k0, std::false_type{});
    if (k0 < a.KB) piece(k0, std::true_type{});
    // acc[p][m] of this lane: columns c0 + 4 (lane / 16) + v, row r0 + 16 m + lane % 16
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        *reinterpret_cast<i32x4 *>(part + wave * S + (p * MT + m) * 256 + l16 * 16 + (lane >> 4) * 4) =
            acc[p][m];
    __syncthreads();
    for (int i = threadIdx.x; i < S; i += NW * 64) {
      if constexpr (I8) {
        int v = part[i];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += part[w * S + i];
        part[i] = v;
      } else {
        float v = __int_as_float(part[i]);
#pragma unroll
        for (int w = 1; w < NW; ++w) v += __int_as_float(part[w * S + i]);
        part[i] = __float_as_int(v);
      }
    }
    __syncthreads();
    // two lanes a row, 8 columns each
    if (threadIdx.x < 32 * MT) {
      const int j = threadIdx.x >> 1, half = (threadIdx.x & 1) * 8, r = r0 + j;
      const bool live = r < r_end;
      float v[NP][8];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int *src = part + (p * MT + (j >> 4)) * 256 + (j & 15) * 16 + half;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (I8) {
            const size_t n = (size_t)e * a.N + (size_t)p * a.C + c0 + half + k;
            const float sx = a.sx[x_row(a, live ? r : r_end - 1)];
            v[p][k] = ((float)src[k] * sx) * a.sw[a.sw_rows ? n : (size_t)e];
          } else {
            v[p][k] = __int_as_float(src[k]);
          }
        }
      }
      finish8<KIND>(a, q, r, c0 + half, v[0], v[NP - 1], live);
    }
    __syncthreads();
  }
}

}  // namespace

// rows of an expert, were they spread evenly, from which the tiles are taken
constexpr int kTileRows = 64;

template <int KIND, bool I8>
static void launch_product(const ProdArgs &a, int R_max, hipStream_t st) {
  if ((R_max + a.E - 1) / a.E > kTileRows) {
    launch_tile_product(a, KIND, I8, R_max, st);
    return;
  }
  // rows of an expert, were they spread evenly
  const int per = (R_max + a.E - 1) / a.E;
  const int mt = per <= 16 ? 1 : per <= 32 ? 2 : 4;
  int z = (per + 16 * mt - 1) / (16 * mt);
  z = z < 64 ? z : 64;
  const dim3 grid(a.C / 16, a.E, z), block(NW * 64);
  if (mt == 1) hipLaunchKernelGGL((k_rows_product<KIND, I8, 1>), grid, block, 0, st, a);
  else if (mt == 2) hipLaunchKernelGGL((k_rows_product<KIND, I8, 2>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_rows_product<KIND, I8, 4>), grid, block, 0, st, a);
}

static ProdArgs prod_args(const void *x, const int32_t *perm, int topk, const int32_t *seg, fq_shape s,
                          const void *w, int elem, int columns) {
  ProdArgs a{};
  a.w = static_cast<const char *>(w);
  a.x = static_cast<const char *>(x);
  a.perm = perm;
  a.topk = FastDiv((uint32_t)topk);
  a.seg = seg;
  a.E = s.E;
  a.N = s.N;
  a.C = columns;
  a.KB = (uint32_t)s.K * elem;
  return a;
}

void launch_int8_product(const uint8_t *xc, const float *sx, const int32_t *perm, int topk, int R_max,
                         const int32_t *seg, fq_shape s, const fq_stored_w &w, bool gated,
                         uint16_t *out, hipStream_t st) {
  ProdArgs a = prod_args(xc, perm, topk, seg, s, w.codes, 1, gated ? s.N / 2 : s.N);
  a.sx = sx;
  a.sw = w.scale;
  a.sw_rows = w.group != FQ_GROUP_TENSOR;
  a.out = out;
  if (gated) launch_product<GATED, true>(a, R_max, st);
  else launch_product<PLAIN, true>(a, R_max, st);
}

void launch_gated(const uint16_t *daq, const uint16_t *x, const int32_t *perm, int topk, int R_max,
                  const int32_t *seg, fq_shape s, const uint16_t *w, int afmt, const float *ascale,
                  uint16_t *out, uint16_t *aq, hipStream_t st) {
  ProdArgs a = prod_args(x, perm, topk, seg, s, w, 2, s.N / 2);
  a.daq = daq;
  a.afmt = afmt;
  a.ascale = ascale;
  a.out = out;
  a.aq = aq;
  if (daq) launch_product<GATED_BWD, false>(a, R_max, st);
  else launch_product<GATED, false>(a, R_max, st);
}

}  // namespace fq
