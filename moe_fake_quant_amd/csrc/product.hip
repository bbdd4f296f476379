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
#include "tile.hpp"

namespace fq {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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
// expert and MT * 16 rows; its waves share out the contraction in pieces of U * 64
// bytes, read both operands from global memory straight into MFMA fragments, the
// next piece's before this one's are multiplied, and leave their sums in LDS, where
// they are added in wave order. Grid: (columns / 16, E, row chunks, strided).
// Measured, the kernel alone: one int8 row of [4096 x 4096] 8.3 us (2.0 TB/s of weights),
// four gated bf16 rows of [8192 x 2048] 12 us (2.8 TB/s; the fastest 10.9): a block's life is a few
// dependent trips to HBM, which the short stream does not hide. More pieces in
// flight or 4 or 16 waves instead of 8 were not faster.
template <int KIND, bool I8, int MT, int NW>
__global__ __launch_bounds__(NW * 64) void k_rows_product(ProdArgs a) {
  constexpr int NP = KIND == PLAIN ? 1 : 2;   // gate and up
  constexpr int U = MT > 2 ? 2 : 4;
  constexpr int S = NP * MT * 256;            // sums of a block
  __shared__ __attribute__((aligned(16))) int part[NW * S];
  const int e = blockIdx.y, c0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, kq = (lane >> 4) * 16;
  struct Piece {
    i32x4 w[NP][U], x[MT][U];
  };
  const char *wrow[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p)
    wrow[p] = a.w + ((size_t)e * a.N + (size_t)p * a.C + c0 + l16) * a.KB;
  // the last piece may end inside: chunks past the row's end are zero in both operands
  auto load_w = [&](Piece &d, uint32_t k0) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const uint32_t k = k0 + 64 * s + kq;
#pragma unroll
      for (int p = 0; p < NP; ++p)
        d.w[p][s] = k < a.KB ? *reinterpret_cast<const i32x4 *>(wrow[p] + k) : i32x4{0, 0, 0, 0};
    }
  };
  const uint32_t first = U * 64 * wave;
  Piece cur;
  // one expert: its weights are on the way before the row count is known
  if (gridDim.y == 1) load_w(cur, first);
  const int r_end = a.seg[e + 1];
  const ActQ q = load_actq(KIND == PLAIN ? FQ_FMT_NONE : a.afmt, a.ascale);
  for (int r0 = a.seg[e] + blockIdx.z * (16 * MT); r0 < r_end; r0 += gridDim.z * (16 * MT)) {
    const char *xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
      xrow[m] = a.x + (size_t)x_row(a, min(r0 + 16 * m + l16, r_end - 1)) * a.KB;
    auto load_x = [&](Piece &d, uint32_t k0) {
#pragma unroll
      for (int s = 0; s < U; ++s) {
        const uint32_t k = k0 + 64 * s + kq;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          d.x[m][s] = k < a.KB ? *reinterpret_cast<const i32x4 *>(xrow[m] + k) : i32x4{0, 0, 0, 0};
      }
    };
    i32x4 acc[NP][MT];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[p][m] = i32x4{0, 0, 0, 0};
    if (gridDim.y != 1 || r0 != a.seg[e] + blockIdx.z * (16 * MT)) load_w(cur, first);
    load_x(cur, first);
    for (uint32_t k0 = first; k0 < a.KB; k0 += U * 64 * NW) {
      Piece next;
      if (k0 + U * 64 * NW < a.KB) {
        load_w(next, k0 + U * 64 * NW);
        load_x(next, k0 + U * 64 * NW);
      }
#pragma unroll
      for (int s = 0; s < U; ++s)
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int m = 0; m < MT; ++m) mfma16<I8>(cur.w[p][s], cur.x[m][s], acc[p][m]);
      cur = next;
    }
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
        sums8<I8>(a, e, live ? r : r_end - 1, p * a.C + c0 + half, src, v[p]);
      }
      finish8<KIND>(a, q, r, c0 + half, v[0], v[NP - 1], live);
    }
    __syncthreads();
  }
}

}  // namespace

// The form of a call, by the work units that R_max rows spread evenly over the experts
// would give. us of one call on 256 CUs, int8 / gated int8 / gated bf16, its backward:
//   rows an expert      few rows          64 x 64             128 x 128           256 x 256
//   one [4096 x 4096]
//     16                8 / 9 / 15, 15    12 / 12 / 20, 20    17 / 17 / 30, 31    36 / 37 / 66, 69
//     32                10 / 11 / 19, 19  12 / 12 / 20, 20    17 / 17 / 30, 31    36 / 37 / 67, 70
//     48                13 / 15 / 26, 26  12 / 12 / 20, 20    17 / 17 / 31, 32    36 / 37 / 67, 70
//     64                14 / 16 / 26, 27  12 / 12 / 21, 21    17 / 17 / 31, 32    36 / 37 / 67, 71
//     128               24 / 16 / 27, 28  12 / 12 / 21, 21    18 / 18 / 36, 37    40 / 41 / 75, 79
//     512               87 / 55 / 94, 97  17 / 17 / 30, 31    19 / 19 / 33, 36    44 / 46 / 81, 86
//     1024                                29 / 29 / 55, 57    22 / 21 / 37, 40    44 / 46 / 82, 86
//     2048                                55 / 54 / 107, 117  37 / 36 / 66, 72    50 / 49 / 83, 86
//   rows of one expert over short contractions, where the few-row form's stream is over soon
//     [2048 x 2048] 64  7.8 / 9.4 / 15, 15    7.9 / 7.9 / 12, 12
//     [1024 x 1024] 64  4.9 / 6.0 / 8.5, 8.9  5.6 / 5.6 / 7.8, 8.0
//     8 of [256 x 512]  4.0 / 4.9 / 5.9, 6.4  5.4 / 5.4 / 6.2, 6.7  (64 rows each)
//   128 of [1536 x 2048]
//     16            121 / 131 / 211, 227  80 / 79 / 146, 155  86 / 83 / 155, 158  90 / 90 / 162, 170
//     64                                  95 / 92 / 167, 178  94 / 89 / 164, 180  93 / 92 / 202, 214
//     128                                 143 / 140 / 249, 259  120 / 111 / 201, 233  104 / 98 / 200, 217
//     256                                 250 / 245 / 416, 443  190 / 175 / 273, 306  132 / 126 / 215, 237
//   64 of [2048 x 768], 1024 rows         298 / 279 / 411, 503  211 / 179 / 281, 366  154 / 143 / 216, 270
// The rows that are really there are known on the device alone. 32 of [1536 x 2048] with
// room for 512 rows an expert, which the rule gives tiles of 256, with fewer live:
//     256                                 64 / 62 / 106, 114  47 / 46 / 79, 89    37 / 41 / 64, 68
//     128                                 38 / 39 / 66, 68    33 / 32 / 56, 59    37 / 35 / 57, 60
//     64                                  26 / 26 / 51, 50    29 / 29 / 52, 54    34 / 34 / 56, 59
enum Form { kRows, kMid64, kMid128, kTile256 };

static Form pick_form(int kind, int E, int C, uint32_t KB, int R_max) {
  const int64_t cus = device_cus(), per = ((int64_t)R_max + E - 1) / E;
  auto units = [&](int64_t tile) {
    const int64_t cols = kind == PLAIN ? tile : tile / 2;
    return (C + cols - 1) / cols * E * ((per + tile - 1) / tile);
  };
  // blocks of 16 columns and up to 64 rows: two rounds of them at most for up to 32 rows
  // an expert; beyond, one round, and only over rows of 2 KB (gated: 1 KB)
  const int64_t blocks = (int64_t)(C / 16) * E * ((per + 63) / 64);
  const bool few = per <= 32 ? blocks <= 2 * cus
                             : blocks <= cus && KB <= (kind == PLAIN ? 2048u : 1024u);
  if (few) return kRows;
  if (per > 64 && units(256) >= cus) return kTile256;
  if (per > 64 && units(128) * 4 >= cus * 3) return kMid128;
  return kMid64;
}

// Not part of fq.h: the form (0 to 3) that a call takes on the current device, for the
// tests that aim at each of them. kind: 0 plain, 1 gated, 2 its backward.
extern "C" int32_t fq_internal_product_form(int32_t kind, int32_t E, int32_t columns, int32_t row_bytes,
                                            int32_t R_max) {
  return pick_form(kind, E, columns, (uint32_t)row_bytes, R_max);
}

template <int KIND, bool I8>
static void launch_product(const ProdArgs &a, int R_max, hipStream_t st) {
  const Form form = pick_form(KIND, a.E, a.C, a.KB, R_max);
  if (form == kTile256) return launch_tile_product(a, KIND, I8, R_max, st);
  if (form != kRows) return launch_mid_product(a, KIND, I8, form == kMid64 ? 64 : 128, R_max, st);
  const int per = (R_max + a.E - 1) / a.E;
  const int mt = per <= 16 ? 1 : per <= 32 ? 2 : 4;
  int z = (per + 16 * mt - 1) / (16 * mt);
  z = z < 64 ? z : 64;
  const dim3 grid(a.C / 16, a.E, z);
  if (mt == 1) hipLaunchKernelGGL((k_rows_product<KIND, I8, 1, 8>), grid, dim3(512), 0, st, a);
  else if (mt == 2) hipLaunchKernelGGL((k_rows_product<KIND, I8, 2, 8>), grid, dim3(512), 0, st, a);
  else hipLaunchKernelGGL((k_rows_product<KIND, I8, 4, 8>), grid, dim3(512), 0, st, a);
}

static ProdArgs prod_args(const void *x, const int32_t *perm, int topk, const int32_t *seg, fq_shape s,
                          const void *w, int elem, int columns) {
  ProdArgs a{};
  a.w = static_cast<const char *>(w);
  a.x = static_cast<const char *>(x);
  a.perm = perm;
  // direct rows have no topk (a division by any value that the caller left there)
  a.topk = perm ? FastDiv((uint32_t)topk) : FastDiv();
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
