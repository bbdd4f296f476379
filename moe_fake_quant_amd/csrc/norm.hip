// Norms before and after a block, fused with the block's gate and residual scale,
// and their backward (gfx950).
//
//   p = b * rb * w_post       rb = 1 / sqrt(mean(b^2) + eps)   (w_post NULL: p = b)
//   y = x + alpha * gate_t * p
//   n = y * ry * w_pre        ry = 1 / sqrt(mean(y^2) + eps)
// n leaves as bf16 or as int8 codes with one scale a token (the operand of the
// int8 product). n is formed from the unrounded y.
// Backward, from the stored y, with v = dn * w_pre and q = alpha * gate_t:
//   gy = dy + ry * (v - (y ry) * mean(v y) ry)             -> dx
//   dw_pre = sum_t dn y ry
//   S = sum_h gy b w_post     dgate = alpha rb S
//   db = q rb (gy w_post - (b rb) rb S / H) (w_post NULL: db = q gy)
//   dw_post = sum_t q gy b rb
// so one pass takes three row sums (y^2, v y, b^2) and, from registers, a fourth (S).
//
// All passes are HBM streams: a row stays in registers between its sums and its
// outputs, so every tensor is read once and written once. Measured with a device copy
// at 5.2 TB/s: the forward over 16384 x 2048 52 us (5.1 TB/s); the backward over 8191 x
// 2048 44 us without the weights' gradients (4.6 TB/s), with them 49 us (4.1 TB/s, without
// the block sums, 17 MB) and 5 us for the kernel that adds those in block order. The vector
// units are busy 35 to 41 % of the time (46 instructions an element): the backward waits
// for HBM, since a block's next row is asked for after the row before has been stored.
#include <type_traits>

#include "internal.hpp"
#include "rowq.hpp"

namespace fq {

namespace {

struct NormArgs {
  const bf16x8_t *x, *b;  // b may be NULL
  const float *gate;      // [T] or NULL
  const bf16x8_t *w_post, *w_pre;
  float alpha, eps, inv_h;
  int T, nv;  // rows, vectors of 8 a row
  bf16x8_t *y, *n;
  uint2 *codes;
  float *scale;
  // backward (x is the stored y)
  const bf16x8_t *dy, *dn;
  bf16x8_t *dx, *db;
  float *dgate;
  float *part_post, *part_pre;  // [grid, H] block sums of dw_post, dw_pre
};

template <int WPR, int VPT>
__global__ __launch_bounds__(kRowThreads<WPR>) void k_norm_fwd(NormArgs a) {
  __shared__ float red[3 * WPR];
  const int lane = threadIdx.x & (WPR * 64 - 1);
  const uint32_t t = grid_row<WPR>();
  if (t >= (uint32_t)a.T) return;  // whole rows: with WPR > 1 the whole block
  const size_t row = (size_t)t * a.nv;
  bf16x8_t vx[VPT], vb[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * WPR * 64;
    if (c < a.nv) {
      vx[i] = a.x[row + c];
      if (a.b) vb[i] = a.b[row + c];
    } else {
      vx[i] = vb[i] = bf16x8_t{{0, 0, 0, 0}};
    }
  }
  float y[VPT][8];
  float q = a.alpha;
  if (a.b && a.gate) q *= a.gate[t];
  if (a.b && a.w_post) {
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8(vb[i], y[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
    }
    row_sum<WPR>(s, red);
    const float rb = rsqrtf(s[0] * a.inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = lane + i * WPR * 64;
      float w[8], x[8];
      if (c < a.nv) unpack8(a.w_post[c], w);
      unpack8(vx[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = c < a.nv ? fmaf(q, (y[i][j] * rb) * w[j], x[j]) : 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8(vx[i], y[i]);
      if (a.b) {
        float b[8];
        unpack8(vb[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] = fmaf(q, b[j], y[i][j]);
      }
    }
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = lane + i * WPR * 64;
      if (c < a.nv) a.y[row + c] = pack8(y[i]);
    }
  }
  if (!a.w_pre) return;
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] = fmaf(y[i][j], y[i][j], s[0]);
  row_sum<WPR>(s, red + WPR);
  const float ry = rsqrtf(s[0] * a.inv_h + a.eps);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * WPR * 64;
    if (c < a.nv) {
      float w[8];
      unpack8(a.w_pre[c], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[i][j] = (y[i][j] * ry) * w[j];
        top = max(top, __float_as_uint(y[i][j]) & 0x7FFFFFFFu);
      }
      if (a.n) a.n[row + c] = pack8(y[i]);
    }
  }
  if (!a.codes) return;
  const TokenScale ts = token_scale(row_max_bits<WPR>(top, reinterpret_cast<uint32_t *>(red + 2 * WPR)));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * WPR * 64;
    if (c < a.nv) a.codes[row + c] = token_codes8(y[i], ts);
  }
  if (lane == 0) a.scale[t] = ts.s;
}

// Rows t = block's first, + grid stride. DW: the block keeps its rows' sums of
// dw_post and dw_pre in registers (each lane owns its columns) and leaves them,
// added over the block's waves in order, in part_*[block, H].
template <int WPR, int VPT, bool DW>
__global__ __launch_bounds__(kRowThreads<WPR>) void k_norm_bwd(NormArgs a) {
  __shared__ float red[2][4 * WPR];
  constexpr int RPB = kBlockRows<WPR>;
  const int lane = threadIdx.x & (WPR * 64 - 1);
  const int sub = threadIdx.x / (WPR * 64);
  float ap[DW ? VPT : 1][8] = {}, aq[DW ? VPT : 1][8] = {};
  int flip = 0;
  for (int t = blockIdx.x * RPB + sub; t < a.T; t += gridDim.x * RPB, flip ^= 1) {
    const size_t row = (size_t)t * a.nv;
    bf16x8_t vy[VPT], vb[VPT], vdn[VPT], vdy[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = lane + i * WPR * 64;
      vy[i] = vb[i] = vdn[i] = vdy[i] = bf16x8_t{{0, 0, 0, 0}};
      if (c < a.nv) {
        if (a.dn) {
          vy[i] = a.x[row + c];
          vdn[i] = a.dn[row + c];
        }
        if (a.b) vb[i] = a.b[row + c];
        if (a.dy) vdy[i] = a.dy[row + c];
      }
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = lane + i * WPR * 64;
      float y[8], dn[8], b[8], w[8];
      unpack8(vy[i], y);
      unpack8(vdn[i], dn);
      unpack8(vb[i], b);
      if (a.dn && c < a.nv) unpack8(a.w_pre[c], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] = fmaf(y[j], y[j], s[0]);
        if (a.dn && c < a.nv) s[1] = fmaf(dn[j] * w[j], y[j], s[1]);
        s[2] = fmaf(b[j], b[j], s[2]);
      }
    }
    row_sum<WPR>(s, red[flip]);
    const float ry = a.dn ? rsqrtf(s[0] * a.inv_h + a.eps) : 0.0f;
    // mean(v y) ry: with y ry beside it no power of the root is formed, which would leave
    // fp32's range before the row's sum of squares does (rows about 1e15 large, eps below 1e-26)
    const float my = ry * (s[1] * a.inv_h);
    const float rb = a.w_post ? rsqrtf(s[2] * a.inv_h + a.eps) : 1.0f;
    const float q = a.b ? a.alpha * (a.gate ? a.gate[t] : 1.0f) : 0.0f;
    float gy[VPT][8];
    float sb[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = lane + i * WPR * 64;
      float y[8], dn[8], b[8], w[8];
      unpack8(vdy[i], gy[i]);
      if (c < a.nv) {
        if (a.dn) {
          unpack8(vy[i], y);
          unpack8(vdn[i], dn);
          unpack8(a.w_pre[c], w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float yr = y[j] * ry;
            gy[i][j] = fmaf(ry, fmaf(-my, yr, dn[j] * w[j]), gy[i][j]);
            if (DW) ap[i][j] = fmaf(dn[j], yr, ap[i][j]);
          }
        }
        if (a.dx) a.dx[row + c] = pack8(gy[i]);
        if (a.b) {
          unpack8(vb[i], b);
          if (a.w_post) unpack8(a.w_post[c], w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float g = a.w_post ? gy[i][j] * w[j] : gy[i][j];
            sb[0] = fmaf(g, b[j], sb[0]);
            if (DW && a.w_post) aq[i][j] = fmaf(q * gy[i][j], b[j] * rb, aq[i][j]);
          }
        }
      }
    }
    if (!a.b) continue;
    row_sum<WPR>(sb, red[flip] + 3 * WPR);
    if (a.dgate && lane == 0) a.dgate[t] = a.alpha * (rb * sb[0]);
    if (a.db) {
      const float mb = rb * (sb[0] * a.inv_h);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * WPR * 64;
        if (c < a.nv) {
          float b[8], w[8], o[8];
          unpack8(vb[i], b);
          if (a.w_post) unpack8(a.w_post[c], w);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = a.w_post ? (q * rb) * fmaf(-mb, b[j] * rb, gy[i][j] * w[j]) : q * gy[i][j];
          a.db[row + c] = pack8(o);
        }
      }
    }
  }
  if constexpr (DW) {
    extern __shared__ float acc[];  // [RPB][H], WPR = 1 only
    const int H = a.nv * 8;
    for (int which = 0; which < 2; ++which) {
      float *out = which ? a.part_post : a.part_pre;
      if (!out) continue;  // the same in every thread
      out += (size_t)blockIdx.x * H;
      if constexpr (RPB > 1) __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * WPR * 64;
        if (c < a.nv) {
          float *d = RPB > 1 ? acc + sub * H + c * 8 : out + c * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = which ? aq[i][j] : ap[i][j];
        }
      }
      if constexpr (RPB > 1) {
        __syncthreads();
        for (int h = threadIdx.x; h < H; h += kRowThreads<WPR>)
          out[h] = ((acc[h] + acc[H + h]) + acc[2 * H + h]) + acc[3 * H + h];
      }
    }
  }
}

// out[h] = sum over the blocks of part[block, h]: 32 columns a block, 32 groups of
// blocks summed side by side and added in group order
__global__ __launch_bounds__(1024) void k_norm_dw(const float *__restrict__ part_post,
                                                  const float *__restrict__ part_pre, int nb, int H,
                                                  float *__restrict__ dw_post,
                                                  float *__restrict__ dw_pre) {
  __shared__ float s[32][32];
  const float *part = blockIdx.y ? part_post : part_pre;
  float *out = blockIdx.y ? dw_post : dw_pre;
  if (!out) return;
  const int g = threadIdx.x >> 5, c = threadIdx.x & 31, h = blockIdx.x * 32 + c;
  const int per = (nb + 31) / 32, b1 = min(nb, (g + 1) * per);
  float v = 0.0f;
  if (h < H) {
#pragma unroll 8
    for (int b = g * per; b < b1; ++b) v += part[(size_t)b * H + h];
  }
  s[g][c] = v;
  __syncthreads();
  if (g == 0 && h < H) {
    for (int k = 1; k < 32; ++k) v += s[k][c];
    out[h] = v;
  }
}

// x [rows, K] -> codes [rows, K] with a scale for each row; rows too long for the
// registers are read twice. An HBM stream: 131072 rows of 768 in 59 us (5.1 TB/s
// with the codes; the fastest 54), 2048 rows of 4096 in 6.9.
template <int WPR, int VPT>
__global__ __launch_bounds__(kRowThreads<WPR>) void k_quantize_tokens(const bf16x8_t *__restrict__ x,
                                                                 int rows, int nv,
                                                                 const int32_t *__restrict__ n_rows,
                                                                 uint2 *__restrict__ codes,
                                                                 float *__restrict__ scale) {
  __shared__ uint32_t red[WPR];
  if (n_rows) rows = min(rows, n_rows[0]);
  const int lane = threadIdx.x & (WPR * 64 - 1);
  const uint32_t t = grid_row<WPR>();
  if ((int64_t)t >= rows) return;  // (n_rows may be negative)
  const size_t row = (size_t)t * nv;
  bf16x8_t v[VPT];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * WPR * 64;
    if (c < nv) {
      v[i] = x[row + c];
      top = max(top, max_bits8(v[i]));
    }
  }
  for (int c = lane + VPT * WPR * 64; c < nv; c += WPR * 64) top = max(top, max_bits8(x[row + c]));
  const TokenScale ts = token_scale(row_max_bits<WPR>(top, red));
  float f[8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * WPR * 64;
    if (c < nv) {
      unpack8(v[i], f);
      codes[row + c] = token_codes8(f, ts);
    }
  }
  for (int c = lane + VPT * WPR * 64; c < nv; c += WPR * 64) {
    unpack8(x[row + c], f);
    codes[row + c] = token_codes8(f, ts);
  }
  if (lane == 0) scale[t] = ts.s;
}

}  // namespace

// Waves a row and vectors a lane for rows of H. One vector a lane while the block has
// the waves for it: more rows are then in different phases at a time (the backward with
// weight gradients over 16384 rows of 4096: 174 us, with four waves of up to four vectors
// 315; 8191 rows of 2048: 54 us, one wave of four vectors 70). 1024 threads leave the
// backward too few registers (rows of 8192: 16 waves of one vector spill).
template <class F>
static void with_row_form(int H, F f) {
  using std::integral_constant;
  if (H <= kNormWaveRow) f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (H <= 2048) f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (H <= 4096) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (H <= 8192) f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  else f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
}

// Blocks of the backward with weight gradients: enough rows in flight to stream,
// few enough that the block sums stay small beside the tensors.
static int norm_bwd_blocks(int T, int H) {
  const int rpb = H <= kNormWaveRow ? 4 : 1;
  const int need = (T + rpb - 1) / rpb, most = H <= 2048 ? 1024 : 512;
  return need < most ? need : most;
}
size_t norm_ws_bytes(int T, int H) {
  return T > 0 ? (size_t)2 * norm_bwd_blocks(T, H) * H * 4 : 0;
}

static NormArgs norm_args(const uint16_t *x, const uint16_t *b, const float *gate, float alpha,
                          const uint16_t *w_post, const uint16_t *w_pre, float eps, int T, int H) {
  NormArgs a{};
  a.x = reinterpret_cast<const bf16x8_t *>(x);
  a.b = reinterpret_cast<const bf16x8_t *>(b);
  a.gate = gate;
  a.alpha = alpha;
  a.w_post = reinterpret_cast<const bf16x8_t *>(w_post);
  a.w_pre = reinterpret_cast<const bf16x8_t *>(w_pre);
  a.eps = eps;
  a.inv_h = 1.0f / (float)H;
  a.T = T;
  a.nv = H / 8;
  return a;
}

void launch_norm_fwd(const uint16_t *x, const uint16_t *b, const float *gate, float alpha,
                     const uint16_t *w_post, const uint16_t *w_pre, float eps, int T, int H,
                     uint16_t *y, uint16_t *n, uint8_t *codes, float *scale, hipStream_t st) {
  NormArgs a = norm_args(x, b, gate, alpha, w_post, w_pre, eps, T, H);
  a.y = reinterpret_cast<bf16x8_t *>(y);
  a.n = reinterpret_cast<bf16x8_t *>(n);
  a.codes = reinterpret_cast<uint2 *>(codes);
  a.scale = scale;
  with_row_form(H, [&](auto wpr, auto vpt) {
    constexpr int W = decltype(wpr)::value, V = decltype(vpt)::value;
    hipLaunchKernelGGL((k_norm_fwd<W, V>), block_grid(ceil_div(T, kBlockRows<W>)), dim3(kRowThreads<W>), 0,
                       st, a);
  });
}

void launch_norm_bwd(const uint16_t *dy, const uint16_t *dn, const uint16_t *y, const uint16_t *b,
                     const float *gate, float alpha, const uint16_t *w_post, const uint16_t *w_pre,
                     float eps, int T, int H, uint16_t *dx, uint16_t *db, float *dgate,
                     float *dw_post, float *dw_pre, float *ws, hipStream_t st) {
  NormArgs a = norm_args(y, b, gate, alpha, w_post, w_pre, eps, T, H);
  a.dy = reinterpret_cast<const bf16x8_t *>(dy);
  a.dn = reinterpret_cast<const bf16x8_t *>(dn);
  a.dx = reinterpret_cast<bf16x8_t *>(dx);
  a.db = reinterpret_cast<bf16x8_t *>(db);
  a.dgate = dgate;
  if (T == 0) {  // no rows: the weights' gradients are zero
    if (dw_pre) launch_fill_u32(reinterpret_cast<uint32_t *>(dw_pre), 0, H, st);
    if (dw_post) launch_fill_u32(reinterpret_cast<uint32_t *>(dw_post), 0, H, st);
    return;
  }
  const bool dw = dw_post || dw_pre;
  const int nb = norm_bwd_blocks(T, H);
  if (dw) {
    a.part_pre = dw_pre ? ws : nullptr;
    a.part_post = dw_post ? ws + (size_t)nb * H : nullptr;
  }
  with_row_form(H, [&](auto wpr, auto vpt) {
    constexpr int W = decltype(wpr)::value, V = decltype(vpt)::value;
    const dim3 threads(kRowThreads<W>);
    if (dw)
      hipLaunchKernelGGL((k_norm_bwd<W, V, true>), dim3(nb), threads, W == 1 ? (size_t)4 * H * 4 : 0, st,
                         a);
    else
      // (the kernel strides over the rows: along x alone)
      hipLaunchKernelGGL((k_norm_bwd<W, V, false>), dim3(block_grid(ceil_div(T, kBlockRows<W>)).x), threads, 0,
                         st, a);
  });
  if (dw)
    hipLaunchKernelGGL(k_norm_dw, dim3((H + 31) / 32, 2), dim3(1024), 0, st, a.part_post, a.part_pre, nb, H,
                       dw_post, dw_pre);
}

void launch_quantize_tokens(const uint16_t *x, int rows, int K, const int32_t *n_rows, uint8_t *codes,
                            float *scale, hipStream_t st) {
  const bf16x8_t *v = reinterpret_cast<const bf16x8_t *>(x);
  uint2 *c = reinterpret_cast<uint2 *>(codes);
  if (K <= 1024)
    hipLaunchKernelGGL((k_quantize_tokens<1, 2>), block_grid(ceil_div(rows, 4)), dim3(256), 0, st, v, rows,
                       K / 8, n_rows, c, scale);
  else
    hipLaunchKernelGGL((k_quantize_tokens<4, 4>), block_grid(rows), dim3(256), 0, st, v, rows, K / 8, n_rows,
                       c, scale);
}

}  // namespace fq
