// Activation checkpoints in 8 bits on gfx950: what a layer's backward needs of
// its forward, kept as INT8 or E4M3 codes with one fp32 scale per group of
// elements along a row.
//
// Saved:  s = max(amax * fp32(1/D), 2^-126) per group (D = 127 or 448, the
//         grid's largest value; 1 for an all-zero group), r = 1/s, code =
//         Q(clamp(x * r)). The rounded 1/D moves s by at most one part in
//         2^24, which the clamp absorbs at the group's largest element.
// Loaded: x~ = code * s.
// The floor keeps r finite for groups of subnormals (x~ is then off by at most
// 2^-127). |x - x~| <= s/2 (INT8), resp. half an E4M3 step of x/s times s. A
// group that holds an infinity or NaN stores the scale NaN and codes 0, so
// that it loads as NaN: a step that has diverged stays visible.
//
// The SwiGLU forward saves h in the pass that reads it anyway, and the
// backward decodes it in registers: g~, u~ feed the derivative, and a~ =
// bf16(silu(g~) u~) its activation-FQ mask and, when asked for, FQ_a(a~), the
// down projection's wgrad operand. So neither h [R, 2F] nor FQ_a(A) [R, F]
// lives from the forward to the backward in bf16: 6F bytes per row become
// 2F + 8F/group.
//
// All passes are HBM-bound streams of 16-byte vectors per lane, one per thread as
// in the elementwise passes. Measured: the SwiGLU forward with save 160 us and
// the backward 182 us at 131072 rows of F = 768 (0.81 and 1.01 GB: 5.1 and 5.6
// TB/s; a 1 GiB device copy runs at 5.2), save 23 and load 19 us at 16384 x 2048
// (4.4 and 5.4 TB/s). Fewer VALU operations (med3 clamps) change nothing. The group's
// amax is a max of the bf16 magnitudes as integers (two per instruction, and a
// NaN or infinity is simply the largest), then a butterfly over the group's
// lanes.
#include "actq.hpp"
#include "internal.hpp"

namespace fq {

namespace {

constexpr int kThreads = 256;

inline int grid_for(long work_items) {
  long b = (work_items + kThreads - 1) / kThreads;
  if (b < 1) b = 1;
  if (b > (1 << 22)) b = 1 << 22;
  return (int)b;
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// the larger magnitude bits of two bf16 pairs, half by half
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                __builtin_bit_cast(u16x2, b)));
}

struct Group {
  float s, r;  // r = 0 for a group that is not finite
  bool finite;
};

// Scale of the group that this lane's 8 elements belong to; the group spans
// `lanes` lanes (a power of two, aligned), all of which run the call.
template <int FMT>
__device__ __forceinline__ Group group_scale(const bf16x8_t &v, int lanes) {
  uint32_t m = max_pair(max_pair(v.w[0] & 0x7FFF7FFFu, v.w[1] & 0x7FFF7FFFu),
                        max_pair(v.w[2] & 0x7FFF7FFFu, v.w[3] & 0x7FFF7FFFu));
  for (int o = 1; o < lanes; o <<= 1) m = max_pair(m, (uint32_t)__shfl_xor((int)m, o, 64));
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  Group g;
  g.finite = top < 0x7F80u;
  constexpr float kInvD = FMT == FQ_FMT_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  g.s = fmaxf(bf16_to_f32(top) * kInvD, 0x1p-126f);
  if (top == 0) g.s = 1.0f;
  if (!g.finite) g.s = __uint_as_float(0x7FC00000u);
  g.r = g.finite ? 1.0f / g.s : 0.0f;
  return g;
}

// the 8 codes of a lane, element j in byte j
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float *x, const Group &g) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float *p = x + 4 * h;
    if (FMT == FQ_FMT_INT8) {
      // z + 1.5 * 2^23 rounds z to an integer (ties to even); its two's
      // complement is the sum's low byte
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = __float_as_uint(fminf(fmaxf(p[j] * g.r, -128.0f), 127.0f) + 12582912.0f);
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
      w[h] = lo | hi;
    } else {
      float v0, v1;
      const uint32_t lo = e4m3_pair(clamp448(p[0] * g.r), clamp448(p[1] * g.r), v0, v1);
      const uint32_t hi = e4m3_pair(clamp448(p[2] * g.r), clamp448(p[3] * g.r), v0, v1);
      w[h] = lo | (hi << 16);
    }
    if (!g.finite) w[h] = 0u;
  }
  return make_uint2(w[0], w[1]);
}

// the 4 values of one word of codes
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float s, float *x) {
  if (FMT == FQ_FMT_INT8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = (float)((int)(w << (24 - 8 * j)) >> 24) * s;
  } else {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    x[0] = lo.x * s;
    x[1] = lo.y * s;
    x[2] = hi.x * s;
    x[3] = hi.y * s;
  }
}

// number of vectors to process: all, or those of the first n_rows[0] rows
__device__ __forceinline__ uint32_t live_vecs(uint32_t max_vec, const int32_t *n_rows,
                                              uint32_t vpr) {
  return n_rows ? (uint32_t)min((uint64_t)n_rows[0] * vpr, (uint64_t)max_vec) : max_vec;
}

// x [rows, K] -> codes [rows, K], scale [rows, K / group]. Groups lie whole in
// a row, so vector c belongs to group c >> lg (2^lg lanes per group). The grid
// stride and the vector count are multiples of the group's lanes.
template <int FMT>
__global__ __launch_bounds__(kThreads) void k_ckpt_save(const bf16x8_t *__restrict__ x,
                                                        uint32_t max_vec,
                                                        const int32_t *__restrict__ n_rows,
                                                        uint32_t vpr, int lg,
                                                        uint2 *__restrict__ codes,
                                                        float *__restrict__ scale) {
  const uint32_t nvec = live_vecs(max_vec, n_rows, vpr);
  for (uint32_t c = blockIdx.x * kThreads + threadIdx.x; c < nvec; c += gridDim.x * kThreads) {
    const bf16x8_t v = x[c];
    const Group g = group_scale<FMT>(v, 1 << lg);
    float f[8];
    unpack8(v, f);
    codes[c] = encode8<FMT>(f, g);
    if ((c & ((1u << lg) - 1u)) == 0) scale[c >> lg] = g.s;
  }
}

// codes, scale -> x; 16 elements per lane (they share a group)
template <int FMT>
__global__ __launch_bounds__(kThreads) void k_ckpt_load(const uint4 *__restrict__ codes,
                                                        const float *__restrict__ scale,
                                                        uint32_t max_vec,
                                                        const int32_t *__restrict__ n_rows,
                                                        uint32_t vpr, int lg,
                                                        bf16x8_t *__restrict__ x) {
  const uint32_t nvec = live_vecs(max_vec, n_rows, vpr);
  for (uint32_t c = blockIdx.x * kThreads + threadIdx.x; c < nvec; c += gridDim.x * kThreads) {
    const uint4 w = codes[c];
    const float s = scale[c >> lg];
    float f[16];
    decode4<FMT>(w.x, s, f);
    decode4<FMT>(w.y, s, f + 4);
    decode4<FMT>(w.z, s, f + 8);
    decode4<FMT>(w.w, s, f + 12);
    store16(x + 2 * (size_t)c, f);
  }
}

// k_swiglu_actfq that also saves h: each lane holds 8 gate and 8 up elements,
// a 16-block of the activation FQ spans a lane pair, a group 2^lg lanes of
// either half (group divides F, so no group crosses from gate to up).
template <int FMT>
__global__ __launch_bounds__(kThreads) void k_swiglu_actfq_ckpt(
    const bf16x8_t *__restrict__ h, FastDiv vec_per_row, uint32_t max_vec,
    const int32_t *__restrict__ n_rows, int lg, int afmt, const float *__restrict__ ascale,
    bf16x8_t *__restrict__ a_out, bf16x8_t *__restrict__ aq_out, uint2 *__restrict__ codes,
    float *__restrict__ scale) {
  const ActQ q = load_actq(afmt, ascale);
  const uint32_t vpr = vec_per_row.d;  // F / 8
  const uint32_t nvec = live_vecs(max_vec, n_rows, vpr);
  for (uint32_t c = blockIdx.x * kThreads + threadIdx.x; c < nvec; c += gridDim.x * kThreads) {
    const uint32_t r = vec_per_row.div(c);
    const uint32_t cc = c - r * vpr;
    const size_t ig = (size_t)r * 2 * vpr + cc, iu = ig + vpr;
    const bf16x8_t vg = h[ig], vu = h[iu];
    float g[8], u[8], a[8];
    unpack8(vg, g);
    unpack8(vu, u);
    const Group sg = group_scale<FMT>(vg, 1 << lg), su = group_scale<FMT>(vu, 1 << lg);
    codes[ig] = encode8<FMT>(g, sg);
    codes[iu] = encode8<FMT>(u, su);
    if ((cc & ((1u << lg) - 1u)) == 0) {
      scale[ig >> lg] = sg.s;
      scale[iu >> lg] = su.s;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a[j] = bf16_to_f32(f32_to_bf16((g[j] * sigmoid_hw(g[j])) * u[j]));
    if (a_out) a_out[c] = pack8(a);
    act_fq8_pair(q, a);
    aq_out[c] = pack8(a);
  }
}

// k_swiglu_bwd from the saved h: 16 elements per lane and half, each within
// one group. aq_out (may be NULL): FQ_a(a~). DS: the block's share of dS_a.
template <int FMT, bool DS>
__global__ __launch_bounds__(kThreads) void k_swiglu_bwd_ckpt(
    const bf16x8_t *__restrict__ daq, const uint4 *__restrict__ codes,
    const float *__restrict__ scale, FastDiv chunks_per_row, uint32_t max_chunks,
    const int32_t *__restrict__ n_rows, int lg, int afmt, const float *__restrict__ ascale,
    bf16x8_t *__restrict__ dh, bf16x8_t *__restrict__ aq_out, float *__restrict__ ds_part) {
  const ActQ q = load_actq(afmt, ascale);
  const uint32_t cpr = chunks_per_row.d;  // F / 16
  const uint32_t nchunk = live_vecs(max_chunks, n_rows, cpr);
  float part = 0.0f;
  for (uint32_t c = blockIdx.x * kThreads + threadIdx.x; c < nchunk; c += gridDim.x * kThreads) {
    const uint32_t r = chunks_per_row.div(c);
    const uint32_t cc = c - r * cpr;
    const size_t ig = (size_t)r * 2 * cpr + cc, iu = ig + cpr;
    const uint4 wg = codes[ig], wu = codes[iu];
    const float sg = scale[ig >> lg], su = scale[iu >> lg];
    float d[16];
    load16(daq + 2 * (size_t)c, d);
    float g[16], u[16], a[16], sig[16];
    decode4<FMT>(wg.x, sg, g);
    decode4<FMT>(wg.y, sg, g + 4);
    decode4<FMT>(wg.z, sg, g + 8);
    decode4<FMT>(wg.w, sg, g + 12);
    decode4<FMT>(wu.x, su, u);
    decode4<FMT>(wu.y, su, u + 4);
    decode4<FMT>(wu.z, su, u + 8);
    decode4<FMT>(wu.w, su, u + 12);
    swiglu16(g, u, a, sig);
    uint32_t m;
    if (DS) {
      float dv[16];
      m = act_fq16_ds(q, a, dv);
#pragma unroll
      for (int j = 0; j < 16; ++j) part = fmaf(d[j], dv[j], part);
    } else {
      m = act_fq16(q, a);
    }
    if (aq_out) store16(aq_out + 2 * (size_t)c, a);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float da = ((m >> j) & 1u) ? d[j] : 0.0f;
      const float gj = g[j], s = sig[j];
      g[j] = da * u[j] * s * (1.0f + gj * (1.0f - s));
      u[j] = da * gj * s;
    }
    store16(dh + 2 * ig, g);
    store16(dh + 2 * iu, u);
  }
  if (DS) {
    part = block_sum_fixed<kThreads>(part);
    if (threadIdx.x == 0) ds_part[blockIdx.x] = part;
  }
}

int log2i(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

}  // namespace

void launch_ckpt_save(const uint16_t *x, int rows, int K, const int32_t *n_rows, int fmt, int group,
                      uint8_t *codes, float *scale, hipStream_t st) {
  const uint32_t nvec = (uint32_t)((size_t)rows * K / 8);
  if (!nvec) return;
  const dim3 grid(grid_for(nvec)), block(kThreads);
  auto xv = reinterpret_cast<const bf16x8_t *>(x);
  auto cv = reinterpret_cast<uint2 *>(codes);
  const int lg = log2i(group / 8);
  if (fmt == FQ_FMT_INT8)
    hipLaunchKernelGGL(k_ckpt_save<FQ_FMT_INT8>, grid, block, 0, st, xv, nvec, n_rows,
                       (uint32_t)K / 8, lg, cv, scale);
  else
    hipLaunchKernelGGL(k_ckpt_save<FQ_FMT_FP8_E4M3>, grid, block, 0, st, xv, nvec, n_rows,
                       (uint32_t)K / 8, lg, cv, scale);
}

void launch_ckpt_load(const uint8_t *codes, const float *scale, int rows, int K,
                      const int32_t *n_rows, int fmt, int group, uint16_t *x, hipStream_t st) {
  const uint32_t nvec = (uint32_t)((size_t)rows * K / 16);
  if (!nvec) return;
  const dim3 grid(grid_for(nvec)), block(kThreads);
  auto xv = reinterpret_cast<bf16x8_t *>(x);
  auto cv = reinterpret_cast<const uint4 *>(codes);
  const int lg = log2i(group / 16);
  if (fmt == FQ_FMT_INT8)
    hipLaunchKernelGGL(k_ckpt_load<FQ_FMT_INT8>, grid, block, 0, st, cv, scale, nvec, n_rows,
                       (uint32_t)K / 16, lg, xv);
  else
    hipLaunchKernelGGL(k_ckpt_load<FQ_FMT_FP8_E4M3>, grid, block, 0, st, cv, scale, nvec, n_rows,
                       (uint32_t)K / 16, lg, xv);
}

void launch_swiglu_actfq_ckpt(const uint16_t *h, int R_max, const int32_t *n_rows, int F, int afmt,
                              const float *ascale, int fmt, int group, uint16_t *a, uint16_t *aq,
                              uint8_t *codes, float *scale, hipStream_t st) {
  const uint32_t nvec = (uint32_t)((size_t)R_max * F / 8);
  if (!nvec) return;
  const dim3 grid(grid_for(nvec)), block(kThreads);
  auto hv = reinterpret_cast<const bf16x8_t *>(h);
  auto av = reinterpret_cast<bf16x8_t *>(a);
  auto qv = reinterpret_cast<bf16x8_t *>(aq);
  auto cv = reinterpret_cast<uint2 *>(codes);
  const int lg = log2i(group / 8);
  if (fmt == FQ_FMT_INT8)
    hipLaunchKernelGGL(k_swiglu_actfq_ckpt<FQ_FMT_INT8>, grid, block, 0, st, hv, FastDiv(F / 8),
                       nvec, n_rows, lg, afmt, ascale, av, qv, cv, scale);
  else
    hipLaunchKernelGGL(k_swiglu_actfq_ckpt<FQ_FMT_FP8_E4M3>, grid, block, 0, st, hv, FastDiv(F / 8),
                       nvec, n_rows, lg, afmt, ascale, av, qv, cv, scale);
}

void launch_swiglu_bwd_ckpt(const uint16_t *daq, const uint8_t *codes, const float *scale,
                            int R_max, const int32_t *n_rows, int F, int fmt, int group, int afmt,
                            const float *ascale, uint16_t *dh, uint16_t *aq, float *dscale_a,
                            float *part, hipStream_t st) {
  const uint32_t nchunk = (uint32_t)((size_t)R_max * F / 16);
  const dim3 grid(grid_for(nchunk)), block(kThreads);
  auto dq = reinterpret_cast<const bf16x8_t *>(daq);
  auto cv = reinterpret_cast<const uint4 *>(codes);
  auto dv = reinterpret_cast<bf16x8_t *>(dh);
  auto qv = reinterpret_cast<bf16x8_t *>(aq);
  const int lg = log2i(group / 16);
#define FQ_BWD(FMT, DS)                                                                            \
  hipLaunchKernelGGL((k_swiglu_bwd_ckpt<FMT, DS>), grid, block, 0, st, dq, cv, scale,              \
                     FastDiv(F / 16), nchunk, n_rows, lg, afmt, ascale, dv, qv, part)
  if (nchunk) {
    if (fmt == FQ_FMT_INT8) {
      if (dscale_a) FQ_BWD(FQ_FMT_INT8, true);
      else FQ_BWD(FQ_FMT_INT8, false);
    } else {
      if (dscale_a) FQ_BWD(FQ_FMT_FP8_E4M3, true);
      else FQ_BWD(FQ_FMT_FP8_E4M3, false);
    }
  }
#undef FQ_BWD
  if (dscale_a) launch_sum_partials(part, nchunk ? grid.x : 0u, dscale_a, st);
}

}  // namespace fq
