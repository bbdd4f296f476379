// Device helpers of the activation passes (gfx950): the activation fake-quant
// of a lane's 8 or 16 elements, SwiGLU, and a block sum of fixed order. Shared
// by the elementwise passes and the kernels that fuse them.
#pragma once

#include "codec.hpp"

namespace fq {

// Per-tensor frozen activation quantizer, resolved once per thread.
struct ActQ {
  int fmt;
  float s;  // s_a (fp8 / int8) or g_a (nvfp4)
  float r;  // 1/s_a
};

__device__ __forceinline__ ActQ load_actq(int fmt, const float *scale) {
  ActQ q;
  q.fmt = fmt;
  q.s = (fmt == FQ_FMT_NONE) ? 1.0f : scale[0];
  q.r = (fmt == FQ_FMT_NONE) ? 1.0f : 1.0f / q.s;
  return q;
}

// 16 consecutive elements along K (one NVFP4 block): values in place, mask bits out.
__device__ __forceinline__ uint32_t act_fq16(const ActQ &q, float *x) {
  uint32_t mask = 0;
  if (q.fmt == FQ_FMT_NONE) return 0xFFFFu;
  if (q.fmt == FQ_FMT_NVFP4 || q.fmt == FQ_FMT_FP8_E4M3) {
    float s = q.s, r = q.r;
    const float mx = q.fmt == FQ_FMT_NVFP4 ? kE2M1Max : kE4M3Max;
    if (q.fmt == FQ_FMT_NVFP4) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(x[j]));
      s = nvfp4_dynamic_scale(amax, q.s);
      if (s == 0.0f) {  // zero block: +0.0, mask 0
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        return 0u;
      }
      r = 1.0f / s;
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float z0 = x[2 * p] * r, z1 = x[2 * p + 1] * r;
      float v0, v1;
      if (q.fmt == FQ_FMT_NVFP4) e2m1_pair(z0, z1, v0, v1);
      else e4m3_pair(clamp448(z0), clamp448(z1), v0, v1);
      mask |= (uint32_t)(fabsf(z0) <= mx) << (2 * p);
      mask |= (uint32_t)(fabsf(z1) <= mx) << (2 * p + 1);
      x[2 * p] = v0 * s;
      x[2 * p + 1] = v1 * s;
    }
    return mask;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    FQElem e = fq_int8(x[j], q.s, q.r);
    x[j] = e.v;
    mask |= (uint32_t)e.m << j;
  }
  return mask;
}

// 8 elements along K, one half of a 16-element block; the other half is on
// lane ^ PARTNER, which must run the same call (NVFP4 takes the block amax over
// both halves, so the result equals act_fq16 on the whole block). Values in
// place, 8 mask bits out.
template <int PARTNER = 1>
__device__ __forceinline__ uint32_t act_fq8_pair(const ActQ &q, float *x) {
  uint32_t mask = 0;
  if (q.fmt == FQ_FMT_NONE) return 0xFFu;
  if (q.fmt == FQ_FMT_NVFP4 || q.fmt == FQ_FMT_FP8_E4M3) {
    float s = q.s, r = q.r;
    const float mx = q.fmt == FQ_FMT_NVFP4 ? kE2M1Max : kE4M3Max;
    if (q.fmt == FQ_FMT_NVFP4) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
      amax = fmaxf(amax, __shfl_xor(amax, PARTNER, 64));
      s = nvfp4_dynamic_scale(amax, q.s);
      if (s == 0.0f) {  // zero block: +0.0, mask 0
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.0f;
        return 0u;
      }
      r = 1.0f / s;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float z0 = x[2 * p] * r, z1 = x[2 * p + 1] * r;
      float v0, v1;
      if (q.fmt == FQ_FMT_NVFP4) e2m1_pair(z0, z1, v0, v1);
      else e4m3_pair(clamp448(z0), clamp448(z1), v0, v1);
      mask |= (uint32_t)(fabsf(z0) <= mx) << (2 * p);
      mask |= (uint32_t)(fabsf(z1) <= mx) << (2 * p + 1);
      x[2 * p] = v0 * s;
      x[2 * p + 1] = v1 * s;
    }
    return mask;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    FQElem e = fq_int8(x[j], q.s, q.r);
    x[j] = e.v;
    mask |= (uint32_t)e.m << j;
  }
  return mask;
}

// 4 elements of a per-tensor format (FP8, INT8 or none): values in place, 4 mask bits out
__device__ __forceinline__ uint32_t act_fq4(const ActQ &q, float *x) {
  if (q.fmt == FQ_FMT_NONE) return 0xFu;
  uint32_t mask = 0;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (q.fmt == FQ_FMT_FP8_E4M3) {
      const float z0 = x[2 * p] * q.r, z1 = x[2 * p + 1] * q.r;
      const f32x2_t v = __builtin_amdgcn_cvt_pk_f32_fp8(
          __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(z0), clamp448(z1), 0, false), false);
      mask |= (uint32_t)(fabsf(z0) <= kE4M3Max) << (2 * p);
      mask |= (uint32_t)(fabsf(z1) <= kE4M3Max) << (2 * p + 1);
      x[2 * p] = v.x * q.s;
      x[2 * p + 1] = v.y * q.s;
    } else {
#pragma unroll
      for (int j = 2 * p; j < 2 * p + 2; ++j) {
        const FQElem e = fq_int8(x[j], q.s, q.r);
        x[j] = e.v;
        mask |= (uint32_t)e.m << j;
      }
    }
  }
  return mask;
}

__device__ __forceinline__ void load16(const bf16x8_t *p, float *x) {
  bf16x8_t a = p[0], b = p[1];
  unpack8(a, x);
  unpack8(b, x + 8);
}
__device__ __forceinline__ void store16(bf16x8_t *p, const float *x) {
  p[0] = pack8(x);
  p[1] = pack8(x + 8);
}

// FP8 / INT8 activation fake-quant of 16 elements that also yields each
// element's straight-through factor dv/ds_a = value(c) - m*z (the factor of a
// learnable per-tensor scale, the same as a weight scale's). Values in place,
// factors to dvds, mask bits returned.
__device__ __forceinline__ uint32_t act_fq16_ds(const ActQ &q, float *x, float *dvds) {
  uint32_t mask = 0;
  if (q.fmt == FQ_FMT_FP8_E4M3) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float z0 = x[2 * p] * q.r, z1 = x[2 * p + 1] * q.r;
      float v0, v1;
      e4m3_pair(clamp448(z0), clamp448(z1), v0, v1);
      const bool m0 = fabsf(z0) <= kE4M3Max, m1 = fabsf(z1) <= kE4M3Max;
      mask |= ((uint32_t)m0 << (2 * p)) | ((uint32_t)m1 << (2 * p + 1));
      dvds[2 * p] = v0 - (m0 ? z0 : 0.0f);
      dvds[2 * p + 1] = v1 - (m1 ? z1 : 0.0f);
      x[2 * p] = v0 * q.s;
      x[2 * p + 1] = v1 * q.s;
    }
    return mask;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    FQElem e = fq_int8(x[j], q.s, q.r);
    x[j] = e.v;
    dvds[j] = e.dvds;
    mask |= (uint32_t)e.m << j;
  }
  return mask;
}

// sigmoid(g) = 1 / (1 + exp(-g)) on the hardware exp and reciprocal (a few
// ulp; 0 and 1 at the extremes). The forward and the backward both call it,
// so the backward sees exactly the forward's A.
__device__ __forceinline__ float sigmoid_hw(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}
// SwiGLU value of 16 elements in fp32, silu(g) = g * sigmoid(g), rounded to
// bf16 (the stored A); sig receives sigmoid(g).
__device__ __forceinline__ void swiglu16(const float *g, const float *u, float *a, float *sig) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    sig[j] = sigmoid_hw(g[j]);
    a[j] = bf16_to_f32(f32_to_bf16((g[j] * sig[j]) * u[j]));
  }
}

// Sum of v over the block, the same in every thread and bitwise reproducible:
// a butterfly inside each wave (both partners of a step add the same two
// values, so every lane ends with the same sum), then the waves in index order.
template <int NT>
__device__ __forceinline__ float block_sum_fixed(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __shared__ float red[NT / 64];
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int k = 1; k < NT / 64; ++k) s += red[k];
  return s;
}

}  // namespace fq
