// One MoE layer for a few tokens (T <= 128) over the stored form of its
// weights, in two kernels on gfx950: the serving counterpart of the grouped
// GEMM path, without a decoded copy of the stacks, a permutation or a gather.
//
//   k_tok_gate_up  h = W_gu[e] FQ_a1(x),  a = silu(h_g) h_u,  A = FQ_a2(a)
//   k_tok_down     out[t] = bf16(sum_j p[t,j] W_d[e_tj] A[t,j])
//
// What bounds it: the codes of the distinct experts of the batch are read once
// and everything else is small, so the floor is the weight stream from HBM;
// next come the VALU operations that turn 4-bit codes into MFMA operands.
//
// Operands are exact. A weight's grid value (E4M3, int8, int4 minus zero
// point, E2M1 times its E4M3 block scale: at most 8 significant bits) is a
// bf16 number, and so is an activation's; the fp32 scales that are constant
// over a contraction (per channel, per tensor, per 128-group, the NVFP4 tensor
// scale, s_a) multiply the fp32 sums instead. Only weight groups smaller than
// a chunk (see Fmt) fold their scale into the operand, which rounds it to the
// bf16 value the training forward uses, and A without an activation format is
// stored as bf16, as in the training forward. h stays in fp32.
//
// Contraction: v_mfma_f32_16x16x32_bf16 with 16 weight rows as the row operand
// and up to 16 tokens as columns. A lane loads 16 bytes of codes of its row
// at once (32 four-bit codes) and feeds them to consecutive MFMAs, so the
// contraction order is permuted, alike for both operands: a wave's load covers
// 16 rows x 64 contiguous bytes.
//
// Sums are taken in a fixed order (no float atomics): the same call gives the
// same bits. A token that names an expert twice counts as one pair with the
// summed weight.
#include "actq.hpp"
#include "internal.hpp"

namespace fq {

namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8v;
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kNT = 512;        // threads per block
constexpr int kWaves = kNT / 64;

// Where a weight scale enters.
enum ScaleMode {
  kEnd = 0,   // constant along the row (per channel / per tensor, or none): the finished sum
  kPost = 1,  // group a multiple of a chunk: the chunk's sum
  kPre = 2    // smaller groups, NVFP4's E4M3 block scale: the operand
};

// Codes a lane takes from one 16-byte load (kSeg), and the chunk of the
// contraction that the four lane groups of a wave cover with them.
template <int FMT>
struct Fmt {
  static constexpr int kSeg = FMT == FQ_FMT_NONE ? 8
                              : FMT == FQ_FMT_INT8 || FMT == FQ_FMT_FP8_E4M3 ? 16 : 32;
  static constexpr int kChunk = 4 * kSeg;
  static constexpr int kSteps = kSeg / 8;  // MFMAs per chunk
  static constexpr bool k4bit = FMT == FQ_FMT_INT4 || FMT == FQ_FMT_NVFP4;
};

struct TokStack {  // one projection's stored weights
  const uint8_t *codes;
  const float *scale;       // kEnd: [E] or [E, N]; else [E, N, K / group]
  const uint8_t *sbytes;    // NVFP4 [E, N, K / 16]
  const uint8_t *zp;        // INT4 [E, N, K / group]
  const float *g;           // NVFP4 [E]
  int N, K, group;
  int groups;               // scale groups per row; 0: one scale per matrix
};

struct TokArgs {
  const uint16_t *x;        // [T, H]
  const int32_t *ids;       // [T, topk]
  const float *probs;       // [T, topk]
  int T, topk, P, ebegin, E, slots;
  FastDiv dtopk;
  int afmt1, afmt2;
  const float *as1, *as2;
  TokStack gu, d;
  int H, F;
  int ncol;                 // columns (tokens) staged at a time by the gate_up kernel
  int splits;               // k_tok_down blocks per 16 output columns
  // workspace
  uint16_t *a;              // [P, F] A's grid values, row = the pair's index
  int32_t *cnt;             // [slots] pairs of a slot's expert (0: nothing to do)
  int32_t *list;            // [slots, T] their pair indexes, ascending
  float *pw;                // [slots, T] their weights
  float *part;              // [splits, T, H] with splits > 1
  uint32_t *done;           // [H / 16] blocks finished, cleared by the gate_up kernel
  uint16_t *out;
};

// The expert of a slot: with fewer pairs than experts a slot is a pair (and
// only the first pair that names an expert does its work), else an expert.
__device__ __forceinline__ int slot_expert(const TokArgs &a, int slot) {
  if (a.P >= a.E) return slot;
  const int e = a.ids[slot] - a.ebegin;
  return (unsigned)e < (unsigned)a.E ? e : -1;
}

// ------------------------------------------------------------ weight codes --
struct Raw {
  uint32_t w[4];
  float s0, s1;  // kPre: scale of the segment (NVFP4: of its two 16-blocks); INT4: s1 = zero point
};

// One lane's segment of its row: k0 .. k0 + kSeg - 1 of row `row` of expert e.
// Past the end of the row nothing is read and the codes are 0.
template <int FMT, int MODE>
__device__ __forceinline__ Raw load_raw(const TokStack &t, size_t row, int k0) {
  Raw r;
  r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
  r.s0 = r.s1 = 0.0f;
  if (k0 >= t.K) return r;
  if (Fmt<FMT>::k4bit) {
    const uint8_t *p = t.codes + row * (size_t)(t.K >> 1) + (k0 >> 1);
    if ((t.K & 31) == 0) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p);
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {  // rows are multiples of 8 bytes, the last segment holds 16 codes
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      r.w[0] = v.x; r.w[1] = v.y;
      if (k0 + 16 < t.K) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + 8);
        r.w[2] = u.x; r.w[3] = u.y;
      }
    }
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(
        t.codes + (row * (size_t)t.K + k0) * (FMT == FQ_FMT_NONE ? 2 : 1));
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  }
  if (FMT == FQ_FMT_NVFP4) {
    const uint8_t *p = t.sbytes + row * (size_t)(t.K >> 4) + (k0 >> 4);
    uint32_t b;
    if ((t.K & 31) == 0) b = *reinterpret_cast<const uint16_t *>(p);
    else b = (uint32_t)p[0] | (k0 + 16 < t.K ? (uint32_t)p[1] << 8 : 0u);
    const f32x2_t th = __builtin_amdgcn_cvt_pk_f32_fp8(b, false);
    r.s0 = th.x;
    r.s1 = th.y;
  } else if (MODE == kPre || FMT == FQ_FMT_INT4) {
    const size_t gi = t.groups ? row * t.groups + k0 / t.group : 0;
    if (MODE == kPre) r.s0 = t.scale[gi];
    if (FMT == FQ_FMT_INT4) r.s1 = (float)t.zp[gi];
  }
  return r;
}

// Operand of MFMA step st of a chunk: 8 consecutive elements in bf16.
template <int FMT, int MODE>
__device__ __forceinline__ bf16x8v operand(const Raw &r, int st) {
  float v[8];
  if (FMT == FQ_FMT_NONE) {
    const bf16x8_t b = {{r.w[0], r.w[1], r.w[2], r.w[3]}};
    return __builtin_bit_cast(bf16x8v, b);
  }
  if (FMT == FQ_FMT_NVFP4) {
    const uint32_t c = r.w[st];
    const float s = st < 2 ? r.s0 : r.s1;
    const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    v[0] = p0.x * s; v[1] = p0.y * s; v[2] = p1.x * s; v[3] = p1.y * s;
    v[4] = p2.x * s; v[5] = p2.y * s; v[6] = p3.x * s; v[7] = p3.y * s;
  } else if (FMT == FQ_FMT_INT4) {
    const uint32_t c = r.w[st];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)((c >> (4 * j)) & 0xFu) - r.s1;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = r.w[2 * st + h];
      if (FMT == FQ_FMT_FP8_E4M3) {
        const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
        const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
        v[4 * h] = lo.x; v[4 * h + 1] = lo.y; v[4 * h + 2] = hi.x; v[4 * h + 3] = hi.y;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * h + j] = (float)((int)(c << (24 - 8 * j)) >> 24);
      }
    }
  }
  if (FMT != FQ_FMT_NVFP4 && MODE == kPre) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * r.s0;
  }
  return __builtin_bit_cast(bf16x8v, pack8(v));
}

// kPost: the chunk's scales of the four rows a lane holds of a result tile
template <int FMT>
__device__ __forceinline__ f32x4 chunk_scales(const TokStack &t, size_t row0, int chunk) {
  const int gi = chunk * Fmt<FMT>::kChunk / t.group;
  f32x4 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = t.scale[(row0 + i) * t.groups + gi];
  return s;
}

// the factor of a finished sum of one row of expert e
template <int FMT, int MODE>
__device__ __forceinline__ float row_scale(const TokStack &t, int e, size_t row) {
  if (FMT == FQ_FMT_NONE) return 1.0f;
  if (FMT == FQ_FMT_NVFP4) return t.g[e];
  if (MODE != kEnd) return 1.0f;
  return t.scale[t.groups ? row : (size_t)e];
}

// ------------------------------------------------------- activation values --
// FQ_a of 8 elements as grid values (without s_a, resp. g_a): the value the
// fake-quant gives is this times the scale. NVFP4: amax is the 16-block's.
__device__ __forceinline__ float block_theta(float amax, float g) {
  return e4m3_round_mag(fminf(amax * (1.0f / (6.0f * g)), kE4M3Max));
}
__device__ __forceinline__ void act_grid8(const ActQ &q, float theta, float *x) {
  if (q.fmt == FQ_FMT_NONE) return;
  if (q.fmt == FQ_FMT_NVFP4) {
    const float s = theta * q.s, r = safe_recip(s);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float v0, v1;
      e2m1_pair(x[2 * p] * r, x[2 * p + 1] * r, v0, v1);
      x[2 * p] = s != 0.0f ? v0 * theta : 0.0f;
      x[2 * p + 1] = s != 0.0f ? v1 * theta : 0.0f;
    }
  } else if (q.fmt == FQ_FMT_FP8_E4M3) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float v0, v1;
      e4m3_pair(clamp448(x[2 * p] * q.r), clamp448(x[2 * p + 1] * q.r), v0, v1);
      x[2 * p] = v0;
      x[2 * p + 1] = v1;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = rintf(fminf(fmaxf(x[j] * q.r, -128.0f), 127.0f));
  }
}
__device__ __forceinline__ float act_grid1(const ActQ &q, float theta, float x) {
  if (q.fmt == FQ_FMT_NONE) return x;
  if (q.fmt == FQ_FMT_NVFP4) {
    const float s = theta * q.s;
    float v0, v1;
    e2m1_pair(x * safe_recip(s), 0.0f, v0, v1);
    return s != 0.0f ? v0 * theta : 0.0f;
  }
  if (q.fmt == FQ_FMT_FP8_E4M3) {
    float v0, v1;
    e4m3_pair(clamp448(x * q.r), 0.0f, v0, v1);
    return v0;
  }
  return rintf(fminf(fmaxf(x * q.r, -128.0f), 127.0f));
}

// ---------------------------------------------------------------- gate_up ---
constexpr int kTile = 16;                        // A channels per block
constexpr int kRedBytes = kWaves * 2 * 64 * 16;  // the waves' sums of both tiles

// bytes of one staged token row: the row padded to whole chunks, and 16 more
// so that the 16 columns of a fragment read fall into different LDS banks
__host__ __device__ inline int xrow_bytes(int K, int chunk) {
  return (K + chunk - 1) / chunk * chunk * 2 + 16;
}

extern __shared__ __attribute__((aligned(16))) char g_tok_lds[];

// The pairs of expert e in ascending order into list (LDS); returns their
// number, and in `first` the first pair that names e (P: none). A pair that
// repeats an expert of its token is left to the first one.
__device__ __forceinline__ int build_list(const TokArgs &a, int e, int32_t *list, int *wcnt,
                                          int &first) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int n = 0;
  first = a.P;
  for (int q0 = 0; q0 < a.P; q0 += kNT) {
    const int q = q0 + tid;
    bool hit = q < a.P && a.ids[q] == e + a.ebegin;
    if (hit) {
      const int t0 = (int)a.dtopk.div((uint32_t)q) * a.topk;
      for (int p = t0; p < q; ++p)
        if (a.ids[p] == e + a.ebegin) { hit = false; break; }
    }
    const uint64_t m = __ballot(hit);
    if (lane == 0) wcnt[wave] = __popcll(m);
    __syncthreads();
    int base = n;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += wcnt[w];
      n += wcnt[w];
    }
    if (hit) list[base + __popcll(m & ((1ull << lane) - 1ull))] = q;
    __syncthreads();
  }
  if (n > 0) first = list[0];
  return n;
}

template <int FMT, int MODE>
__global__ __launch_bounds__(kNT) void k_tok_gate_up(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr int kU = 4;  // chunks a wave has in flight
  __shared__ int32_t list[128];
  __shared__ int wcnt[kWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int slot = blockIdx.x, f0 = blockIdx.y * kTile;
  // the down kernel's counters
  if (slot == 0 && a.done)
    for (int i = blockIdx.y * kNT + tid; i < a.H / 16; i += gridDim.y * kNT) a.done[i] = 0u;

  const int e = slot_expert(a, slot);
  int first = a.P, n = 0;
  if (e >= 0) n = build_list(a, e, list, wcnt, first);
  if (a.P < a.E && first != slot) n = 0;
  if (blockIdx.y == 0) {
    if (tid == 0) a.cnt[slot] = n;
    if (tid < n) {
      const int q = list[tid];
      const int t1 = ((int)a.dtopk.div((uint32_t)q) + 1) * a.topk;
      float p = a.probs[q];
      for (int i = q + 1; i < t1; ++i)
        if (a.ids[i] == e + a.ebegin) p += a.probs[i];
      a.list[(size_t)slot * a.T + tid] = q;
      a.pw[(size_t)slot * a.T + tid] = p;
    }
  }
  if (n == 0) return;

  const TokStack &w = a.gu;
  const ActQ q1 = load_actq(a.afmt1, a.as1), q2 = load_actq(a.afmt2, a.as2);
  const int nch = (w.K + kChunk - 1) / kChunk;
  const int xstride = xrow_bytes(w.K, kChunk);
  const int col = lane & 15, kq = lane >> 4;
  const size_t row_g = (size_t)e * w.N + f0, row_u = row_g + a.F;

  for (int c0 = 0; c0 < n; c0 += a.ncol) {
    const int nc = min(a.ncol, n - c0);
    // ---- the tokens' grid values into LDS (a row's tail chunk is zero-filled)
    const int vpr = nch * kChunk / 8, live = w.K / 8;
    for (int i = tid; i < nc * vpr; i += kNT) {
      const int c = i / vpr, v = i - c * vpr;
      bf16x8_t o = {{0u, 0u, 0u, 0u}};
      if (v < live) {
        const int t = (int)a.dtopk.div((uint32_t)list[c0 + c]);
        float f[8];
        o = reinterpret_cast<const bf16x8_t *>(a.x + (size_t)t * w.K)[v];
        if (q1.fmt != FQ_FMT_NONE) {
          unpack8(o, f);
          float theta = 0.0f;
          if (q1.fmt == FQ_FMT_NVFP4) {
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
            // the block's other half is on the neighbouring lane: vpr and the
            // thread count are even, and so is the number of live vectors
            amax = fmaxf(amax, __shfl_xor(amax, 1, 64));
            theta = block_theta(amax, q1.s);
          }
          act_grid8(q1, theta, f);
          o = pack8(f);
        }
      }
      *reinterpret_cast<bf16x8_t *>(g_tok_lds + c * xstride + v * 16) = o;
    }
    __syncthreads();

    // ---- this wave's chunks of the contraction
    f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const char *xs = g_tok_lds + min(col, nc - 1) * xstride;
    for (int cb = wave; cb < nch; cb += kWaves * kU) {
      Raw raw[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = cb + u * kWaves;
        if (ch < nch) {
          raw[u][0] = load_raw<FMT, MODE>(w, row_g + col, ch * kChunk + kq * kSeg);
          raw[u][1] = load_raw<FMT, MODE>(w, row_u + col, ch * kChunk + kq * kSeg);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = cb + u * kWaves;
        if (ch >= nch) break;
        f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
        if (MODE != kPost) {
          s0 = acc[0];
          s1 = acc[1];
        }
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const bf16x8v b = *reinterpret_cast<const bf16x8v *>(
              xs + (ch * kChunk + kq * kSeg + st * 8) * 2);
          s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FMT, MODE>(raw[u][0], st), b, s0, 0,
                                                       0, 0);
          s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand<FMT, MODE>(raw[u][1], st), b, s1, 0,
                                                       0, 0);
        }
        if (MODE == kPost) {
          acc[0] += s0 * chunk_scales<FMT>(w, row_g + 4 * kq, ch);
          acc[1] += s1 * chunk_scales<FMT>(w, row_u + 4 * kq, ch);
        } else {
          acc[0] = s0;
          acc[1] = s1;
        }
      }
    }
    __syncthreads();  // the staged rows are read: their space takes the sums
    f32x4 *red = reinterpret_cast<f32x4 *>(g_tok_lds);
    red[(wave * 2 + 0) * 64 + lane] = acc[0];
    red[(wave * 2 + 1) * 64 + lane] = acc[1];
    __syncthreads();
    if (tid < 256) {
      // channel f of column c: 16 consecutive lanes hold the 16 channels
      const int f = tid & 15, c = tid >> 4;
      const int idx = ((f >> 2) * 16 + c) * 4 + (f & 3);
      const float *rf = reinterpret_cast<const float *>(g_tok_lds);
      float hg = 0.0f, hu = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        hg += rf[(k * 2 + 0) * 256 + idx];
        hu += rf[(k * 2 + 1) * 256 + idx];
      }
      hg = hg * row_scale<FMT, MODE>(w, e, row_g + f) * q1.s;
      hu = hu * row_scale<FMT, MODE>(w, e, row_u + f) * q1.s;
      const float av = hg * sigmoid_hw(hg) * hu;
      float theta = 0.0f;
      if (q2.fmt == FQ_FMT_NVFP4) {
        float amax = fabsf(av);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
        theta = block_theta(amax, q2.s);
      }
      const float v = act_grid1(q2, theta, av);
      if (c < nc) a.a[(size_t)list[c0 + c] * a.F + f0 + f] = (uint16_t)f32_to_bf16(v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- down ---
// Block (i, s) forms output columns 16 i .. 16 i + 15 of every token, over the
// s-th share of the work: a worker (wave) takes units (expert, part of the
// contraction) in turn and adds each unit's weighted sums to its own [T, 16]
// block in LDS; the waves' blocks are added in wave order, the splits' sums by
// the block that finishes last, in split order.
template <int FMT, int MODE>
__global__ __launch_bounds__(kNT) void k_tok_down(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr int kU = 3;
  __shared__ int32_t act[1024];
  __shared__ int wcnt[kWaves];
  __shared__ uint32_t arrived;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int n0 = blockIdx.x * 16, split = blockIdx.y;
  float *accs = reinterpret_cast<float *>(g_tok_lds);  // [wave][T][16]
  for (int i = tid; i < kWaves * a.T * 16; i += kNT) accs[i] = 0.0f;

  // the slots with work, in slot order
  int na = 0;
  for (int s0 = 0; s0 < a.slots; s0 += kNT) {
    const int s = s0 + tid;
    const bool hit = s < a.slots && a.cnt[s] > 0;
    const uint64_t m = __ballot(hit);
    if (lane == 0) wcnt[wave] = __popcll(m);
    __syncthreads();
    int base = na;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += wcnt[w];
      na += wcnt[w];
    }
    if (hit) act[base + __popcll(m & ((1ull << lane) - 1ull))] = s;
    __syncthreads();
  }

  const TokStack &w = a.d;
  const ActQ q2 = load_actq(a.afmt2, a.as2);
  const int nch = (w.K + kChunk - 1) / kChunk;
  const int col = lane & 15, kq = lane >> 4;
  const int workers = kWaves * a.splits;
  // parts of a contraction, so that few experts still occupy every worker
  int kp = na > 0 ? workers / na : 1;
  kp = max(1, min(kp, nch));
  const int per = (nch + kp - 1) / kp;
  for (int u = split * kWaves + wave; u < na * kp; u += workers) {
    const int slot = act[u / kp], part = u - u / kp * kp;
    const int ch0 = part * per, ch1 = min(nch, ch0 + per);
    if (ch0 >= ch1) continue;
    const int e = slot_expert(a, slot), n = a.cnt[slot];
    const size_t row = (size_t)e * w.N + n0;
    const int32_t *list = a.list + (size_t)slot * a.T;
    const float *pw = a.pw + (size_t)slot * a.T;
    for (int c0 = 0; c0 < n; c0 += 16) {
      const int nc = min(16, n - c0);
      const int q = list[c0 + min(col, nc - 1)];
      const uint16_t *ap = a.a + (size_t)q * a.F;
      f32x4 acc = {0, 0, 0, 0};
      for (int cb = ch0; cb < ch1; cb += kU) {
        Raw raw[kU];
        bf16x8_t b[kU][kSteps];
#pragma unroll
        for (int i = 0; i < kU; ++i)
          if (cb + i < ch1) {
            const int k0 = (cb + i) * kChunk + kq * kSeg;
            raw[i] = load_raw<FMT, MODE>(w, row + col, k0);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
              b[i][st] = {{0u, 0u, 0u, 0u}};
              if (k0 + st * 8 < w.K)
                b[i][st] = *reinterpret_cast<const bf16x8_t *>(ap + k0 + st * 8);
            }
          }
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          if (cb + i >= ch1) break;
          f32x4 s = {0, 0, 0, 0};
          if (MODE != kPost) s = acc;
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
            s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                operand<FMT, MODE>(raw[i], st), __builtin_bit_cast(bf16x8v, b[i][st]), s, 0, 0, 0);
          if (MODE == kPost) acc += s * chunk_scales<FMT>(w, row + 4 * kq, cb + i);
          else acc = s;
        }
      }
      if (col < nc) {
        const int t = (int)a.dtopk.div((uint32_t)q);
        const float p = pw[c0 + col] * q2.s;
        f32x4 *dst = reinterpret_cast<f32x4 *>(accs + ((size_t)wave * a.T + t) * 16 + 4 * kq);
        f32x4 v = *dst;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = fmaf(acc[i] * row_scale<FMT, MODE>(w, e, row + 4 * kq + i), p, v[i]);
        *dst = v;
      }
    }
  }
  __syncthreads();

  for (int i = tid; i < a.T * 16; i += kNT) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) v += accs[k * a.T * 16 + i];
    const size_t o = (size_t)(i >> 4) * a.H + n0 + (i & 15);
    if (a.splits == 1) a.out[o] = (uint16_t)f32_to_bf16(v);
    else a.part[(size_t)split * a.T * a.H + o] = v;
  }
  if (a.splits == 1) return;
  // every thread's sums are visible to the device before the block counts itself
  __threadfence();
  __syncthreads();
  if (tid == 0) arrived = atomicAdd(&a.done[blockIdx.x], 1u);
  __syncthreads();
  if (arrived + 1u != (uint32_t)a.splits) return;
  __threadfence();
  for (int i = tid; i < a.T * 16; i += kNT) {
    const size_t o = (size_t)(i >> 4) * a.H + n0 + (i & 15);
    float v = 0.0f;
    for (int s = 0; s < a.splits; ++s) v += a.part[(size_t)s * a.T * a.H + o];
    a.out[o] = (uint16_t)f32_to_bf16(v);
  }
}

TokStack tok_stack(const fq_stored_w &w, int N, int K) {
  TokStack t;
  t.codes = static_cast<const uint8_t *>(w.codes);
  t.scale = w.scale;
  t.sbytes = w.scale_bytes;
  t.zp = w.zero_point_bytes;
  t.g = w.global_scale;
  t.N = N;
  t.K = K;
  t.group = w.group > 0 ? w.group : K;
  t.groups = w.group > 0 ? K / w.group : 0;
  return t;
}

template <int FMT>
int scale_mode(const TokStack &t) {
  if (t.groups <= 1) return kEnd;
  return t.group % Fmt<FMT>::kChunk == 0 ? kPost : kPre;
}

template <int FMT, int MODE>
void launch_one(bool down, const TokArgs &a, dim3 grid, int lds, hipStream_t st) {
  if (down) hipLaunchKernelGGL((k_tok_down<FMT, MODE>), grid, dim3(kNT), lds, st, a);
  else hipLaunchKernelGGL((k_tok_gate_up<FMT, MODE>), grid, dim3(kNT), lds, st, a);
}

template <int FMT>
void launch_mode(bool down, const TokArgs &a, dim3 grid, int lds, hipStream_t st) {
  switch (scale_mode<FMT>(down ? a.d : a.gu)) {
    case kEnd: launch_one<FMT, kEnd>(down, a, grid, lds, st); break;
    case kPost: launch_one<FMT, kPost>(down, a, grid, lds, st); break;
    default: launch_one<FMT, kPre>(down, a, grid, lds, st); break;
  }
}

void launch_fmt(int fmt, bool down, const TokArgs &a, dim3 grid, int lds, hipStream_t st) {
  switch (fmt) {
    case FQ_FMT_INT8: launch_mode<FQ_FMT_INT8>(down, a, grid, lds, st); break;
    case FQ_FMT_FP8_E4M3: launch_mode<FQ_FMT_FP8_E4M3>(down, a, grid, lds, st); break;
    case FQ_FMT_INT4: launch_mode<FQ_FMT_INT4>(down, a, grid, lds, st); break;
    case FQ_FMT_NVFP4: launch_one<FQ_FMT_NVFP4, kPre>(down, a, grid, lds, st); break;
    default: launch_one<FQ_FMT_NONE, kEnd>(down, a, grid, lds, st); break;
  }
}

inline int chunk_of(int fmt) {
  return fmt == FQ_FMT_NONE ? Fmt<FQ_FMT_NONE>::kChunk
         : fmt == FQ_FMT_INT8 || fmt == FQ_FMT_FP8_E4M3 ? Fmt<FQ_FMT_INT8>::kChunk
                                                         : Fmt<FQ_FMT_INT4>::kChunk;
}

// blocks per 16 output columns of the down kernel: enough of them for every
// CU, but at least eight slots to each
int down_splits(int slots, int H) {
  const int want = (256 + H / 16 - 1) / (H / 16);
  const int most = slots / 8 > 1 ? slots / 8 : 1;
  return want < most ? want : most;
}

inline size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct TokWs {
  size_t a, cnt, list, pw, part, done, total;
};
TokWs tok_ws(int T, int topk, int E, int H, int F) {
  const size_t P = (size_t)T * topk, slots = P < (size_t)E ? P : (size_t)E;
  const int S = down_splits((int)slots, H);
  TokWs w;
  size_t o = 0;
  w.a = o;     o += up256(P * F * 2);
  w.cnt = o;   o += up256(slots * 4);
  w.list = o;  o += up256(slots * T * 4);
  w.pw = o;    o += up256(slots * T * 4);
  w.part = o;  o += S > 1 ? up256((size_t)S * T * H * 4) : 0;
  w.done = o;  o += up256((size_t)H / 16 * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t moe_tokens_ws_bytes(int T, int topk, int E, int H, int F) {
  return tok_ws(T, topk, E, H, F).total;
}

void launch_moe_tokens(const uint16_t *x, int T, int H, int F, const int32_t *ids,
                       const float *probs, int topk, int ebegin, int E, const fq_stored_w &w_gu,
                       const fq_stored_w &w_d, int afmt1, const float *as1, int afmt2,
                       const float *as2, uint16_t *out, void *ws, hipStream_t st) {
  const TokWs o = tok_ws(T, topk, E, H, F);
  char *b = static_cast<char *>(ws);
  TokArgs a;
  a.x = x;
  a.ids = ids;
  a.probs = probs;
  a.T = T;
  a.topk = topk;
  a.P = T * topk;
  a.ebegin = ebegin;
  a.E = E;
  a.slots = a.P < E ? a.P : E;
  a.dtopk = FastDiv((uint32_t)topk);
  a.afmt1 = afmt1;
  a.afmt2 = afmt2;
  a.as1 = as1;
  a.as2 = as2;
  a.gu = tok_stack(w_gu, 2 * F, H);
  a.d = tok_stack(w_d, H, F);
  a.H = H;
  a.F = F;
  a.splits = down_splits(a.slots, H);
  a.a = reinterpret_cast<uint16_t *>(b + o.a);
  a.cnt = reinterpret_cast<int32_t *>(b + o.cnt);
  a.list = reinterpret_cast<int32_t *>(b + o.list);
  a.pw = reinterpret_cast<float *>(b + o.pw);
  a.part = reinterpret_cast<float *>(b + o.part);
  a.done = reinterpret_cast<uint32_t *>(b + o.done);
  a.out = out;
  // token rows staged at a time: 16 columns of an MFMA, or what 72 KB hold
  // (two blocks to a CU), at least one
  const int row = xrow_bytes(H, chunk_of(w_gu.fmt));
  int nc = (72 << 10) / row;
  nc = nc < 1 ? 1 : nc > 16 ? 16 : nc;
  a.ncol = nc < T ? nc : T;
  int lds = a.ncol * row;
  if (lds < kRedBytes) lds = kRedBytes;
  launch_fmt(w_gu.fmt, false, a, dim3(a.slots, F / kTile), lds, st);
  launch_fmt(w_d.fmt, true, a, dim3(H / 16, a.splits), kWaves * T * 16 * 4, st);
}

}  // namespace fq
