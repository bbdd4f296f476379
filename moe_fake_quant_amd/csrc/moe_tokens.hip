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
typedef __attribute__((__vector_size__(8 * sizeof(_Float16)))) _Float16 f16x8v;
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kNT = 512;        // threads per block of the gate_up kernel
constexpr int kWaves = kNT / 64;
constexpr int kNTd = 1024;      // of the down kernel
constexpr int kWavesD = kNTd / 64;

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
  int N, K;
  int groups;               // scale groups per row; 0: one scale per matrix
  int nch;                  // chunks per row
  int whole;                // rows are whole chunks
  int f16;                  // operands are f16 (NVFP4 with quantized activations)
  FastDiv dgroup;           // / group
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
  FastDiv dvpr;             // / 8-element vectors of a staged token row
  // workspace. Rows are ordered by expert; a slot's rows are off .. off + cnt - 1.
  uint16_t *a;              // [P, F] A's grid values
  int2 *span;               // [slots] {off, cnt} (cnt 0: nothing to do)
  int32_t *tok;             // [P] a row's token
  float *pw;                // [P] its weight
  uint16_t *out;
};

// The expert of a slot: with fewer pairs than experts a slot is a pair (and
// only the first pair that names an expert does its work), else an expert.
__device__ __forceinline__ int local_id(const TokArgs &a, int q) {  // wraps, never overflows
  return (int)((uint32_t)a.ids[q] - (uint32_t)a.ebegin);
}
__device__ __forceinline__ int slot_expert(const TokArgs &a, int slot) {
  if (a.P >= a.E) return slot;
  const int e = local_id(a, slot);
  return (unsigned)e < (unsigned)a.E ? e : -1;
}

// ------------------------------------------------------------ weight codes --
struct Raw {
  uint32_t w[4];
  uint32_t sb;   // NVFP4: the block scale bytes of the segment's two 16-blocks
  float s0, zp;  // kPre: the segment's scale; INT4: its zero point
};

// One lane's row, from the lane's segment of chunk 0 on. A chunk is 64 bytes of
// codes in every format (4 lane groups x 16 bytes).
struct RowPtr {
  const uint8_t *c, *sb, *zp;
  const float *sc;
};
template <int FMT, int MODE>
__device__ __forceinline__ RowPtr row_ptr(const TokStack &t, size_t row, int kq) {
  RowPtr p;
  const size_t bytes = FMT == FQ_FMT_NONE ? (size_t)t.K * 2
                       : Fmt<FMT>::k4bit ? (size_t)t.K / 2 : (size_t)t.K;
  p.c = t.codes + row * bytes + kq * 16;
  p.sb = FMT == FQ_FMT_NVFP4 ? t.sbytes + row * (size_t)(t.K >> 4) + kq * 2 : nullptr;
  p.zp = FMT == FQ_FMT_INT4 ? t.zp + row * (size_t)t.groups : nullptr;
  p.sc = MODE == kPre && FMT != FQ_FMT_NVFP4 ? t.scale + row * (size_t)t.groups : nullptr;
  return p;
}

// The lane's segment of chunk ch. Past the end of the row nothing is read and
// the codes are 0 (what they meet there is 0 too).
template <int FMT, int MODE>
__device__ __forceinline__ Raw load_raw(const TokStack &t, const RowPtr &p, int ch, int kq) {
  const int k0 = ch * Fmt<FMT>::kChunk + kq * Fmt<FMT>::kSeg;
  Raw r;
  if (t.whole) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p.c + ch * 64);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    if (FMT == FQ_FMT_NVFP4) r.sb = *reinterpret_cast<const uint16_t *>(p.sb + ch * 8);
  } else {
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = r.sb = 0u;
    r.s0 = r.zp = 0.0f;
    if (k0 >= t.K) return r;
    const uint8_t *c = p.c + ch * 64;
    if (Fmt<FMT>::k4bit && (t.K & 31)) {
      // rows are multiples of 8 bytes, the last segment may hold 16 codes
      const uint2 v = *reinterpret_cast<const uint2 *>(c);
      r.w[0] = v.x; r.w[1] = v.y;
      if (k0 + 16 < t.K) {
        const uint2 u = *reinterpret_cast<const uint2 *>(c + 8);
        r.w[2] = u.x; r.w[3] = u.y;
      }
    } else {
      const uint4 v = *reinterpret_cast<const uint4 *>(c);
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
    if (FMT == FQ_FMT_NVFP4) {
      const uint8_t *b = p.sb + ch * 8;
      r.sb = (uint32_t)b[0] | (k0 + 16 < t.K ? (uint32_t)b[1] << 8 : 0u);
    }
  }
  if (FMT == FQ_FMT_INT4 || (MODE == kPre && FMT != FQ_FMT_NVFP4)) {
    const uint32_t gi = t.dgroup.div((uint32_t)k0);
    if (MODE == kPre) r.s0 = p.sc[gi];
    if (FMT == FQ_FMT_INT4) r.zp = (float)p.zp[gi];
  }
  return r;
}

// One MFMA over step st of a chunk: 8 consecutive elements of the lane's row
// against the 8 activation grid values in x (bf16, or f16 with F16).
//
// VALU operations per 8 codes: E4M3 4 (the converter makes bf16 pairs), NVFP4
// 8 in f16 (convert and multiply pairs by the block scale) or 16 through fp32
// in bf16, int4 23, int8 about 16. f16 holds every NVFP4, E4M3 and int8 grid
// value exactly (at most 8 bits, 2^-10 <= |v| <= 2688), but not any bf16
// activation, so it is used for quantized activations.
template <int FMT, int MODE, bool F16>
__device__ __forceinline__ f32x4 mfma_step(const Raw &r, int st, const bf16x8_t &x, f32x4 acc) {
  if (FMT == FQ_FMT_NVFP4 && F16) {
    const uint32_t c = r.w[st];
    const f16x2 th = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(r.sb, 1.0f, false);
    const _Float16 s = st < 2 ? th.x : th.y;
    const f16x2 ss = {s, s};
    f16x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * ss;
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * ss;
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * ss;
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * ss;
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, v),
                                                  __builtin_bit_cast(f16x8v, x), acc, 0, 0, 0);
  }
  bf16x8_t o;
  if (FMT == FQ_FMT_NONE) {
    o = {{r.w[0], r.w[1], r.w[2], r.w[3]}};
  } else if (FMT == FQ_FMT_FP8_E4M3 && MODE != kPre) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = r.w[2 * st + h];
      o.w[2 * h] = __builtin_bit_cast(uint32_t,
                                      __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
      o.w[2 * h + 1] = __builtin_bit_cast(uint32_t,
                                          __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
    }
  } else {
    float v[8];
    if (FMT == FQ_FMT_NVFP4) {
      const uint32_t c = r.w[st];
      const f32x2_t th = __builtin_amdgcn_cvt_pk_f32_fp8(r.sb, false);
      const float s = st < 2 ? th.x : th.y;
      const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
      const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
      const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
      const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
      v[0] = p0.x * s; v[1] = p0.y * s; v[2] = p1.x * s; v[3] = p1.y * s;
      v[4] = p2.x * s; v[5] = p2.y * s; v[6] = p3.x * s; v[7] = p3.y * s;
    } else if (FMT == FQ_FMT_INT4) {
      // even and odd codes to bytes, which convert in one instruction each
      const uint32_t ev = r.w[st] & 0x0F0F0F0Fu, od = (r.w[st] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = (float)((ev >> (8 * j)) & 0xFFu) - r.zp;
        v[2 * j + 1] = (float)((od >> (8 * j)) & 0xFFu) - r.zp;
      }
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
    o = pack8(v);
  }
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, o),
                                                 __builtin_bit_cast(bf16x8v, x), acc, 0, 0, 0);
}

// kPost: the chunk's scales of the four rows a lane holds of a result tile
template <int FMT>
__device__ __forceinline__ f32x4 chunk_scales(const TokStack &t, size_t row0, int chunk) {
  const float *p = t.scale + row0 * t.groups + t.dgroup.div((uint32_t)(chunk * Fmt<FMT>::kChunk));
  f32x4 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = p[(size_t)i * t.groups];
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
// rg6: 1 / (6 g_a)
__device__ __forceinline__ float block_theta(float amax, float rg6) {
  float v0, v1;
  e4m3_pair(fminf(amax * rg6, kE4M3Max), 0.0f, v0, v1);
  return v0;
}
// N (even) elements; with a zero block scale every value is a zero
template <int N>
__device__ __forceinline__ void act_grid(const ActQ &q, float theta, float *x) {
  if (q.fmt == FQ_FMT_NONE) return;
  if (q.fmt == FQ_FMT_NVFP4) {
    const float r = safe_recip(theta * q.s);
#pragma unroll
    for (int p = 0; p < N; p += 2) {
      float v0, v1;
      e2m1_pair(x[p] * r, x[p + 1] * r, v0, v1);
      x[p] = v0 * theta;
      x[p + 1] = v1 * theta;
    }
  } else if (q.fmt == FQ_FMT_FP8_E4M3) {
#pragma unroll
    for (int p = 0; p < N; p += 2)
      e4m3_pair(clamp448(x[p] * q.r), clamp448(x[p + 1] * q.r), x[p], x[p + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = rintf(fminf(fmaxf(x[j] * q.r, -128.0f), 127.0f));
  }
}

// ---------------------------------------------------------------- gate_up ---
constexpr int kTile = 16;                        // A channels of one wave's pair of tiles
constexpr int kRedBytes = kWaves * 2 * 64 * 16;  // the waves' sums of their two tiles

// bytes of one staged token row: the row padded to whole chunks, and 16 more
// so that the 16 columns of a fragment read fall into different LDS banks
__host__ __device__ inline int xrow_bytes(int K, int chunk) {
  return (K + chunk - 1) / chunk * chunk * 2 + 16;
}

extern __shared__ __attribute__((aligned(16))) char g_tok_lds[];

// A slot's rows: its expert's pairs in ascending order, a pair that repeats an
// expert of its token left to the first one (which takes the summed weight).
struct SlotRows {
  int32_t tok[128];
  float pw[128];
  int32_t ids[kNT];
  int wcnt[2][kWaves];
  int first;
};

// Fills r (LDS) for expert e and returns the number of rows; `off`: the rows of
// experts below e come before; `first`: the pair of the first row (P: none).
__device__ __forceinline__ int build_rows(const TokArgs &a, int e, SlotRows &r, int &off,
                                          int &first) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int per = (int)a.dtopk.div((uint32_t)kNT) * a.topk;  // whole tokens per pass
  int n = 0;
  off = 0;
  first = a.P;
  for (int q0 = 0; q0 < a.P; q0 += per) {
    const int q = q0 + tid;
    const bool in = tid < per && q < a.P;
    const int id = in ? local_id(a, q) : -1;
    float p = in ? a.probs[q] : 0.0f;
    r.ids[tid] = id;
    // a pair below the expert takes a row, whether or not it repeats one
    const uint64_t below = __ballot(id >= 0 && id < e);
    __syncthreads();
    bool hit = in && id == e;
    const int t = (int)a.dtopk.div((uint32_t)tid);
    if (hit) {
      for (int i = t * a.topk; i < tid; ++i)
        if (r.ids[i] == e) hit = false;
      if (hit)
        for (int i = tid + 1; i < (t + 1) * a.topk; ++i)
          if (r.ids[i] == e) p += a.probs[q0 + i];
    }
    const uint64_t m = __ballot(hit);
    if (lane == 0) {
      r.wcnt[0][wave] = __popcll(m);
      r.wcnt[1][wave] = __popcll(below);
    }
    __syncthreads();
    int base = n;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += r.wcnt[0][w];
      n += r.wcnt[0][w];
      off += r.wcnt[1][w];
    }
    if (hit) {
      const int i = base + __popcll(m & ((1ull << lane) - 1ull));
      r.tok[i] = (int)a.dtopk.div((uint32_t)q);
      r.pw[i] = p;
      if (i == 0) r.first = q;
    }
    __syncthreads();
    if (n > 0) first = r.first;
  }
  return n;
}

// One 8-element vector of a token row as grid values (the neighbouring lane
// holds the other half of its 16-block).
template <bool F16>
__device__ __forceinline__ bf16x8_t stage_vec(const ActQ &q, bf16x8_t o, float rg6) {
  if (q.fmt == FQ_FMT_NONE) return o;
  float f[8];
  unpack8(o, f);
  float theta = 0.0f;
  if (q.fmt == FQ_FMT_NVFP4) {
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
    amax = fmaxf(amax, __shfl_xor(amax, 1, 64));
    theta = block_theta(amax, rg6);
  }
  act_grid<8>(q, theta, f);
  if (!F16) return pack8(f);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o.w[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(f[2 * j], f[2 * j + 1]));
  return o;
}

// A block forms MT x 16 channels of A for one expert and its tokens. Its eight
// waves are MT channel groups (gate and up rows of the same 16 channels) times
// 8 / MT shares of the contraction. MT follows from the number of blocks: more
// channels to a block spread the staging of the tokens over more weights, fewer
// keep every CU busy for a handful of tokens (see launch_moe_tokens).
template <int FMT, int MODE, bool F16, int MT>
__global__ __launch_bounds__(kNT, 4) void k_tok_gate_up(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr int kWK = kWaves / MT;
  constexpr int kU = 2;  // chunks of a batch; one batch computes while the next loads
  constexpr int kX = 2;  // token vectors a thread has in flight
  __shared__ SlotRows rows;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int slot = blockIdx.x;

  const int e = slot_expert(a, slot);
  int first = a.P, n = 0, off = 0;
  if (e >= 0) n = build_rows(a, e, rows, off, first);
  if (a.P < a.E && first != slot) n = 0;
  if (blockIdx.y == 0) {
    if (tid == 0) a.span[slot] = make_int2(off, n);
    if (tid < n) {
      a.tok[off + tid] = rows.tok[tid];
      a.pw[off + tid] = rows.pw[tid];
    }
  }
  if (n == 0) return;

  const TokStack &w = a.gu;
  const ActQ q1 = load_actq(a.afmt1, a.as1), q2 = load_actq(a.afmt2, a.as2);
  const float rg1 = 1.0f / (6.0f * q1.s);
  const int xstride = xrow_bytes(w.K, kChunk);
  const int col = lane & 15, kq = lane >> 4;
  const int wm = wave / kWK, wk = wave % kWK;
  const int f0 = (blockIdx.y * MT + wm) * kTile;
  const bool live_w = f0 < a.F;  // the last block's waves past F only stage and sync
  const size_t row_g = (size_t)e * w.N + (live_w ? f0 : 0), row_u = row_g + a.F;
  const RowPtr pg = row_ptr<FMT, MODE>(w, row_g + col, kq);
  const RowPtr pu = row_ptr<FMT, MODE>(w, row_u + col, kq);
  const int nch = live_w ? w.nch : 0;
  const int vpr = w.nch * kChunk / 8, live = w.K / 8;

  Raw raw[2][kU][2];
  auto load = [&](Raw (&r)[kU][2], int cb) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (cb + u * kWK < nch) {
        r[u][0] = load_raw<FMT, MODE>(w, pg, cb + u * kWK, kq);
        r[u][1] = load_raw<FMT, MODE>(w, pu, cb + u * kWK, kq);
      }
  };

  for (int c0 = 0; c0 < n; c0 += a.ncol) {
    const int nc = min(a.ncol, n - c0), nvec = nc * vpr;
    // ---- the tokens' grid values into LDS, a row's vectors beyond K zero. The
    // first weights are requested behind the first token vectors and arrive
    // while those are quantized. (vpr is even: both lanes of a 16-block take
    // part together.)
    for (int i0 = 0; i0 < nvec; i0 += kX * kNT) {
      bf16x8_t xv[kX];
      int dst[kX];
#pragma unroll
      for (int j = 0; j < kX; ++j) {
        const int i = i0 + j * kNT + tid;
        const int c = (int)a.dvpr.div((uint32_t)i), v = i - c * vpr;
        dst[j] = i < nvec ? c * xstride + v * 16 : -1;
        xv[j] = {{0u, 0u, 0u, 0u}};
        if (i < nvec && v < live)
          xv[j] = reinterpret_cast<const bf16x8_t *>(a.x + (size_t)rows.tok[c0 + c] * w.K)[v];
      }
      if (i0 == 0) load(raw[0], wk);
#pragma unroll
      for (int j = 0; j < kX; ++j)
        if (dst[j] >= 0)
          *reinterpret_cast<bf16x8_t *>(g_tok_lds + dst[j]) = stage_vec<F16>(q1, xv[j], rg1);
    }
    __syncthreads();

    // ---- this wave's chunks of the contraction, two batches of loads in turn
    f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    const char *xs = g_tok_lds + min(col, nc - 1) * xstride + kq * kSeg * 2;
    auto compute = [&](Raw (&r)[kU][2], int cb) {
      f32x4 cs[kU][2];
      if (MODE == kPost) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (cb + u * kWK < nch) {
            cs[u][0] = chunk_scales<FMT>(w, row_g + 4 * kq, cb + u * kWK);
            cs[u][1] = chunk_scales<FMT>(w, row_u + 4 * kq, cb + u * kWK);
          }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = cb + u * kWK;
        if (ch >= nch) break;
        f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
        if (MODE != kPost) {
          s0 = acc[0];
          s1 = acc[1];
        }
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const bf16x8_t b =
              *reinterpret_cast<const bf16x8_t *>(xs + (ch * kChunk + st * 8) * 2);
          s0 = mfma_step<FMT, MODE, F16>(r[u][0], st, b, s0);
          s1 = mfma_step<FMT, MODE, F16>(r[u][1], st, b, s1);
        }
        if (MODE == kPost) {
          acc[0] += s0 * cs[u][0];
          acc[1] += s1 * cs[u][1];
        } else {
          acc[0] = s0;
          acc[1] = s1;
        }
      }
    };
    for (int cb = wk; cb < nch; cb += 2 * kU * kWK) {
      load(raw[1], cb + kU * kWK);
      compute(raw[0], cb);
      load(raw[0], cb + 2 * kU * kWK);
      compute(raw[1], cb + kU * kWK);
    }
    __syncthreads();  // the staged rows are read: their space takes the sums

    // ---- the shares' sums, SwiGLU, FQ_a2. Each wave holds its group's tiles.
    f32x4 *red = reinterpret_cast<f32x4 *>(g_tok_lds);
    red[(wave * 2 + 0) * 64 + lane] = acc[0];
    red[(wave * 2 + 1) * 64 + lane] = acc[1];
    __syncthreads();
    // channel f of column c: 16 consecutive lanes hold a group's 16 channels
    for (int i = tid; i < MT * 256; i += kNT) {
      const int m = i >> 8, f = i & 15, c = (i >> 4) & 15;
      const int fb = (blockIdx.y * MT + m) * kTile;
      const int idx = ((f >> 2) * 16 + c) * 4 + (f & 3);
      const float *rf = reinterpret_cast<const float *>(g_tok_lds) + m * kWK * 512;
      float hg = 0.0f, hu = 0.0f;
#pragma unroll
      for (int k = 0; k < kWK; ++k) {
        hg += rf[k * 512 + idx];
        hu += rf[k * 512 + 256 + idx];
      }
      if (fb >= a.F) continue;  // whole groups of 16 lanes
      const size_t row = (size_t)e * w.N + fb + f;
      hg = hg * row_scale<FMT, MODE>(w, e, row) * q1.s;
      hu = hu * row_scale<FMT, MODE>(w, e, row + a.F) * q1.s;
      float av[2] = {hg * sigmoid_hw(hg) * hu, 0.0f};
      float theta = 0.0f;
      if (q2.fmt == FQ_FMT_NVFP4) {
        float amax = fabsf(av[0]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
        theta = block_theta(amax, 1.0f / (6.0f * q2.s));
      }
      act_grid<2>(q2, theta, av);
      const uint32_t v =
          a.d.f16 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(av[0], 0.0f))
                  : f32_to_bf16(av[0]);
      if (c < nc) a.a[(size_t)(off + c0 + c) * a.F + fb + f] = (uint16_t)v;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- down ---
// A block forms 8 output columns of every token, over all experts: nothing is
// shared between blocks. An MFMA's 16 weight rows are the same 8 rows of two
// experts and its 16 columns up to 8 tokens of each; the two diagonal blocks of
// the result are used (the MFMAs have time to spare, the weights are decoded
// once either way). A wave takes units (two experts, part of the contraction)
// in turn and adds their weighted sums to its own [T, 8] block in LDS; the
// waves' blocks are added in wave order.
template <int FMT, int MODE, bool F16>
__global__ __launch_bounds__(kNTd) void k_tok_down(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr int kU = FMT == FQ_FMT_NONE ? 6 : Fmt<FMT>::k4bit ? 3 : 4;
  __shared__ int32_t act_e[1024];
  __shared__ int2 act_span[1024];
  __shared__ int wcnt[kWavesD];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int n0 = blockIdx.x * 8;
  float *accs = reinterpret_cast<float *>(g_tok_lds);  // [wave][T][8]

  // the slots with work, in slot order (there are at most as many as threads)
  const int2 sp = tid < a.slots ? a.span[tid] : make_int2(0, 0);
  const int my_e = sp.y > 0 ? slot_expert(a, tid) : 0;
  for (int i = tid; i < kWavesD * a.T * 8; i += kNTd) accs[i] = 0.0f;
  const uint64_t m = __ballot(sp.y > 0);
  if (lane == 0) wcnt[wave] = __popcll(m);
  __syncthreads();
  int base = 0, na = 0;
  for (int w = 0; w < kWavesD; ++w) {
    if (w < wave) base += wcnt[w];
    na += wcnt[w];
  }
  if (sp.y > 0) {
    const int i = base + __popcll(m & ((1ull << lane) - 1ull));
    act_e[i] = my_e;
    act_span[i] = sp;
  }
  __syncthreads();

  const TokStack &w = a.d;
  const ActQ q2 = load_actq(a.afmt2, a.as2);
  const int nch = w.nch;
  const int col = lane & 15, kq = lane >> 4;
  const int pairs = (na + 1) / 2;
  // parts of a contraction, so that few experts still occupy every wave
  int kp = pairs > 0 ? kWavesD / pairs : 1;
  kp = max(1, min(kp, nch));
  const int per = (nch + kp - 1) / kp;
  for (int u = wave; u < pairs * kp; u += kWavesD) {
    const int pr = u / kp, part = u - pr * kp;
    const int ch0 = part * per, ch1 = min(nch, ch0 + per);
    // this lane's weight row, its column's row of A, and the rows and column
    // of the result it holds
    // (without a second expert its lanes repeat the first: their part of the
    // result is not used)
    const int i1 = min(2 * pr + 1, na - 1);
    const int iw = (col >> 3) ? i1 : 2 * pr, ir = (kq >> 1) ? i1 : 2 * pr;
    const bool has_w = 2 * pr + (col >> 3) < na;
    const int2 sc = act_span[iw];
    const RowPtr pw = row_ptr<FMT, MODE>(w, (size_t)act_e[iw] * w.N + n0 + (col & 7), kq);
    const int er = act_e[ir];
    const size_t row_r = (size_t)er * w.N + n0 + 4 * (kq & 1);
    const int nmax = max(act_span[2 * pr].y, act_span[i1].y);
    for (int c0 = 0; c0 < nmax; c0 += 8) {
      // a column past the expert's last repeats it, and is not used
      const bool live_c = has_w && c0 + (col & 7) < sc.y;
      const int r = sc.x + min(c0 + (col & 7), sc.y - 1);
      const uint16_t *ap = a.a + (size_t)r * a.F + kq * kSeg;
      const int t = a.tok[r];
      const float p = a.pw[r];
      f32x4 acc = {0, 0, 0, 0};
      for (int cb = ch0; cb < ch1; cb += kU) {
        Raw raw[kU];
        f32x4 cs[kU];
        bf16x8_t b[kU][kSteps];
#pragma unroll
        for (int i = 0; i < kU; ++i)
          if (cb + i < ch1) {
            raw[i] = load_raw<FMT, MODE>(w, pw, cb + i, kq);
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
              const int k = (cb + i) * kChunk + st * 8;
              if (w.whole) {
                b[i][st] = *reinterpret_cast<const bf16x8_t *>(ap + k);
              } else {
                b[i][st] = {{0u, 0u, 0u, 0u}};
                if (k + kq * kSeg < w.K)
                  b[i][st] = *reinterpret_cast<const bf16x8_t *>(ap + k);
              }
            }
            if (MODE == kPost) cs[i] = chunk_scales<FMT>(w, row_r, cb + i);
          }
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          if (cb + i >= ch1) break;
          f32x4 s = {0, 0, 0, 0};
          if (MODE != kPost) s = acc;
#pragma unroll
          for (int st = 0; st < kSteps; ++st) s = mfma_step<FMT, MODE, F16>(raw[i], st, b[i][st], s);
          if (MODE == kPost) acc += s * cs[i];
          else acc = s;
        }
      }
      const float ps = p * q2.s;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = acc[i] * row_scale<FMT, MODE>(w, er, row_r + i) * ps;
      // a token may be in both experts' columns: one expert's lanes after the
      // other's (a wave's LDS accesses execute in order)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (live_c && (col >> 3) == h && (kq >> 1) == h) {
          f32x4 *dst =
              reinterpret_cast<f32x4 *>(accs + ((size_t)wave * a.T + t) * 8 + 4 * (kq & 1));
          *dst += acc;
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
      }
    }
  }
  __syncthreads();

  for (int i = tid; i < a.T * 8; i += kNTd) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWavesD; ++k) v += accs[k * a.T * 8 + i];
    a.out[(size_t)(i >> 3) * a.H + n0 + (i & 7)] = (uint16_t)f32_to_bf16(v);
  }
}

inline int chunk_of(int fmt) {
  return fmt == FQ_FMT_NONE ? Fmt<FQ_FMT_NONE>::kChunk
         : fmt == FQ_FMT_INT8 || fmt == FQ_FMT_FP8_E4M3 ? Fmt<FQ_FMT_INT8>::kChunk
                                                         : Fmt<FQ_FMT_INT4>::kChunk;
}

TokStack tok_stack(const fq_stored_w &w, int N, int K, int afmt) {
  TokStack t;
  const int chunk = chunk_of(w.fmt), group = w.group > 0 ? w.group : K;
  t.codes = static_cast<const uint8_t *>(w.codes);
  t.scale = w.scale;
  t.sbytes = w.scale_bytes;
  t.zp = w.zero_point_bytes;
  t.g = w.global_scale;
  t.N = N;
  t.K = K;
  t.groups = w.group > 0 ? K / w.group : 0;
  t.nch = (K + chunk - 1) / chunk;
  t.whole = K % chunk == 0;
  t.f16 = w.fmt == FQ_FMT_NVFP4 && afmt != FQ_FMT_NONE;
  t.dgroup = FastDiv((uint32_t)group);
  return t;
}

struct Launch {
  bool down;
  int mt;  // channel groups per gate_up block
  dim3 grid;
  int lds;
};

template <int FMT, int MODE, bool F16>
void launch_one(const Launch &l, const TokArgs &a, hipStream_t st) {
  if (l.down)
    hipLaunchKernelGGL((k_tok_down<FMT, MODE, F16>), l.grid, dim3(kNTd), l.lds, st, a);
  else if (l.mt == 4)
    hipLaunchKernelGGL((k_tok_gate_up<FMT, MODE, F16, 4>), l.grid, dim3(kNT), l.lds, st, a);
  else if (l.mt == 2)
    hipLaunchKernelGGL((k_tok_gate_up<FMT, MODE, F16, 2>), l.grid, dim3(kNT), l.lds, st, a);
  else
    hipLaunchKernelGGL((k_tok_gate_up<FMT, MODE, F16, 1>), l.grid, dim3(kNT), l.lds, st, a);
}

template <int FMT>
void launch_mode(const Launch &l, const TokArgs &a, int group, hipStream_t st) {
  const TokStack &t = l.down ? a.d : a.gu;
  if (t.groups <= 1) launch_one<FMT, kEnd, false>(l, a, st);
  else if (group % Fmt<FMT>::kChunk == 0) launch_one<FMT, kPost, false>(l, a, st);
  else launch_one<FMT, kPre, false>(l, a, st);
}

void launch_fmt(const fq_stored_w &w, const Launch &l, const TokArgs &a, hipStream_t st) {
  switch (w.fmt) {
    case FQ_FMT_INT8: launch_mode<FQ_FMT_INT8>(l, a, w.group, st); break;
    case FQ_FMT_FP8_E4M3: launch_mode<FQ_FMT_FP8_E4M3>(l, a, w.group, st); break;
    case FQ_FMT_INT4: launch_mode<FQ_FMT_INT4>(l, a, w.group, st); break;
    case FQ_FMT_NVFP4:
      if ((l.down ? a.d : a.gu).f16) launch_one<FQ_FMT_NVFP4, kPre, true>(l, a, st);
      else launch_one<FQ_FMT_NVFP4, kPre, false>(l, a, st);
      break;
    default: launch_one<FQ_FMT_NONE, kEnd, false>(l, a, st); break;
  }
}

inline size_t up256(size_t b) { return (b + 255) / 256 * 256; }

struct TokWs {
  size_t a, span, tok, pw, total;
};
TokWs tok_ws(int T, int topk, int E, int F) {
  const size_t P = (size_t)T * topk, slots = P < (size_t)E ? P : (size_t)E;
  TokWs w;
  size_t o = 0;
  w.a = o;     o += up256(P * F * 2);
  w.span = o;  o += up256(slots * 8);
  w.tok = o;   o += up256(P * 4);
  w.pw = o;    o += up256(P * 4);
  w.total = o;
  return w;
}

}  // namespace

size_t moe_tokens_ws_bytes(int T, int topk, int E, int F) {
  return tok_ws(T, topk, E, F).total;
}

void launch_moe_tokens(const uint16_t *x, int T, int H, int F, const int32_t *ids,
                       const float *probs, int topk, int ebegin, int E, const fq_stored_w &w_gu,
                       const fq_stored_w &w_d, int afmt1, const float *as1, int afmt2,
                       const float *as2, uint16_t *out, void *ws, hipStream_t st) {
  const TokWs o = tok_ws(T, topk, E, F);
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
  a.gu = tok_stack(w_gu, 2 * F, H, afmt1);
  a.d = tok_stack(w_d, H, F, afmt2);
  a.H = H;
  a.F = F;
  a.a = reinterpret_cast<uint16_t *>(b + o.a);
  a.span = reinterpret_cast<int2 *>(b + o.span);
  a.tok = reinterpret_cast<int32_t *>(b + o.tok);
  a.pw = reinterpret_cast<float *>(b + o.pw);
  a.out = out;
  // token rows staged at a time: 16 columns of an MFMA, or what 40 KB hold
  // (three blocks to a CU), at least one
  const int chunk = chunk_of(w_gu.fmt), row = xrow_bytes(H, chunk);
  int nc = (40 << 10) / row;
  nc = nc < 1 ? 1 : nc > 16 ? 16 : nc;
  a.ncol = nc < T ? nc : T;
  a.dvpr = FastDiv((uint32_t)(a.gu.nch * (chunk / 8)));
  // channel groups per gate_up block: the most that leave four blocks to a CU
  const int groups = F / kTile;
  int mt = 4;
  while (mt > 1 && (long)a.slots * ((groups + mt - 1) / mt) < 1024) mt /= 2;
  int lds = a.ncol * row;
  if (lds < kRedBytes) lds = kRedBytes;
  launch_fmt(w_gu, {false, mt, dim3(a.slots, (groups + mt - 1) / mt), lds}, a, st);
  launch_fmt(w_d, {true, 0, dim3(H / 8), kWavesD * T * 8 * 4}, a, st);
}

}  // namespace fq
