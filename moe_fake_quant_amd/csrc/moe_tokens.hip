// One MoE layer for a few tokens (T <= 128) over the stored form of its
// weights, in two kernels on gfx950: the serving counterpart of the grouped
// GEMM path, without a decoded copy of the stacks, a permutation or a gather.
//
//   k_tok_gate_up  h = W_gu[e] FQ_a1(x),  a = silu(h_g) h_u,  A = FQ_a2(a)
//   k_tok_down     out[t] = bf16(sum_j p[t,j] W_d[e_tj] A[t,j])
//
// What bounds it: the codes of the distinct experts of the batch are read and
// everything else is small, so the floor is the weight stream from HBM; next
// come the VALU operations that turn 4-bit codes into MFMA operands. An expert
// of more rows than one pass of columns takes (16 or what fits into LDS in
// gate_up, 8 in down) has its codes loaded and decoded again for each pass.
//
// Operands are exact. A weight's grid value (E4M3, int8, int4 minus zero
// point, E2M1 times its E4M3 block scale: at most 8 significant bits) is a
// bf16 number, and so is an activation's; the fp32 scales that are constant
// over a contraction (per channel, per tensor, per 128-group, the NVFP4 tensor
// scale, s_a) multiply the fp32 sums instead. h stays in fp32.
//
// Two operands are no grid values: A without an activation format, and weights in
// groups that are no multiple of a chunk (see Fmt), whose scale enters the operand.
// Each is taken as two bf16 numbers, the value rounded and what that leaves, with
// an MFMA for either. Together they are within 2^-16 of it (half a bf16 step of half
// a bf16 step), so that the rounding of the output is the only one that counts:
// against float64 the output is off by 0.0017 (root mean squares), as with fp32
// operands. One bf16 number for A gave 0.0024, one for the weights 0.0034 and, where
// an activation quantizer follows, 0.0125 (FP8, groups of 32).
//
// Contraction: v_mfma_f32_16x16x32 (bf16, or f16: see operand) with 16 weight rows
// as the row operand and up to 16 tokens as columns. A lane loads 16 bytes of codes of its row
// at once (32 four-bit codes) and feeds them to consecutive MFMAs, so the
// contraction order is permuted, alike for both operands: a wave's load covers
// 16 rows x 64 contiguous bytes.
//
// Measured at 128 experts, H 2048, F 768, top 8 (gate_up + down, us; the bytes of
// the named experts): NVFP4, 1 token 13.5 + 5.4 (21 MB, latency); 64 tokens 61 + 41
// (226 + 109 MB: 3.7 and 2.7 TB/s); FP8, 16 tokens 53 + 31 (260 + 130 MB: 4.9 and
// 4.2 TB/s); INT4 with bf16 activations, 7 tokens 39 + 24. A 1 GiB device copy runs
// at 5.2 TB/s.
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
  kPre = 2    // other groups, NVFP4's E4M3 block scale: the operand
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
  int parts;                // bf16 numbers to an activation: 2 for A without a format, else 1
  int seg;                  // Fmt::kSeg
  FastDiv dgroup;           // / group
};

// The scales of an item's rows pass through LDS: the rows of a tile lie behind
// one another, so they are fetched in whole cache lines, where a load per lane
// and segment would touch 16 lines for a few bytes of each. A row's bytes, and
// its distance in LDS (8 more, so that a column of rows falls into different
// banks).
struct RowBytes {
  int n, stride;
  FastDiv per8, per1;  // / 8-byte units, / bytes of a row
};
inline RowBytes row_bytes(int n) {
  RowBytes r;
  r.n = n;
  r.stride = (n + 7) / 8 * 8 + 8;
  r.per8 = FastDiv((uint32_t)(n >= 8 ? n / 8 : 1));
  r.per1 = FastDiv((uint32_t)(n > 0 ? n : 1));
  return r;
}

struct TokArgs {
  const uint16_t *x;        // [T, H]
  const int32_t *ids;       // [T, topk]
  const float *probs;       // [T, topk]
  int T, topk, P, ebegin, E;
  FastDiv dtopk;
  int afmt1, afmt2;
  const float *as1, *as2;
  TokStack gu, d;
  int H, F;
  int ncol;                 // columns (tokens) staged at a time by the gate_up kernel
  int ny;                   // channel blocks of a gate_up expert
  FastDiv dny;
  FastDiv dvpr, dncol;      // / 8-element vectors of a staged token row, / ncol
  FastDiv dgrid;            // / blocks of the gate_up kernel
  int idb, xb;              // gate_up LDS: bytes of the ids, of the staged rows
  RowBytes rsc, rzp;        // gate_up: scale (or scale byte) and zero point bytes of a row
  int agroups, arow;        // A's 16-channel groups and row length, padded to whole chunks
  // workspace. Rows are the pairs in expert order.
  uint16_t *a;              // [P, arow, parts] A's grid values, expert by expert (see a_offset)
  int4 *act;                // [min(P, E)] the experts with rows: {expert, first row, rows, 0}
  int32_t *nact;            // their number
  int32_t *tok;             // [P] a row's token
  float *pw;                // [P] its weight
  uint16_t *out;
};

// ------------------------------------------------------------ weight codes --
struct Codes {
  uint32_t w[4];
};
struct Scales {  // of one segment
  uint32_t sb;   // NVFP4: the block scale bytes of its two 16-blocks
  float s0, zp;  // kPre: its scale; INT4: its zero point
};

__device__ __forceinline__ const uint8_t *row_codes(const TokStack &t, int fmt4, size_t row,
                                                    int kq) {
  const size_t bytes = fmt4 == 0 ? (size_t)t.K * 2 : fmt4 == 2 ? (size_t)t.K / 2 : (size_t)t.K;
  return t.codes + row * bytes + kq * 16;
}
template <int FMT>
__device__ __forceinline__ const uint8_t *row_codes(const TokStack &t, size_t row, int kq) {
  return row_codes(t, FMT == FQ_FMT_NONE ? 0 : Fmt<FMT>::k4bit ? 2 : 1, row, kq);
}

// The lane's segment of chunk ch of a row (p: row_codes; a chunk is 64 bytes in
// every format, 4 lane groups x 16 bytes). Past the end of the row nothing is
// read and the codes are 0 (what they meet there is 0 too).
template <int FMT, bool WHOLE>
__device__ __forceinline__ Codes load_codes(const TokStack &t, const uint8_t *p, int ch, int kq) {
  Codes r;
  p += ch * 64;
  if (WHOLE) {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    return r;
  }
  const int k0 = ch * Fmt<FMT>::kChunk + kq * Fmt<FMT>::kSeg;
  r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
  if (k0 >= t.K) return r;
  if (Fmt<FMT>::k4bit && (t.K & 31)) {
    // rows are multiples of 8 bytes, the last segment may hold 16 codes
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    r.w[0] = v.x; r.w[1] = v.y;
    if (k0 + 16 < t.K) {
      const uint2 u = *reinterpret_cast<const uint2 *>(p + 8);
      r.w[2] = u.x; r.w[3] = u.y;
    }
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(p);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  }
  return r;
}

// Does a format and mode have scales (sb or s0) / zero points per segment?
template <int FMT, int MODE>
struct Has {
  static constexpr bool kSb = FMT == FQ_FMT_NVFP4;
  static constexpr bool kS = FMT != FQ_FMT_NONE && FMT != FQ_FMT_NVFP4 && MODE != kEnd;
  static constexpr bool kZp = FMT == FQ_FMT_INT4;
};

// bf16 numbers to a weight
template <int FMT, int MODE>
constexpr int weight_parts() { return MODE == kPre && FMT != FQ_FMT_NVFP4 ? 2 : 1; }
template <int N>
struct Operand {
  bf16x8_t p[N];
};

// The row operand of step st of a chunk: 8 consecutive elements of the lane's row
// (bf16, or f16 with F16).
//
// VALU operations per 8 codes: E4M3 4 (the converter makes bf16 pairs), NVFP4
// 8 in f16 (convert and multiply pairs by the block scale) or 16 through fp32
// in bf16, int4 23, int8 about 16, and 20 more for two parts. f16 holds every
// NVFP4, E4M3 and int8 grid value exactly (at most 8 bits, 2^-10 <= |v| <= 2688),
// but not any bf16 activation, so it is used for quantized activations.
template <int FMT, int MODE, bool F16>
__device__ __forceinline__ Operand<weight_parts<FMT, MODE>()> operand(const Codes &r,
                                                                      const Scales &q, int st) {
  constexpr int kParts = weight_parts<FMT, MODE>();
  Operand<kParts> o;
  if (FMT == FQ_FMT_NVFP4 && F16) {
    const uint32_t c = r.w[st];
    const f16x2 th = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(q.sb, 1.0f, false);
    const _Float16 s = st < 2 ? th.x : th.y;
    const f16x2 ss = {s, s};
    f16x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 0) * ss;
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 1) * ss;
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 2) * ss;
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, 1.0f, 3) * ss;
    o.p[0] = __builtin_bit_cast(bf16x8_t, v);
    return o;
  }
  if (FMT == FQ_FMT_NONE) {
    o.p[0] = {{r.w[0], r.w[1], r.w[2], r.w[3]}};
  } else if (FMT == FQ_FMT_FP8_E4M3 && MODE != kPre) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t c = r.w[2 * st + h];
      o.p[0].w[2 * h] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
      o.p[0].w[2 * h + 1] = __builtin_bit_cast(
          uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
    }
  } else {
    float v[8];
    if (FMT == FQ_FMT_NVFP4) {
      const uint32_t c = r.w[st];
      const f32x2_t th = __builtin_amdgcn_cvt_pk_f32_fp8(q.sb, false);
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
        v[2 * j] = (float)((ev >> (8 * j)) & 0xFFu) - q.zp;
        v[2 * j + 1] = (float)((od >> (8 * j)) & 0xFFu) - q.zp;
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
      for (int j = 0; j < 8; ++j) v[j] = v[j] * q.s0;
    }
    o.p[0] = pack8(v);
    if constexpr (kParts == 2) {
      float f[8];
      unpack8(o.p[0], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] -= f[j];
      o.p[1] = pack8(v);
    }
  }
  return o;
}

// acc plus the products of a row operand and 8 activation values of its type.
// Both in two parts: three products, the rests' own is below 2^-16 of the whole.
template <bool F16>
__device__ __forceinline__ f32x4 mfma(const bf16x8_t &o, const bf16x8_t &x, f32x4 acc) {
  if (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, o),
                                                  __builtin_bit_cast(f16x8v, x), acc, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, o),
                                                 __builtin_bit_cast(bf16x8v, x), acc, 0, 0, 0);
}
template <bool F16, int WP, int XP>
__device__ __forceinline__ f32x4 mfma(const Operand<WP> &o, const bf16x8_t (&x)[XP], f32x4 acc) {
#pragma unroll
  for (int h = 0; h < XP; ++h) acc = mfma<F16>(o.p[0], x[h], acc);
  if constexpr (WP == 2) acc = mfma<F16>(o.p[1], x[0], acc);
  return acc;
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
constexpr float kBf16Max = 0x1.FEp127f;
constexpr int kRedBytes = kWaves * 2 * 64 * 16;  // the waves' sums of their two tiles

// bytes of one staged token row: the row padded to whole chunks, and 16 more
// so that the 16 columns of a fragment read fall into different LDS banks
__host__ __device__ inline int xrow_bytes(int K, int chunk) {
  return (K + chunk - 1) / chunk * chunk * 2 + 16;
}

extern __shared__ __attribute__((aligned(16))) char g_tok_lds[];

// A barrier for data in LDS. (__syncthreads also waits for every global load in
// flight, which would end each request made ahead of a barrier: measured 2-4 us
// a barrier here.)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// v, but not known to be the same each time: index arithmetic made from it is
// done again where it is used, instead of being kept in registers over the
// contraction loop (which then spill).
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The plan of a batch, made by every gate_up block for itself (it costs less
// than waiting for another kernel): rows = the local pairs in expert order,
// within an expert in pair order, a pair that repeats an expert of its token
// left to the first one (which takes the summed weight).
constexpr uint16_t kNoId = 0x7FFF;   // not local
constexpr uint16_t kRepeat = 0x8000;
struct Plan {
  int cnt[1024];       // rows of an expert
  uint16_t off[1024];  // its first row
  uint16_t act[1024];  // the experts with rows, ascending
  uint16_t pass[1025]; // column passes (of ncol rows) of the experts before
  uint32_t wsum[kWaves], psum[kWaves];
  int32_t tok[128];    // tokens of the current expert's rows
  int32_t pair[128];   // their pairs
  int wcnt[kWaves];
  int it[2];
};

// ids: LDS, P entries: the pair's local expert | kRepeat. Returns the number of
// experts with rows.
__device__ __forceinline__ int make_plan(const TokArgs &a, Plan &p, uint16_t *ids) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int q = tid; q < a.P; q += kNT) {
    const uint32_t id = (uint32_t)a.ids[q] - (uint32_t)a.ebegin;  // wraps, never overflows
    ids[q] = id < (uint32_t)a.E ? (uint16_t)id : kNoId;
  }
  for (int e = tid; e < a.E; e += kNT) p.cnt[e] = 0;
  lds_barrier();
  uint32_t repeat = 0;  // one bit per pair of this thread (P <= 128 * 64 = 16 kNT)
  for (int q = tid, k = 0; q < a.P; q += kNT, ++k) {
    const uint16_t id = ids[q];
    if (id == kNoId) continue;
    bool again = false;
    for (int i = (int)a.dtopk.div((uint32_t)q) * a.topk; i < q; ++i) again |= ids[i] == id;
    if (again) repeat |= 1u << k;
    else atomicAdd(&p.cnt[id], 1);
  }
  lds_barrier();
  for (int q = tid, k = 0; q < a.P; q += kNT, ++k)
    if ((repeat >> k) & 1u) ids[q] |= kRepeat;
  // prefix sums over the experts, rows in the low half, experts with rows in the high
  uint32_t run = 0, prun = 0;
  for (int e0 = 0; e0 < a.E; e0 += kNT) {
    const int e = e0 + tid;
    const int c = e < a.E ? p.cnt[e] : 0;
    const uint32_t v = (uint32_t)c | (c > 0 ? 0x10000u : 0u);
    const uint32_t u = a.dncol.div((uint32_t)(c + a.ncol - 1));
    uint32_t x = v, z = u;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t xo = __shfl_up(x, o, 64), zo = __shfl_up(z, o, 64);
      if (lane >= o) {
        x += xo;
        z += zo;
      }
    }
    if (lane == 63) {
      p.wsum[wave] = x;
      p.psum[wave] = z;
    }
    lds_barrier();
    uint32_t base = run, pbase = prun;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) {
        base += p.wsum[w];
        pbase += p.psum[w];
      }
      run += p.wsum[w];
      prun += p.psum[w];
    }
    if (c > 0) {
      const uint32_t ex = base + x - v;
      p.off[e] = (uint16_t)(ex & 0xFFFFu);
      p.act[ex >> 16] = (uint16_t)e;
      p.pass[ex >> 16] = (uint16_t)(pbase + z - u);
    }
    if (tid == 0) p.pass[run >> 16] = (uint16_t)prun;
    lds_barrier();
  }
  return (int)(run >> 16);
}

// This block's items: those that begin in its share of the passes (an
// expert's items count its passes each, so that a hot expert's weigh as much as
// they take).
__device__ __forceinline__ void my_items(const TokArgs &a, Plan &p, int na, int &it0, int &it1) {
  const uint32_t total = (uint32_t)p.pass[na] * a.ny;
  const uint32_t share = a.dgrid.div(total), rest = total - share * gridDim.x;
  const int tid = threadIdx.x;
  if (p.pass[na] == na) {  // every expert takes one pass: an item is a pass
    it0 = (int)(blockIdx.x * share + min(blockIdx.x, rest));
    it1 = (int)((blockIdx.x + 1) * share + min(blockIdx.x + 1, rest));
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t b = blockIdx.x + h, at = b * share + min(b, rest);
    for (int sl = tid; sl < na; sl += kNT) {
      const uint32_t p0 = p.pass[sl], n = p.pass[sl + 1] - p0;
      if (at >= p0 * a.ny && at < (p0 + n) * a.ny)
        p.it[h] = sl * a.ny + (int)((at - p0 * a.ny + n - 1) / n);
    }
    if (tid == 0 && at == total) p.it[h] = na * a.ny;
  }
  lds_barrier();
  it0 = __builtin_amdgcn_readfirstlane(p.it[0]);
  it1 = __builtin_amdgcn_readfirstlane(p.it[1]);
}

// The tokens and pairs of expert e's rows.
__device__ __forceinline__ void list_rows(const TokArgs &a, Plan &p, const uint16_t *ids, int e) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int n = 0;
  for (int q0 = 0; q0 < a.P; q0 += kNT) {
    const int q = q0 + tid;
    const bool hit = q < a.P && ids[q] == (uint16_t)e;
    const uint64_t m = __ballot(hit);
    if (lane == 0) p.wcnt[wave] = __popcll(m);
    lds_barrier();
    int base = n;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += p.wcnt[w];
      n += p.wcnt[w];
    }
    if (hit) {
      const int i = base + __popcll(m & ((1ull << lane) - 1ull));
      p.tok[i] = (int)a.dtopk.div((uint32_t)q);
      p.pair[i] = q;
    }
    lds_barrier();
  }
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

// A's order. Channel f of a row comes at a_index(f): within a chunk of the down
// projection the 32 elements of one MFMA step (4 lane groups x 8) are contiguous.
// Such a piece of 64 bytes lies beside the same piece of the expert's other rows
// (element i of piece p of row r: (p * rows + r) * 32 + i), so that a step's
// operand is one contiguous stretch of rows * 64 bytes: a load's time goes with
// the cache lines it touches. With two parts to an element, a row's piece is its
// 32 rounded values and behind them the 32 rests.
template <int SEG>
__device__ __forceinline__ int a_index(int f) {
  const int in = f & (4 * SEG - 1);
  return (f - in) + (in & (SEG - 1)) / 8 * 32 + in / SEG * 8 + (in & 7);
}
__device__ __forceinline__ size_t a_offset(int seg, int parts, int f, int row, int rows) {
  const int i = seg == 32 ? a_index<32>(f) : seg == 16 ? a_index<16>(f) : f;
  return ((size_t)(i >> 5) * rows + row) * (32 * parts) + (i & 31);
}

// An item is MT x 16 channels of A for one expert and its tokens; a block takes
// a contiguous share of the items in (expert, channels) order, so it stages an
// expert's tokens once and streams the weights of several items past them. Its
// eight waves are MT channel groups (gate and up rows of the same 16 channels)
// times 8 / MT shares of the contraction. The first weights of an item are
// requested before the sums of the one before are added up. (One block per item
// with a plan and staging of its own took 98 us where this takes 61: 64 tokens,
// NVFP4, 227 MB. A launch for one token, all latency, takes 13.5 us.)
template <int FMT, int MODE, bool F16, bool WHOLE, int MT>
__global__ __launch_bounds__(kNT, 4) void k_tok_gate_up(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr bool kSb = Has<FMT, MODE>::kSb, kS = Has<FMT, MODE>::kS, kZp = Has<FMT, MODE>::kZp;
  constexpr int kWK = kWaves / MT;
  constexpr int kU = 2;   // chunks of a batch; one batch computes while the next loads
  constexpr int kX = 2;   // token vectors a thread has in flight
  constexpr int kOut = (MT * 256 + kNT - 1) / kNT;  // channels x columns per thread
  __shared__ Plan plan;
  __shared__ float rsl[2 * MT * kTile];  // factors of the item's rows
  uint16_t *ids = reinterpret_cast<uint16_t *>(g_tok_lds);
  char *xrows = g_tok_lds + a.idb;
  // scales and zero points of the item's rows (MT * 16 gate rows, then the up
  // rows); the waves' sums take their space once they are used
  char *scl = g_tok_lds + a.idb + a.xb;
  f32x4 *red = reinterpret_cast<f32x4 *>(scl);
  char *zpl = scl + (kSb || kS ? 2 * MT * kTile * a.rsc.stride : 0);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: scalar loop control
  const TokStack &w = a.gu;
  const ActQ q1 = load_actq(a.afmt1, a.as1), q2 = load_actq(a.afmt2, a.as2);

  const int na = __builtin_amdgcn_readfirstlane(make_plan(a, plan, ids));
  if (blockIdx.x == 0) {
    if (tid == 0) a.nact[0] = na;
    for (int i = tid; i < na; i += kNT) {
      const int e = plan.act[i];
      a.act[i] = make_int4(e, plan.off[e], plan.cnt[e], 0);
    }
  }
  if (na == 0) return;
  int it0, it1;
  my_items(a, plan, na, it0, it1);
  if (it0 >= it1) return;

  const float rg1 = 1.0f / (6.0f * q1.s), rg2 = 1.0f / (6.0f * q2.s);
  const int xstride = xrow_bytes(w.K, kChunk);
  const int col = lane & 15, kq = lane >> 4;
  const int wm = wave / kWK, wk = wave % kWK;
  const int vpr = w.nch * kChunk / 8, live = w.K / 8;

  Codes raw[2][kU][2];
  const uint8_t *pg = nullptr, *pu = nullptr;
  int nch = 0;
  auto point = [&](int it) {  // this wave's rows of an item (none past F)
    const int sl = (int)a.dny.div((uint32_t)it);
    const int f0 = ((it - sl * a.ny) * MT + wm) * kTile;
    nch = f0 < a.F ? w.nch : 0;
    const size_t row0 =
        (size_t)__builtin_amdgcn_readfirstlane(plan.act[sl]) * w.N + (f0 < a.F ? f0 : 0);
    const size_t row = row0 + col;
    pg = row_codes<FMT>(w, row, kq);
    pu = row_codes<FMT>(w, row + a.F, kq);
  };
  auto load = [&](Codes (&r)[kU][2], int cb) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (cb + u < nch) {
        r[u][0] = load_codes<FMT, WHOLE>(w, pg, cb + u, kq);
        r[u][1] = load_codes<FMT, WHOLE>(w, pu, cb + u, kq);
      }
  };
  // Rows of n bytes (a multiple of 8) are copied in 8-byte units: unit i of an
  // item is unit i - r * n / 8 of its row r. Rows past F are left out.
  const uint8_t *sbase = kSb ? w.sbytes : reinterpret_cast<const uint8_t *>(w.scale);
  auto item_row = [&](int it, int r, size_t &row) {
    const int sl = (int)a.dny.div((uint32_t)it);
    const int f0 = (it - sl * a.ny) * MT * kTile, half = r >= MT * kTile;
    const int f = f0 + r - half * MT * kTile;
    row = (size_t)__builtin_amdgcn_readfirstlane(plan.act[sl]) * w.N + half * a.F + f;
    return f < a.F;
  };
  const int units = a.rsc.n % 8 == 0 ? 2 * MT * kTile * (a.rsc.n / 8) : 0;
  constexpr int kPf = kSb || kS ? 4 : 1;  // units a thread requests ahead
  uint2 pf[kPf];
  float rsv = 0.0f;
  // what an item needs besides its codes, requested before them: loads return in order
  auto request = [&](int it) {
    const int tid = anew(threadIdx.x);
    if (kSb || kS) {
#pragma unroll
      for (int j = 0; j < kPf; ++j) {
        const int i = tid + j * kNT;
        const int r = (int)a.rsc.per8.div((uint32_t)i), o = (i - r * (a.rsc.n / 8)) * 8;
        size_t row;
        if (i < units && item_row(it, r, row))
          pf[j] = *reinterpret_cast<const uint2 *>(sbase + row * a.rsc.n + o);
      }
    }
    size_t row;
    if (tid < 2 * MT * kTile && item_row(it, tid, row)) {
      const int sl = (int)a.dny.div((uint32_t)it);
      rsv = row_scale<FMT, MODE>(w, plan.act[sl], row);
    }
  };
  auto store_scales = [&](int it, bool requested) {
    const int tid = anew(threadIdx.x);
    if (requested && tid < 2 * MT * kTile) rsl[tid] = rsv;
    if (kSb || kS) {
      if (requested) {
#pragma unroll
        for (int j = 0; j < kPf; ++j) {
          const int i = tid + j * kNT;
          const int r = (int)a.rsc.per8.div((uint32_t)i), o = (i - r * (a.rsc.n / 8)) * 8;
          if (i < units) *reinterpret_cast<uint2 *>(scl + r * a.rsc.stride + o) = pf[j];
        }
      }
      for (int i = tid + (requested ? kPf * kNT : 0); i < units; i += kNT) {
        const int r = (int)a.rsc.per8.div((uint32_t)i), o = (i - r * (a.rsc.n / 8)) * 8;
        size_t row;
        if (item_row(it, r, row))
          *reinterpret_cast<uint2 *>(scl + r * a.rsc.stride + o) =
              *reinterpret_cast<const uint2 *>(sbase + row * a.rsc.n + o);
      }
      if (units == 0)  // rows of an odd number of 4-byte scales or of single bytes
        for (int i = tid; i < 2 * MT * kTile * a.rsc.n; i += kNT) {
          const int r = (int)a.rsc.per1.div((uint32_t)i), o = i - r * a.rsc.n;
          size_t row;
          if (item_row(it, r, row))
            scl[r * a.rsc.stride + o] = (char)sbase[row * a.rsc.n + o];
        }
    }
    if (kZp)
      for (int i = tid; i < 2 * MT * kTile * a.rzp.n; i += kNT) {
        const int r = (int)a.rzp.per1.div((uint32_t)i), o = i - r * a.rzp.n;
        size_t row;
        if (item_row(it, r, row)) zpl[r * a.rzp.stride + o] = (char)w.zp[row * a.rzp.n + o];
      }
  };
  // one segment's scales from LDS (r: the row in the item)
  auto scales = [&](int r, int ch) {
    Scales q;
    const int k0 = ch * kChunk + kq * kSeg;
    if (kSb) {
      const char *p = scl + r * a.rsc.stride + ch * 8 + kq * 2;
      if (WHOLE) {
        q.sb = *reinterpret_cast<const uint16_t *>(p);
      } else {
        q.sb = k0 < w.K ? (uint32_t)(uint8_t)p[0] : 0u;
        if (k0 + 16 < w.K) q.sb |= (uint32_t)(uint8_t)p[1] << 8;
      }
    }
    if (kZp || (kS && MODE == kPre)) {
      const int gi = (int)w.dgroup.div((uint32_t)min(k0, w.K - 1));
      if (kS && MODE == kPre) q.s0 = *reinterpret_cast<const float *>(scl + r * a.rsc.stride + gi * 4);
      if (kZp) q.zp = (float)(uint8_t)zpl[r * a.rzp.stride + gi];
    }
    return q;
  };
  auto chunk_scales = [&](int r, int ch) {  // kPost: of the four rows of a result that a lane holds
    const int gi = (int)w.dgroup.div((uint32_t)(ch * kChunk));
    f32x4 s;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s[i] = *reinterpret_cast<const float *>(scl + (r + 4 * kq + i) * a.rsc.stride + gi * 4);
    return s;
  };

  // A turn computes pass (it, c0), requests what the next one needs, and adds
  // the shares' sums up while that arrives; the first turn only requests.
  int cur = -1, staged = -1;  // the listed expert, the column group in LDS
  int it = it0, c0 = -1;
  while (true) {
    const bool run = c0 >= 0;
    const int sl = (int)a.dny.div((uint32_t)it), y = it - sl * a.ny;
    const int e = __builtin_amdgcn_readfirstlane(plan.act[sl]);
    const int n = __builtin_amdgcn_readfirstlane(plan.cnt[e]);
    const int off = __builtin_amdgcn_readfirstlane(plan.off[e]);
    f32x4 acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (run) {
      if (sl != cur) {
        list_rows(a, plan, ids, e);
        cur = sl;
        staged = -1;
      }
      store_scales(it, c0 == 0);
      const int nc = min(a.ncol, n - c0), nvec = nc * vpr;
      // ---- the tokens' grid values into LDS, a row's vectors beyond K zero
      // (vpr is even: both lanes of a 16-block take part together)
      if (staged != c0) {
        const int tid = anew(threadIdx.x);
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
              xv[j] = reinterpret_cast<const bf16x8_t *>(a.x + (size_t)plan.tok[c0 + c] * w.K)[v];
          }
#pragma unroll
          for (int j = 0; j < kX; ++j)
            if (dst[j] >= 0)
              *reinterpret_cast<bf16x8_t *>(xrows + dst[j]) = stage_vec<F16>(q1, xv[j], rg1);
        }
        staged = c0;
      }
      lds_barrier();

      // ---- this wave's chunks of the contraction, two batches of loads in turn
      const char *xs = xrows + min(col, nc - 1) * xstride + kq * kSeg * 2;
      const int rg = wm * kTile, ru = (MT + wm) * kTile;
      auto compute = [&](Codes (&r)[kU][2], int cb) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int ch = cb + u;
          if (ch >= nch) break;
          const Scales qg = scales(rg + col, ch), qu = scales(ru + col, ch);
          f32x4 s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
          if (MODE != kPost) {
            s0 = acc[0];
            s1 = acc[1];
          }
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const bf16x8_t b[1] = {
                *reinterpret_cast<const bf16x8_t *>(xs + (ch * kChunk + st * 8) * 2)};
            s0 = mfma<F16>(operand<FMT, MODE, F16>(r[u][0], qg, st), b, s0);
            s1 = mfma<F16>(operand<FMT, MODE, F16>(r[u][1], qu, st), b, s1);
          }
          if (MODE == kPost) {
            acc[0] += s0 * chunk_scales(rg, ch);
            acc[1] += s1 * chunk_scales(ru, ch);
          } else {
            acc[0] = s0;
            acc[1] = s1;
          }
        }
      };
      for (int cb = wk * kU; cb < nch; cb += 2 * kU * kWK) {
        load(raw[1], cb + kU * kWK);
        compute(raw[0], cb);
        load(raw[0], cb + 2 * kU * kWK);
        compute(raw[1], cb + kU * kWK);
      }
    }
    // the next pass: this item's next columns, or the next item
    const int nit = !run || c0 + a.ncol < n ? it : it + 1;
    const int nc0 = run && nit == it ? c0 + a.ncol : 0;
    if (nit < it1) {
      if (nc0 == 0) {
        point(nit);
        request(nit);
      }
      load(raw[0], wk * kU);
    }
    if (run) {
      const int nc = min(a.ncol, n - c0);
      if (y == 0 && c0 == 0 && tid < n) {  // what the down kernel needs of this expert's rows
        const int q = plan.pair[tid], t = plan.tok[tid];
        float v = a.probs[q];
        for (int j = q + 1; j < (t + 1) * a.topk; ++j)
          if (ids[j] == (uint16_t)(e | kRepeat)) v += a.probs[j];
        a.tok[off + tid] = t;
        a.pw[off + tid] = v;
      }
      // ---- the shares' sums, SwiGLU, FQ_a2. Each wave holds its group's tiles.
      lds_barrier();
      red[(wave * 2 + 0) * 64 + lane] = acc[0];
      red[(wave * 2 + 1) * 64 + lane] = acc[1];
      lds_barrier();
      // channel f of column c: 16 consecutive lanes hold a group's 16 channels
      const int tid_e = anew(threadIdx.x);
#pragma unroll
      for (int j = 0; j < kOut; ++j) {
        const int i = tid_e + j * kNT;
        const int m = i >> 8, f = i & 15, c = (i >> 4) & 15;
        const int g = y * MT + m;  // past F: the zero tail of A's row
        if (i >= MT * 256 || g >= a.agroups) continue;  // whole groups of 16 lanes
        const int idx = ((f >> 2) * 16 + c) * 4 + (f & 3);
        const float *rf = reinterpret_cast<const float *>(red) + m * kWK * 512;
        float hg = 0.0f, hu = 0.0f;
#pragma unroll
        for (int k = 0; k < kWK; ++k) {
          hg += rf[k * 512 + idx];
          hu += rf[k * 512 + 256 + idx];
        }
        hg = hg * rsl[m * kTile + f] * q1.s;
        hu = hu * rsl[(MT + m) * kTile + f] * q1.s;
        float av[2] = {hg * sigmoid_hw(hg) * hu, 0.0f};
        float theta = 0.0f;
        if (q2.fmt == FQ_FMT_NVFP4) {
          float amax = fabsf(av[0]);
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, 64));
          theta = block_theta(amax, rg2);
        }
        act_grid<2>(q2, theta, av);
        uint32_t v = a.d.f16 ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(av[0], 0.0f))
                             : f32_to_bf16(fminf(fmaxf(av[0], -kBf16Max), kBf16Max));
        // what v leaves of A (a NaN or infinity: itself)
        uint32_t rest = f32_to_bf16(av[0] - bf16_to_f32(v));
        if (g * kTile >= a.F) v = rest = 0u;
        if (c < nc) {
          uint16_t *to = a.a + (size_t)off * a.arow * a.d.parts +
                         a_offset(a.d.seg, a.d.parts, g * kTile + f, c0 + c, n);
          to[0] = (uint16_t)v;
          if (a.d.parts == 2) to[32] = (uint16_t)rest;
        }
      }
      lds_barrier();
    }
    if (nit >= it1) break;
    it = nit;
    c0 = nc0;
  }
}

// ------------------------------------------------------------------- down ---
// A block forms 8 output columns of every token, over all experts: nothing is
// shared between blocks. An MFMA's 16 weight rows are the same 8 rows of two
// experts and its 16 columns up to 8 tokens of each; the two diagonal blocks of
// the result are used (the MFMAs have time to spare, the weights are decoded
// once either way). A wave takes units (two experts, part of the contraction)
// in turn and adds their weighted sums to its own [T, 8] block in LDS; the
// waves' blocks are added in wave order. (Splitting the experts over blocks, the
// last one adding the parts, cost 40 us in device-wide fences alone.) Bound by its
// gather loads: 64 tokens took 47 us with A row by row, 34 without the A loads, 33
// without the weight loads, and 40 with A in its present order. H / 8 blocks are one
// round of the CUs at H = 2048; narrower layers leave CUs idle.
template <int FMT, int MODE, bool F16, bool WHOLE, int PARTS>
__global__ __launch_bounds__(kNTd) void k_tok_down(TokArgs a) {
  constexpr int kChunk = Fmt<FMT>::kChunk, kSeg = Fmt<FMT>::kSeg, kSteps = Fmt<FMT>::kSteps;
  constexpr bool kSb = Has<FMT, MODE>::kSb, kS = Has<FMT, MODE>::kS, kZp = Has<FMT, MODE>::kZp;
  // chunks whose codes are requested together (4 of int4 in two parts would spill: 141 us
  // where 2 take 138, 16 tokens in groups of 32)
  constexpr int kU = FMT == FQ_FMT_INT4 && MODE == kPre ? 2 : 4;
  // chunks whose activations are: 32 registers of them
  constexpr int kB = FMT == FQ_FMT_NONE ? 4 : (Fmt<FMT>::k4bit ? 2 : 4) / PARTS;
  __shared__ int4 act[1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 8;
  const TokStack &w = a.d;
  const ActQ q2 = load_actq(a.afmt2, a.as2);
  float *accs = reinterpret_cast<float *>(g_tok_lds);  // [wave][T][8]
  const int na = a.nact[0];
  if (tid < min(a.P, a.E)) act[tid] = a.act[tid];  // behind na: stale, not used
  for (int i = tid; i < kWavesD * a.T * 8; i += kNTd) accs[i] = 0.0f;
  lds_barrier();

  const int nch = w.nch;
  const int col = lane & 15, kq = lane >> 4;
  const int pairs = (na + 1) / 2;
  // parts of a contraction (whole pairs of chunks), so that few experts still
  // occupy every wave
  int kp = pairs > 0 ? kWavesD / pairs : 1;
  kp = max(1, min(kp, (nch + 1) / 2));
  const int per = ((nch + kp - 1) / kp + 1) / 2 * 2;

  // Where a wave stands: unit u (two experts, a part of the contraction), the
  // batch of chunks from cb on, the columns from c0 on. Without a second expert
  // its lanes repeat the first: their part of the result is not used.
  struct At {
    int u, cb, ch0, ch1, c0, nmax, i0, i1;
    size_t row;        // the lane's weight row
    const uint8_t *p;  // its codes
  };
  auto enter = [&](At &t) {
    if (t.u >= pairs * kp) return;
    const int pr = t.u / kp, part = t.u - pr * kp;
    t.ch0 = t.cb = part * per;
    t.ch1 = min(nch, t.ch0 + per);
    t.c0 = 0;
    t.i0 = 2 * pr;
    t.i1 = min(2 * pr + 1, na - 1);
    t.nmax = max(__builtin_amdgcn_readfirstlane(act[t.i0].z),
                 __builtin_amdgcn_readfirstlane(act[t.i1].z));
    t.row = (size_t)act[(col >> 3) ? t.i1 : t.i0].x * w.N + n0 + (col & 7);
    t.p = row_codes<FMT>(w, t.row, kq);
  };
  struct Batch {
    Codes c[kU];
    uint2 sb[kU];  // NVFP4: the chunk's eight block scale bytes of the lane's row
    float s[kU];   // kS: the segment's scale (kPost: the chunk's)
    uint8_t zp[kU];
  };
  auto load = [&](Batch &r, const At &t) {
    const uint8_t *ps = w.sbytes + t.row * (size_t)(w.K >> 4) + t.cb * 8;
    // rows of whole pairs of chunks: both chunks' scale bytes in one load
    const bool wide = WHOLE && kSb && (w.K & 255) == 0;
    if (wide) {
#pragma unroll
      for (int i = 0; i < kU; i += 2)
        if (t.cb + i < t.ch1) {
          const uint4 v = *reinterpret_cast<const uint4 *>(ps + i * 8);
          r.sb[i] = make_uint2(v.x, v.y);
          r.sb[i + 1] = make_uint2(v.z, v.w);
        }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (t.cb + i < t.ch1) {
        r.c[i] = load_codes<FMT, WHOLE>(w, t.p, t.cb + i, kq);
        if (kSb && !wide) {
          if (WHOLE) {
            r.sb[i] = *reinterpret_cast<const uint2 *>(ps + i * 8);
          } else {
            const int k0 = (t.cb + i) * kChunk + kq * kSeg;
            const uint8_t *b = ps + i * 8 + kq * 2;
            uint32_t v = k0 < w.K ? (uint32_t)b[0] : 0u;
            if (k0 + 16 < w.K) v |= (uint32_t)b[1] << 8;
            v <<= (kq & 1) * 16;  // where the others have it
            r.sb[i] = make_uint2(v, v);
          }
        }
        if (kS || kZp) {
          const int k0 = (t.cb + i) * kChunk + (MODE == kPost ? 0 : kq * kSeg);
          const size_t gi = t.row * w.groups + w.dgroup.div((uint32_t)min(k0, w.K - 1));
          if (kS) r.s[i] = w.scale[gi];
          if (kZp) r.zp[i] = w.zp[gi];
        }
      }
  };

  f32x4 acc = {0, 0, 0, 0};
  f32x4 rs = {1, 1, 1, 1};  // factors of the four rows of the result a lane holds
  int tok = 0;              // its column's token and weight
  float p = 0.0f;
  // One batch: its activation rows are requested first, then the next batch's
  // weights, which are on their way while this one computes.
  auto step = [&](Batch &r, Batch &rn, At &t) {
    const int4 ac = act[(col >> 3) ? t.i1 : t.i0], ar = act[(kq >> 1) ? t.i1 : t.i0];
    // a column past the expert's last repeats it, and is not used
    const int row_e = min(t.c0 + (col & 7), ac.z - 1), row_a = ac.y + row_e;
    if (t.cb == t.ch0) {
      const size_t row_r = (size_t)ar.x * w.N + n0 + 4 * (kq & 1);
      acc = {0, 0, 0, 0};
      tok = a.tok[row_a];
      p = a.pw[row_a];
#pragma unroll
      for (int i = 0; i < 4; ++i) rs[i] = row_scale<FMT, MODE>(w, ar.x, row_r + i);
    }
    const uint16_t *ap = a.a + ((size_t)ac.y * a.arow + row_e * 32) * PARTS + kq * 8;
    const int piece = ac.z * 32 * PARTS;  // elements from a step to the next
    bf16x8_t b[kB][kSteps][PARTS];
    auto load_b = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kB; ++i)
        if (t.cb + i0 + i < t.ch1) {
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int h = 0; h < PARTS; ++h)
              b[i][st][h] = *reinterpret_cast<const bf16x8_t *>(
                  ap + (uint32_t)(((t.cb + i0 + i) * kSteps + st) * piece) + h * 32);
        }
    };
    load_b(0);
    At nx = t;
    nx.cb += kU;
    if (nx.cb >= nx.ch1) {
      nx.cb = nx.ch0;
      nx.c0 += 8;
      if (nx.c0 >= nx.nmax) {
        nx.u += kWavesD;
        enter(nx);
      }
    }
    if (nx.u < pairs * kp) load(rn, nx);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      if (t.cb + i >= t.ch1) break;
      if (i > 0 && i % kB == 0) load_b(i);
      Scales q;
      if (kSb) q.sb = (((kq >> 1) ? r.sb[i].y : r.sb[i].x) >> ((kq & 1) * 16)) & 0xFFFFu;
      if (kS) q.s0 = r.s[i];
      if (kZp) q.zp = (float)r.zp[i];
      f32x4 s = {0, 0, 0, 0};
      if (MODE != kPost) s = acc;
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
        s = mfma<F16>(operand<FMT, MODE, F16>(r.c[i], q, st), b[i % kB][st], s);
      if (MODE == kPost) {
        // weight row 4 kq + i of the result is lane 4 kq + i's row
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += s[j] * __shfl(r.s[i], 4 * kq + j, 64);
      } else {
        acc = s;
      }
    }
    if (t.cb + kU >= t.ch1) {  // these columns' sums are complete
      const bool live_c = 2 * (t.u / kp) + (col >> 3) < na && t.c0 + (col & 7) < ac.z;
      const float ps = p * q2.s;
      const f32x4 v = acc * rs * ps;
      // a token may be in both experts' columns: one expert's lanes after the
      // other's (a wave's LDS accesses execute in order)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (live_c && (col >> 3) == h && (kq >> 1) == h) {
          f32x4 *dst =
              reinterpret_cast<f32x4 *>(accs + ((size_t)wave * a.T + tok) * 8 + 4 * (kq & 1));
          *dst += v;
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
      }
    }
    t = nx;
  };

  At t;
  t.u = wave;
  if (t.u < pairs * kp) {
    Batch r0, r1;
    enter(t);
    load(r0, t);
    while (true) {
      step(r0, r1, t);
      if (t.u >= pairs * kp) break;
      step(r1, r0, t);
      if (t.u >= pairs * kp) break;
    }
  }
  lds_barrier();

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
  t.seg = chunk / 4;
  t.f16 = w.fmt == FQ_FMT_NVFP4 && afmt != FQ_FMT_NONE;
  t.parts = afmt == FQ_FMT_NONE ? 2 : 1;
  t.dgroup = FastDiv((uint32_t)group);
  return t;
}

// channel groups per gate_up item where rows end inside a chunk: this many, or one
// where the scales of its 64 rows do not fit into LDS
constexpr int kMtTail = 2;
constexpr int kLdsBytes = 160 << 10;
constexpr int kPlanBytes = sizeof(Plan) + 2 * 4 * kTile * sizeof(float);  // and the rows' factors

struct Launch {
  bool down;
  int mt;  // channel groups per gate_up block
  dim3 grid;
  int lds;
};

template <int FMT, int MODE, bool F16, bool WHOLE>
void launch_down(const Launch &l, const TokArgs &a, hipStream_t st) {
  // NVFP4 goes through f16 with an activation format and through bf16 without
  constexpr bool kOne = F16 || FMT != FQ_FMT_NVFP4, kTwo = !F16;
  if constexpr (kOne)
    if (a.d.parts == 1)
      hipLaunchKernelGGL((k_tok_down<FMT, MODE, F16, WHOLE, 1>), l.grid, dim3(kNTd), l.lds, st, a);
  if constexpr (kTwo)
    if (a.d.parts == 2)
      hipLaunchKernelGGL((k_tok_down<FMT, MODE, F16, WHOLE, 2>), l.grid, dim3(kNTd), l.lds, st, a);
}
template <int FMT, int MODE, bool F16, bool WHOLE, int MT>
void launch_gate_up(const Launch &l, const TokArgs &a, hipStream_t st) {
  hipLaunchKernelGGL((k_tok_gate_up<FMT, MODE, F16, WHOLE, MT>), l.grid, dim3(kNT), l.lds, st, a);
}

template <int FMT, int MODE, bool F16>
void launch_one(const Launch &l, const TokArgs &a, hipStream_t st) {
  // groups of whole chunks make rows of whole chunks
  if constexpr (MODE != kPost) {
    if (l.down && !a.d.whole) return launch_down<FMT, MODE, F16, false>(l, a, st);
    if (!l.down && !a.gu.whole) {
      // only these have rows of so many scale bytes
      if constexpr (MODE == kPre && FMT != FQ_FMT_NVFP4)
        if (l.mt == 1) return launch_gate_up<FMT, MODE, F16, false, 1>(l, a, st);
      return launch_gate_up<FMT, MODE, F16, false, kMtTail>(l, a, st);
    }
  }
  if (l.down) launch_down<FMT, MODE, F16, true>(l, a, st);
  else if (l.mt == 4) launch_gate_up<FMT, MODE, F16, true, 4>(l, a, st);
  else if (l.mt == 2) launch_gate_up<FMT, MODE, F16, true, 2>(l, a, st);
  else launch_gate_up<FMT, MODE, F16, true, 1>(l, a, st);
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
  size_t a, act, nact, tok, pw, total;
};
TokWs tok_ws(int T, int topk, int E, int F) {
  const int arow = (F + 127) / 128 * 128;  // whole chunks in every format
  const size_t P = (size_t)T * topk, slots = P < (size_t)E ? P : (size_t)E;
  TokWs w;
  size_t o = 0;
  w.a = o;     o += up256(P * arow * 2 * 2);  // two parts to an element at most
  w.act = o;   o += up256(slots * 16);
  w.nact = o;  o += 256;
  w.tok = o;   o += up256(P * 4);
  w.pw = o;    o += up256(P * 4);
  w.total = o;
  return w;
}


// The gate_up launch: items, token rows staged at a time, LDS.
Launch gate_up_launch(TokArgs &a, const fq_stored_w &w_gu) {
  // A's zero tail up to whole chunks of the down projection counts as channels
  a.arow = a.d.nch * a.d.seg * 4;
  a.agroups = a.arow / kTile;
  // channel groups per item: the most that leave two items to a block (fewer
  // items spread the staging of the tokens over more weights, more of them keep
  // every CU busy: one token of the default layer takes 13 us with 1 group, the
  // 64-token batch 63 with 4)
  const int slots = a.P < a.E ? a.P : a.E;
  int mt = 4;
  while (mt > 1 && (long)slots * ((a.agroups + mt - 1) / mt) < 1024) mt /= 2;
  // bytes of a row's scales, fewer channels to an item where they are many
  const int f = w_gu.fmt, ng = a.gu.groups;
  const bool grouped = f != FQ_FMT_NONE && f != FQ_FMT_NVFP4 && ng > 1;
  a.rsc = row_bytes(f == FQ_FMT_NVFP4 ? a.gu.K / 16 : grouped ? 4 * ng : 0);
  a.rzp = row_bytes(f == FQ_FMT_INT4 ? ng : 0);
  const int per_row = (a.rsc.n ? a.rsc.stride : 0) + (a.rzp.n ? a.rzp.stride : 0);
  while (mt > 1 && 2 * mt * kTile * per_row > (20 << 10)) mt /= 2;
  const int chunk = a.gu.seg * 4, row = xrow_bytes(a.gu.K, chunk);
  a.idb = (a.P * 2 + 15) / 16 * 16;
  if (!a.gu.whole)
    mt = 2 * kMtTail * kTile * per_row + row + a.idb + kPlanBytes <= kLdsBytes ? kMtTail : 1;
  a.ny = (a.agroups + mt - 1) / mt;
  a.dny = FastDiv((uint32_t)a.ny);
  // token rows staged at a time: 16 columns of an MFMA, or what leaves two
  // blocks to a CU (80 KB, 11.6 of them the plan), at least one
  int sums = 2 * mt * kTile * per_row;
  if (sums < kRedBytes) sums = kRedBytes;
  int nc = (kLdsBytes / 2 - kPlanBytes - a.idb - sums) / row;
  nc = nc < 1 ? 1 : nc > 16 ? 16 : nc;
  a.ncol = nc < a.T ? nc : a.T;
  a.xb = a.ncol * row;
  a.dvpr = FastDiv((uint32_t)(a.gu.nch * (chunk / 8)));
  a.dncol = FastDiv((uint32_t)a.ncol);
  // blocks: two to a CU, at most one per item
  const long items = (long)slots * a.ny;
  const int blocks = (int)(items < 512 ? items : 512);
  a.dgrid = FastDiv((uint32_t)blocks);
  return {false, mt, dim3(blocks), a.idb + a.xb + sums};
}

void set_sizes(TokArgs &a, int T, int H, int F, int topk, int E, const fq_stored_w &w_gu,
               const fq_stored_w &w_d, int afmt1, int afmt2) {
  a.T = T;
  a.topk = topk;
  a.P = T * topk;
  a.E = E;
  a.H = H;
  a.F = F;
  a.gu = tok_stack(w_gu, 2 * F, H, afmt1);
  a.d = tok_stack(w_d, H, F, afmt2);
}

}  // namespace

size_t moe_tokens_ws_bytes(int T, int topk, int E, int F) {
  return tok_ws(T, topk, E, F).total;
}

size_t moe_tokens_lds_bytes(int T, int H, int F, int topk, int E, const fq_stored_w &w_gu,
                            const fq_stored_w &w_d) {
  TokArgs a{};
  set_sizes(a, T, H, F, topk, E, w_gu, w_d, FQ_FMT_NONE, FQ_FMT_NONE);
  return (size_t)gate_up_launch(a, w_gu).lds + kPlanBytes;
}

void launch_moe_tokens(const uint16_t *x, int T, int H, int F, const int32_t *ids,
                       const float *probs, int topk, int ebegin, int E, const fq_stored_w &w_gu,
                       const fq_stored_w &w_d, int afmt1, const float *as1, int afmt2,
                       const float *as2, uint16_t *out, void *ws, hipStream_t st) {
  const TokWs o = tok_ws(T, topk, E, F);
  char *b = static_cast<char *>(ws);
  TokArgs a{};
  set_sizes(a, T, H, F, topk, E, w_gu, w_d, afmt1, afmt2);
  a.x = x;
  a.ids = ids;
  a.probs = probs;
  a.ebegin = ebegin;
  a.dtopk = FastDiv((uint32_t)topk);
  a.afmt1 = afmt1;
  a.afmt2 = afmt2;
  a.as1 = as1;
  a.as2 = as2;
  a.a = reinterpret_cast<uint16_t *>(b + o.a);
  a.act = reinterpret_cast<int4 *>(b + o.act);
  a.nact = reinterpret_cast<int32_t *>(b + o.nact);
  a.tok = reinterpret_cast<int32_t *>(b + o.tok);
  a.pw = reinterpret_cast<float *>(b + o.pw);
  a.out = out;
  launch_fmt(w_gu, gate_up_launch(a, w_gu), a, st);
  launch_fmt(w_d, {true, 0, dim3(H / 8), kWavesD * T * 8 * 4}, a, st);
}

}  // namespace fq
