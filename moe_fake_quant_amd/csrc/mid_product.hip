// The int8 and gated products of a middling number of rows on gfx950: tiles of 64 x
// 64 or 128 x 128, several to a CU.
//
// The 256 x 256 tiles of tile_product.hip move the fewest bytes, but a call with
// fewer of them than CUs leaves CUs idle, and one block a CU shows its epilogue. Here
// four waves (2 x 2) stream both operands global -> LDS in stages of 128 bytes a row
// through a ring, one barrier a stage, and two blocks of a CU cover each other's
// waits and epilogues. The sums then go through the ring's memory, from where the
// last step (scales, SwiGLU, its gradient, fake-quant, stores) works on 8 columns of
// a row a thread, as in product.hip.
//
// Measured, the kernel alone: int8 over 2048 rows of [4096 x 4096] 38.7 us (1.77 POP/s,
// the matrix unit busy 38 % of the time; a large plain int8 product reaches 2.05); 333
// rows on five experts of [1040 x 368] 6.3 us, where the first stage's wait, the other
// two stages and the epilogue stand one after the other.
//
// Gated: of the weight rows of each wave the first half are gate rows f, the second
// half the up rows F + f.
#include <type_traits>

#include "product.hpp"

namespace fq {

namespace {

constexpr int kThreads = 256;

// weight row (of the expert) behind row p of a tile's P operand, columns from c0
template <int KIND, int T>
__device__ __forceinline__ int weight_row(const ProdArgs &a, int c0, int p) {
  if constexpr (KIND == PLAIN) return min(c0 + p, a.N - 1);
  const int r = p % (T / 2), col = c0 + (p / (T / 2)) * (T / 4) + r % (T / 4);
  return (r >= T / 4 ? a.C : 0) + min(col, a.C - 1);
}

template <int KIND, bool I8, int T, int NSTAGE>
__global__ __launch_bounds__(kThreads, NSTAGE * T > 256 ? 1 : 2) void k_mid_product(ProdArgs a, int n_it, int gm) {
  constexpr int kOp = T * 128;                 // one operand, one stage
  constexpr int NM = T / 64;                   // 32 x 32 MFMA tiles of a wave along i and j
  constexpr int PER = T / 32;                  // DMA instructions of a wave, operand and stage
  constexpr int COLS = KIND == PLAIN ? T : T / 2;
  static_assert(NSTAGE * 2 * kOp >= T * T * 4, "the sums go through the ring");
  __shared__ __attribute__((aligned(1024))) char ring[NSTAGE * 2 * kOp];
  __shared__ int tile_start[kMaxExperts + 1];
  // int8: the scales of the tile's weight rows and routed rows
  __shared__ __attribute__((aligned(16))) float scales[I8 ? 2 * T : 4];
  if (a.E == 1) {
    if (threadIdx.x == 0) {
      tile_start[0] = 0;
      tile_start[1] = (a.seg[1] - a.seg[0] + T - 1) / T;
    }
    __syncthreads();
  } else {
    build_tile_prefix<kThreads>(a.seg, a.E, T, 0, tile_start);
  }
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wi = wave & 1, wj = wave >> 1;
  const int nk = (int)((a.KB + 127u) >> 7), tail = (int)(a.KB - (uint32_t)(nk - 1) * 128u);
  const ActQ q = load_actq(KIND == PLAIN || I8 ? FQ_FMT_NONE : a.afmt, a.ascale);

  // each XCD (block b runs on XCD b % 8) takes a contiguous eighth of the tiles
  // the same in every lane, which the LDS reads hide from the compiler
  const int n_rows = __builtin_amdgcn_readfirstlane(tile_start[a.E]), total = n_rows * n_it;
  const int nslot = gridDim.x >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int chunk = (total + 7) >> 3, w_end = min((xcd + 1) * chunk, total);
  for (int w = xcd * chunk + slot; w < w_end; w += nslot) {
    int tile, it;
    tile_of(w, n_it, gm, n_rows, tile, it);
    const int c0 = it * COLS;
    const int e =
        a.E == 1 ? 0 : __builtin_amdgcn_readfirstlane(expert_of_tile(tile_start, a.E, tile));
    const int j0 = a.seg[e] + (tile - __builtin_amdgcn_readfirstlane(tile_start[e])) * T;
    const int j_end = a.seg[e + 1];

    // this lane's rows of both operands: wave w loads the rows w * T/4 .. of each
    const char *pbase = a.w + (size_t)e * a.N * a.KB;
    const char *qbase = a.perm ? a.x : a.x + (size_t)j0 * a.KB;
    uint32_t poff[PER], qoff[PER];
#pragma unroll
    for (int ii = 0; ii < PER; ++ii) {
      const int r = wave * (T / 4) + 8 * ii + (lane >> 3);
      const uint32_t ch = lane_chunk(lane, ii) * 16u;
      poff[ii] = (uint32_t)weight_row<KIND, T>(a, c0, r) * a.KB + ch;
      const int j = min(j0 + r, j_end - 1);
      const uint32_t row = a.perm ? a.topk.div((uint32_t)a.perm[j]) : (uint32_t)(j - j0);
      qoff[ii] = row * a.KB + ch;
    }
    // on its way during the contraction, put into `scales` behind it
    float scale = 0.0f;
    if constexpr (I8) {
      if (t < T) scale = a.sw[a.sw_rows ? (size_t)e * a.N + weight_row<KIND, T>(a, c0, t) : (size_t)e];
      else if (t < 2 * T) scale = a.sx[x_row(a, min(j0 + t - T, j_end - 1))];
    }
    // lanes past the contraction's end read their stage's first chunk, cleared below
    uint32_t back[2];
    auto look_back = [&](int kt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t at = lane_chunk(lane, k) * 16u;
        back[k] = kt + 1 == nk && at >= (uint32_t)tail ? at : 0u;
      }
    };
    // DMA instruction i of this wave's share of a stage (P first), after look_back
    auto issue1 = [&](int kt, int buf, int i) {
      const uint32_t k0 = (uint32_t)kt * 128u;
      char *dp = ring + buf * 2 * kOp + wave * (T / 4) * 128;
      if (i < PER) dma16(pbase + k0, poff[i % PER] - back[i & 1], dp + i * 1024);
      else dma16(qbase + k0, qoff[i % PER] - back[i & 1], dp + kOp + (i - PER) * 1024);
    };
    auto issue = [&](int kt, int buf) {
      look_back(kt);
#pragma unroll
      for (int i = 0; i < 2 * PER; ++i) issue1(kt, buf, i);
    };

    typename Acc32<I8>::type acc[NM][NM];
#pragma unroll
    for (int s = 0; s < NM; ++s)
#pragma unroll
      for (int u = 0; u < NM; ++u)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[s][u][v] = 0;

    // this wave's chunks of the last stage, landed in `buf`, past the end become zero
    auto zero_tail = [&](int buf) {
      char *dp = ring + buf * 2 * kOp + wave * (T / 4) * 128 + lane * 16;
#pragma unroll
      for (int ii = 0; ii < PER; ++ii)
        if (lane_chunk(lane, ii) * 16u >= (uint32_t)tail) {
          *reinterpret_cast<i32x4 *>(dp + ii * 1024) = i32x4{0, 0, 0, 0};
          *reinterpret_cast<i32x4 *>(dp + kOp + ii * 1024) = i32x4{0, 0, 0, 0};
        }
      wait_lgkm0();
    };
    struct Frags {  // half a stage: two MFMA steps
      i32x4 p[2][NM], q[2][NM];
    };
    // LDS read i of a half's fragments, in the order in which they are multiplied
    auto read1 = [&](Frags &f, int buf, int h, int i) {
      const char *sp = ring + buf * 2 * kOp;
      const int k2 = i / (2 * NM), k = i % (2 * NM), lo = lane & 31;
      const int ch = 2 * (2 * h + k2) + (lane >> 5);
      if (k < NM)
        f.p[k2][k] = *reinterpret_cast<const i32x4 *>(sp + nrm_off(wi * (T / 2) + k * 32 + lo, ch));
      else
        f.q[k2][k - NM] = *reinterpret_cast<const i32x4 *>(
            sp + kOp + nrm_off(wj * (T / 2) + (k - NM) * 32 + lo, ch));
    };
    // Half a stage is multiplied from registers while the next half's fragments come
    // out of LDS and a later stage's loads go out: a wave issues them between its MFMAs,
    // each of which keeps the matrix core busy for 32 cycles. One barrier a stage, in its
    // middle: it publishes stage kt + 1 (every wave has waited for its own loads) and
    // retires the reads of stage kt, whose buffer takes stage kt + NSTAGE.
    constexpr int NMF = 2 * NM * NM, NRD = 4 * NM, NDM = 2 * PER;
    Frags f0, f1;
    int buf = 0;
    auto multiply = [&](const Frags &f, int g) {
      const int k2 = g / (NM * NM), s = (g / NM) % NM, u = g % NM;
      mfma32<I8>(f.p[k2][s], f.q[k2][u], acc[s][u]);
    };
    auto step = [&](int kt, auto load_tag) {
      constexpr bool LOAD = decltype(load_tag)::value;
      wait_lgkm0();  // f0 has arrived
#pragma unroll
      for (int g = 0; g < NMF; ++g) {
        multiply(f0, g);
#pragma unroll
        for (int i = g * NRD / NMF; i < (g + 1) * NRD / NMF; ++i) read1(f1, buf, 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      wait_lgkm0();
      const bool more = LOAD || kt + 1 < nk;
      const int nb = buf + 1 == NSTAGE ? 0 : buf + 1;
      if (more) {
        if (LOAD || kt + NSTAGE - 1 < nk) wait_vm<(NSTAGE - 2) * 2 * PER>();
        else wait_vm<0>();
        if (kt + 2 == nk && tail < 128) zero_tail(nb);
        if (LOAD) look_back(kt + NSTAGE);
        __builtin_amdgcn_sched_barrier(0);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int g = 0; g < NMF; ++g) {
        multiply(f1, g);
        if (more) {
#pragma unroll
          for (int i = g * NRD / NMF; i < (g + 1) * NRD / NMF; ++i) read1(f0, nb, 0, i);
          if (LOAD) {
#pragma unroll
            for (int i = g * NDM / NMF; i < (g + 1) * NDM / NMF; ++i) issue1(kt + NSTAGE, buf, i);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      buf = nb;
    };
#pragma unroll
    for (int k = 0; k < NSTAGE; ++k)
      if (k < nk) issue(k, k);
    if (nk >= NSTAGE) wait_vm<(NSTAGE - 1) * 2 * PER>();
    else wait_vm<0>();
    if (nk == 1 && tail < 128) zero_tail(0);
    block_barrier();
#pragma unroll
    for (int i = 0; i < NRD; ++i) read1(f0, 0, 0, i);
    int kt = 0;
    for (; kt + NSTAGE < nk; ++kt) step(kt, std::true_type{});
    for (; kt < nk; ++kt) step(kt, std::false_type{});

    // sums [routed row j][weight row p], 4 of them a chunk, chunk c of row j at
    // c ^ (j % (T / 4)): a wave's writes (32 rows, one chunk) spread over the banks
    __syncthreads();
    int *sum = reinterpret_cast<int *>(ring);
    if (I8 && t < 2 * T) scales[t] = scale;
    auto at = [&](int j, int p) { return sum + j * T + (((p >> 2) ^ (j & (T / 4 - 1))) << 2); };
#pragma unroll
    for (int s = 0; s < NM; ++s)
#pragma unroll
      for (int u = 0; u < NM; ++u)
#pragma unroll
        for (int qq = 0; qq < 4; ++qq) {
          const int j = wj * (T / 2) + u * 32 + (lane & 31);
          const int p = wi * (T / 2) + s * 32 + 8 * qq + 4 * (lane >> 5);
          i32x4 v;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (I8) v[k] = acc[s][u][4 * qq + k];
            else v[k] = __float_as_int(acc[s][u][4 * qq + k]);
          }
          *reinterpret_cast<i32x4 *>(at(j, p)) = v;
        }
    __syncthreads();
    constexpr int CH = COLS / 8;                 // 8-column pieces of a row
    for (int i = t; i < T * CH; i += kThreads) {
      const int j = i / CH, cc = (i % CH) * 8, r = j0 + j;
      const bool live = r < j_end && c0 + cc < a.C;
      // the piece's place among the tile's weight rows
      const int p = KIND == PLAIN ? cc : (cc / (T / 4)) * (T / 2) + cc % (T / 4);
      auto sums = [&](int p, float *v) {
        int w[8];
        *reinterpret_cast<i32x4 *>(w) = *reinterpret_cast<const i32x4 *>(at(j, p));
        *reinterpret_cast<i32x4 *>(w + 4) = *reinterpret_cast<const i32x4 *>(at(j, p + 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = I8 ? ((float)w[k] * scales[T + j]) * scales[p + k] : __int_as_float(w[k]);
      };
      float g[8], u[8];
      sums(p, g);
      if constexpr (KIND != PLAIN) sums(p + T / 4, u);
      finish8<KIND>(a, q, r, c0 + cc, g, u, live);
    }
    __syncthreads();  // the sums are read before the next tile's stages land
  }
}

// NSTAGE 3 with tiles of 128 leaves room for one block a CU
template <int KIND, bool I8, int T, int NSTAGE>
void launch_ring(const ProdArgs &a, size_t units, int R_max, hipStream_t st) {
  constexpr int kBlocks = NSTAGE * T > 256 ? 1 : 2;
  const int n_it = ceil_div(a.C, KIND == PLAIN ? T : T / 2);
  const size_t most = (size_t)device_cus() * kBlocks, up8 = (units + 7) / 8 * 8;
  hipLaunchKernelGGL((k_mid_product<KIND, I8, T, NSTAGE>), dim3((unsigned)(up8 < most ? up8 : most)),
                     dim3(kThreads), 0, st, a, n_it,
                     tile_group(device_cus() / 8 * kBlocks, n_it, ceil_div(R_max, (long)T * a.E)));
}

template <int KIND, bool I8>
void launch(const ProdArgs &a, int tile, int R_max, hipStream_t st) {
  // row tiles, at most: m non-empty experts hold T (q - 1) + 1 rows or more for q tiles
  const int m = a.E < R_max ? a.E : R_max;
  const size_t units = (size_t)((R_max - m) / tile + m) *
                       (size_t)ceil_div(a.C, KIND == PLAIN ? tile : tile / 2);
  if (tile == 64) launch_ring<KIND, I8, 64, 4>(a, units, R_max, st);
  // no more tiles than CUs: a deeper ring instead of a second block a CU (29 against 34
  // us for int8, 40 against 48 for gated bf16 at 1024 rows of [4096 x 4096]; with two
  // rounds of tiles 57 against 51, 77 against 69)
  else if (units <= (size_t)device_cus()) launch_ring<KIND, I8, 128, 3>(a, units, R_max, st);
  else launch_ring<KIND, I8, 128, 2>(a, units, R_max, st);
}

}  // namespace

void launch_mid_product(const ProdArgs &a, int kind, bool i8, int tile, int R_max, hipStream_t st) {
  if (kind == PLAIN) launch<PLAIN, true>(a, tile, R_max, st);
  else if (kind == GATED && i8) launch<GATED, true>(a, tile, R_max, st);
  else if (kind == GATED) launch<GATED, false>(a, tile, R_max, st);
  else launch<GATED_BWD, false>(a, tile, R_max, st);
}

}  // namespace fq
