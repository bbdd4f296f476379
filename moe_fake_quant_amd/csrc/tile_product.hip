// The int8 and gated products of many routed rows on gfx950: the tiled form of
// product.hip's operators.
//
// A tile is 256 weight rows (i) x 256 routed rows (j), eight waves of 128 x 64 =
// 4 x 2 MFMA 32x32 tiles, operands streamed global -> LDS in stages of 128 bytes a
// row (64 bf16 or 128 int8 elements) through a ring of two, in the two-group
// schedule described at run_tile. A stage costs the same bytes, LDS reads and MFMA
// cycles for both types (32x32x16 bf16, 32x32x32 int8), so int8 does twice the work
// in it.
//
// Gated: the tile's weight rows are 128 gate rows f and the 128 up rows F + f, laid
// out in LDS so that a wave's accumulators s = 0, 1 and s + 2 hold g and u of the
// same (row, column): SwiGLU, its gradient and the activation fake-quant then need
// no exchange but the amax of an NVFP4 block between the lane halves, and h never
// leaves the registers.
//
// A stage takes about 1.8 us with every CU at work, twice what its MFMAs need (the matrix
// unit is busy 46 to 49 % of the time), for both types and also where all operands lie in
// L2; a tile has 5 to 7 us around its stages (28 % busy for int8 with a contraction of
// 768). What bounds a stage is not settled:
// - not the operands' bytes through L1 into LDS: 64 KB in 1.8 us are 9.3 TB/s over the
//   chip, and the 128 x 128 form of mid_product.hip moves 13.9 TB/s that way;
// - not the LDS reads or the barriers: four waves of 128 x 128, with two thirds of the
//   reads and half the barriers, took as long a stage (and 10 to 20 % more in all, for a
//   longer epilogue);
// - more likely the chain of waits: with 32 CUs at work a stage still takes up to 1.4 us
//   (512 rows of one int8 [4096 x 4096]: 44 us), and group A, which carries three quarters
//   of a stage's loads, waits for all of them before it issues the next ones.
// Without its stores the kernel takes 4 % (gated) to 20 % (int8, 768) less. Loads of a
// later stage issued ahead into L2 made it 30 % slower; eighths of the experts starting at
// different stages, 2 % slower at 512 and more rows an expert (at 128 rows of bf16 between
// 0 and 15 % faster, by the card); a higher wave priority for the multiplying group, flat.
// Measured with 128 experts, the kernel alone, fastest and average of 24 launches under the
// trace: gated forward over 65536 rows, H 2048, F 768, FP8 444 and 522 us (929 and 790
// TFLOP/s); its backward over 131072 rows 859 and 927 us (960, 890); int8 over 131072 rows
// of [2048 x 768] 332 and 360 us (1.24 and 1.15 POP/s).
//
// The backward's epilogue needs a few registers more than there are under an activation
// format: 2 go to scratch for INT8 and FP8, 28 for NVFP4, none inside the contraction loop.
//
// Rows and columns past the ends are clamped in the load addresses and not stored.
// A contraction that ends inside a stage: the loading wave overwrites the chunks
// past the end with zeros in LDS before it publishes the stage.
#include <type_traits>

#include "actq.hpp"
#include "internal.hpp"
#include "product.hpp"
#include "tile.hpp"

namespace fq {

namespace {

constexpr int BT = 256;                 // weight rows and routed rows of a tile
constexpr int kOperand = BT * 128;      // one operand, one stage: 32 KiB

__shared__ __attribute__((aligned(1024))) char g_ring[4 * kOperand];
template <int S>
__device__ __forceinline__ char *stage_p() {
  return g_ring + S * kOperand;
}
template <int S>
__device__ __forceinline__ char *stage_q() {
  return g_ring + (2 + S) * kOperand;
}

// int8: the scales of the tile's weight rows (in LDS row order) and routed rows
__shared__ __attribute__((aligned(16))) float g_scale[2 * BT];

struct PTile {
  int e, c0, j0, j_end;  // expert, first output column, routed rows [j0, j_end)
};

// columns of a tile
template <int KIND>
constexpr int kCols = KIND == PLAIN ? 256 : 128;

template <int KIND>
__device__ __forceinline__ PTile decode(const ProdArgs &a, const int *tile_start, int n_it, int gm,
                                        int w) {
  PTile t;
  int tile, it;
  tile_of(w, n_it, gm, __builtin_amdgcn_readfirstlane(tile_start[a.E]), tile, it);
  t.c0 = it * kCols<KIND>;
  // the same in every lane, which the LDS reads hide from the compiler: kept in scalar
  // registers, as the bases and bounds formed from them are
  t.e = __builtin_amdgcn_readfirstlane(expert_of_tile(tile_start, a.E, tile));
  t.j0 = a.seg[t.e] + (tile - __builtin_amdgcn_readfirstlane(tile_start[t.e])) * BT;
  t.j_end = a.seg[t.e + 1];
  return t;
}

// weight row (of the expert) behind row p of the tile's P operand
template <int KIND>
__device__ __forceinline__ int weight_row(const ProdArgs &a, const PTile &t, int p) {
  if constexpr (KIND == PLAIN) return min(t.c0 + p, a.N - 1);
  // rows 64 k .. 64 k + 63: gate (k even) or up of columns 64 (k / 2) ..
  const int up = (p >> 6) & 1, f = t.c0 + (p >> 7) * 64 + (p & 63);
  return up * a.C + min(f, a.C - 1);
}

// The operand streams of one tile. Shares (see run_tile): waves 0-3 load all of P
// (wave w its rows 64 w .. 64 w + 63) and the Q rows 128.. (slot w ^ 4), waves 4-7
// the Q rows 0..127. A slot is 32 rows, 4 DMA instructions of 8 rows.
template <int KIND>
struct Streams {
  const char *pbase, *qbase;  // of this wave's first P row; of x
  uint32_t poff[2];           // lane offset of instruction parity 0, 1 at row lane / 8
  int plast;                  // last valid row from pbase, clamped rows end there
  uint32_t qoff[4];
  int nk, tail;               // stages; bytes of the last one (128: whole)
  float scale;                // int8: this thread's entry of g_scale

  template <bool I8>
  __device__ __forceinline__ void init(const ProdArgs &a, const PTile &t, int wave, int lane) {
    nk = (int)((a.KB + 127u) >> 7);
    tail = (int)(a.KB - (uint32_t)(nk - 1) * 128u);
    const int p0 = 64 * (wave & 3);
    const int r0 = KIND == PLAIN ? t.c0 + p0
                                 : ((wave & 1) ? a.C : 0) + t.c0 + ((wave & 3) >> 1) * 64;
    const int last = KIND == PLAIN ? a.N - 1 : ((wave & 1) ? a.C : 0) + a.C - 1;
    const int rb = min(r0, last);
    plast = last - rb;
    if (r0 > last) plast = 0;
    pbase = a.w + ((size_t)t.e * a.N + rb) * a.KB;
    const int lr = lane >> 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) poff[k] = (uint32_t)lr * a.KB + lane_chunk(lane, k) * 16u;
    const int xs = wave ^ 4;
    // direct rows: offsets from the tile's first row, so that x may pass 4 GiB
    qbase = a.perm ? a.x : a.x + (size_t)t.j0 * a.KB;
#pragma unroll
    for (int ii = 0; ii < 4; ++ii) {
      const int r = min(t.j0 + 32 * xs + 8 * ii + lr, t.j_end - 1);
      const uint32_t row = a.perm ? a.topk.div((uint32_t)a.perm[r]) : (uint32_t)(r - t.j0);
      qoff[ii] = row * a.KB + lane_chunk(lane, ii) * 16u;
    }
    scale = 0.0f;
    if constexpr (I8) {
      const int i = (int)(threadIdx.x & 255);
      if (threadIdx.x < 256)
        scale = a.sw[a.sw_rows ? (size_t)t.e * a.N + weight_row<KIND>(a, t, i) : (size_t)t.e];
      else
        scale = a.sx[x_row(a, min(t.j0 + i, t.j_end - 1))];
      // completed here: a later wait for it would also wait for the DMAs in between
      asm volatile("" : "+v"(scale));
    }
  }

  // this wave's share of stage kt into ring buffer S
  template <int S>
  __device__ __forceinline__ void issue(const ProdArgs &a, int kt, int wave, int lane) const {
    const uint32_t c0 = (uint32_t)kt * 128u;
    // the rare cases form their addresses here: an empty asm keeps them from being
    // hoisted into the contraction loop's registers
    asm volatile("" : "+v"(lane));
    // lanes whose chunk lies past the contraction's end read the stage's first chunk
    // (valid memory); zero_tail clears them
    uint32_t back[2] = {0, 0};
    if (kt + 1 == nk && tail < 128) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t at = lane_chunk(lane, k) * 16u;
        back[k] = at >= (uint32_t)tail ? at : 0u;
      }
    }
    if (wave < 4) {
      char *dst = stage_p<S>() + wave * 8192;
      if (plast >= 63) {
        // (the step hidden from the compiler, which would keep its seven multiples)
        uint32_t step = 8u * a.KB;
        asm volatile("" : "+s"(step));
        const char *p = pbase + c0;
#pragma unroll
        for (int ii = 0; ii < 8; ++ii, p += step)
          dma16(p, poff[ii & 1] - back[ii & 1], dst + ii * 1024);
      } else {
#pragma unroll
        for (int ii = 0; ii < 8; ++ii) {
          const int r = min(8 * ii + (lane >> 3), plast);
          const uint32_t off = (uint32_t)r * a.KB + lane_chunk(lane, ii) * 16u;
          dma16(pbase + c0, off - back[ii & 1], dst + ii * 1024);
        }
      }
    }
    char *dst = stage_q<S>() + (wave ^ 4) * 4096;
#pragma unroll
    for (int ii = 0; ii < 4; ++ii) dma16(qbase + c0, qoff[ii] - back[ii & 1], dst + ii * 1024);
  }

  // the last stage, landed in buffer S: this wave's chunks past the end become zero
  template <int S>
  __device__ __forceinline__ void zero_tail(int wave, int lane) const {
    const i32x4 z = {0, 0, 0, 0};
    asm volatile("" : "+v"(lane));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (lane_chunk(lane, k) * 16u < (uint32_t)tail) continue;
      if (wave < 4) {
#pragma unroll
        for (int ii = k; ii < 8; ii += 2)
          *reinterpret_cast<i32x4 *>(stage_p<S>() + wave * 8192 + ii * 1024 + lane * 16) = z;
      }
#pragma unroll
      for (int ii = k; ii < 4; ii += 2)
        *reinterpret_cast<i32x4 *>(stage_q<S>() + (wave ^ 4) * 4096 + ii * 1024 + lane * 16) = z;
    }
    wait_lgkm0();
  }
};

constexpr int kDmaA = 12, kDmaB = 4;  // DMA instructions of a wave and stage, by group

// A wave's output: its 64 columns from column c (of C) for 32 of its rows, from j, out
// of the slab (rows of 128 bytes, chunk k of row r at k ^ (r & 7)), whole row segments
__device__ __forceinline__ void store_slab32(const char *slab, uint16_t *out, size_t ld, int c, int C,
                                             int j, int j_end, int lane) {
  const int ch = lane & 7;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = 8 * it + (lane >> 3);
    const uint4 v = *reinterpret_cast<const uint4 *>(slab + r * 128 + ((ch ^ (r & 7)) << 4));
    if (j + r < j_end && c + ch * 8 < C) {
      uint4 *dst = reinterpret_cast<uint4 *>(out + (size_t)(j + r) * ld + c + ch * 8);
      __builtin_nontemporal_store(v.x, &dst->x);
      __builtin_nontemporal_store(v.y, &dst->y);
      __builtin_nontemporal_store(v.z, &dst->z);
      __builtin_nontemporal_store(v.w, &dst->w);
    }
  }
}

// One tile: the contraction loop and the epilogue. The first `pre` stages (0 to 2)
// are already in flight; with next_w >= 0 the next tile's first two stages are
// issued as this tile's buffers free up, and the number issued is returned. `ld`
// holds this tile's streams and leaves with the next one's.
//
// Waves w and w + 4 share a SIMD, so the groups A = waves 0-3 and B = waves 4-7
// hold one wave of each. They run a quarter stage apart: between two block barriers
// one group multiplies half a stage from registers while the other reads its
// fragments of the next half from LDS and, twice a stage, issues its share of the
// loads two stages ahead. For the halves h = 0, 1 of stage t:
//   phase 4t     : A multiplies t.0  | B reads t.0
//   phase 4t + 1 : B multiplies t.0  | A reads t.1
//   phase 4t + 2 : A multiplies t.1  | B reads t.1,   loads its share of t+2
//   phase 4t + 3 : B multiplies t.1  | A reads t+1.0, loads its share of t+2
// A load may land as soon as it is issued, so it goes only where nobody reads from
// that phase on: B fills the Q rows that A multiplies (A has read them by phase
// 4t + 2), A the P rows and B's Q rows after the stage's last read.
template <int KIND, bool I8, int AFMT>
__device__ __forceinline__ int run_tile(const ProdArgs &a, const int *tile_start, int n_it, int gm,
                                        const PTile &tl, Streams<KIND> &ld, int pre, int next_w) {
  const int t = threadIdx.x;
  const int lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wi = wave & 1, wj = wave >> 1;
  const bool grp_b = wave >= 4;
  const int nk = ld.nk;
  const bool cut = ld.tail < 128;
  // a wave without rows or without columns skips its reads and MFMAs
  const int wcol = tl.c0 + wi * (kCols<KIND> / 2);
  const bool live = tl.j0 + wj * 64 < tl.j_end && wcol < a.C;

  typename Acc32<I8>::type acc[4][2];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[s][u][v] = 0;

  if constexpr (I8) {  // read in the epilogue, many barriers from here
    g_scale[t] = ld.scale;
    wait_lgkm0();
  }

  struct Frags {
    i32x4 p[4], q[2];
  };
  Frags f[2];
  // One lane address an operand: a step's chunk 2 ks + lane / 32 differs from step 0's in
  // bits 5 and 6 alone, so its address is an exclusive or away. Formed anew in each phase
  // (an empty asm keeps the eight of them out of the loop's registers).
  uint32_t pa = (uint32_t)(uintptr_t)(stage_p<0>() + nrm_off(wi * 128 + (lane & 31), lane >> 5));
  uint32_t qa = (uint32_t)(uintptr_t)(stage_q<0>() + nrm_off(wj * 64 + (lane & 31), lane >> 5));
  auto read_half = [&](auto stage_tag, int h) {
    constexpr int S = decltype(stage_tag)::value;
    typedef __attribute__((address_space(3))) const i32x4 lds_i32x4;
    asm volatile("" : "+v"(pa), "+v"(qa));
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      const uint32_t ks = 32u * (uint32_t)(2 * h + k2);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        f[k2].p[s] = *(lds_i32x4 *)(uintptr_t)((pa ^ ks) + S * kOperand + s * 4096);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        f[k2].q[u] = *(lds_i32x4 *)(uintptr_t)((qa ^ ks) + S * kOperand + u * 4096);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2)
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) mfma32<I8>(f[k2].p[s], f[k2].q[u], acc[s][u]);
  };
  // a block barrier that the scheduler moves nothing across
  auto phase_barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto a_step = [&](auto stage_tag, int kt) {
    constexpr int S = decltype(stage_tag)::value;
    phase_barrier();  // 4kt
    if (live) multiply();
    phase_barrier();  // 4kt+1
    if (live) read_half(stage_tag, 1);
    wait_lgkm0();
    phase_barrier();  // 4kt+2
    if (live) multiply();
    if (kt + 1 < nk) {
      wait_vm<0>();  // this wave's share of stage kt+1
      if (cut && kt + 2 == nk) ld.template zero_tail<S ^ 1>(wave, lane);
      phase_barrier();  // 4kt+3
      if (live) read_half(std::integral_constant<int, S ^ 1>{}, 0);
      wait_lgkm0();
      if (kt + 2 < nk) ld.template issue<S>(a, kt + 2, wave, lane);
    }
  };
  auto b_step = [&](auto stage_tag, int kt) {
    constexpr int S = decltype(stage_tag)::value;
    phase_barrier();  // 4kt
    if (live) read_half(stage_tag, 0);
    wait_lgkm0();
    phase_barrier();  // 4kt+1
    if (live) multiply();
    phase_barrier();  // 4kt+2
    if (live) read_half(stage_tag, 1);
    wait_lgkm0();
    if (kt + 2 < nk) {
      ld.template issue<S>(a, kt + 2, wave, lane);
      wait_vm<kDmaB>();  // this wave's share of stage kt+1 (read by A next phase)
    } else {
      wait_vm<0>();
      if (cut && kt + 2 == nk) ld.template zero_tail<S ^ 1>(wave, lane);
    }
    phase_barrier();  // 4kt+3
    if (live) multiply();
  };

  if (pre < 1) ld.template issue<0>(a, 0, wave, lane);
  if (pre < 2 && nk > 1) ld.template issue<1>(a, 1, wave, lane);
  if (nk <= 1) wait_vm<0>();  // this wave's share of stage 0
  else if (grp_b) wait_vm<kDmaB>();
  else wait_vm<kDmaA>();
  if (cut && nk == 1) ld.template zero_tail<0>(wave, lane);
  phase_barrier();
  if (!grp_b) {
    if (live) read_half(std::integral_constant<int, 0>{}, 0);
    wait_lgkm0();
    for (int kt = 0; kt < nk; kt += 2) {
      a_step(std::integral_constant<int, 0>{}, kt);
      if (kt + 1 < nk) a_step(std::integral_constant<int, 1>{}, kt + 1);
    }
    phase_barrier();  // opens phase 4nk-1, B's last multiply
  } else {
    for (int kt = 0; kt < nk; kt += 2) {
      b_step(std::integral_constant<int, 0>{}, kt);
      if (kt + 1 < nk) b_step(std::integral_constant<int, 1>{}, kt + 1);
    }
  }

  // Nobody reads the ring any more. Stage 0 of the next tile goes to buffer 0 now;
  // buffer 1 serves as staging (A the P half, B the Q half, 8 KiB a wave) and takes
  // stage 1 after the closing barrier.
  char *slab = (wave < 4 ? stage_p<1>() : stage_q<1>()) + (wave & 3) * 8192;
  const int jw = tl.j0 + wj * 64;
  int ln = lane;
  // an empty asm keeps the addresses formed from it out of the loop's registers
  asm volatile("" : "+v"(ln));
  const int h = ln >> 5, jr = ln & 31;
  // the accumulator (s, u, v) of this lane: weight row wi*128 + s*32 + 8*(v/4) + 4*h + v%4
  // of the tile, routed row jw + u*32 + jr
  if constexpr (KIND == GATED_BWD) {
    if (live) {
      // dA's 64 x 64 piece into the slab, laid out as store_slab32 reads it
      const uint32_t ch = (uint32_t)(ln & 7), rr = (uint32_t)(ln >> 3);
      const int col = wcol + (int)((ch ^ (rr & 7u)) * 8u);
      const char *base = reinterpret_cast<const char *>(a.daq + (size_t)jw * a.C);
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int r = min(8 * it + (int)rr, tl.j_end - 1 - jw);
        const uint32_t off = ((uint32_t)r * (uint32_t)a.C + (uint32_t)(col < a.C ? col : wcol)) * 2u;
        dma16(base, off, slab + it * 1024);
      }
    }
  }
  if (next_w >= 0) {
    const PTile nt = decode<KIND>(a, tile_start, n_it, gm, next_w);
    ld.template init<I8>(a, nt, wave, lane);
    ld.template issue<0>(a, 0, wave, lane);
  }
  if constexpr (KIND == PLAIN) {
    if (live) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float sx = I8 ? g_scale[BT + wj * 64 + u * 32 + jr] : 1.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
            const float4 sw = *reinterpret_cast<const float4 *>(g_scale + wi * 128 + s * 32 + 8 * q + 4 * h);
            v[0] = ((float)acc[s][u][4 * q] * sx) * sw.x;
            v[1] = ((float)acc[s][u][4 * q + 1] * sx) * sw.y;
            v[2] = ((float)acc[s][u][4 * q + 2] * sx) * sw.z;
            v[3] = ((float)acc[s][u][4 * q + 3] * sx) * sw.w;
            const uint2 pk = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            const uint32_t c = (uint32_t)(4 * s + q) ^ (uint32_t)(jr & 15);
            *reinterpret_cast<uint2 *>(slab + jr * 256 + c * 16 + h * 8) = pk;
          }
        const int ch = ln & 15;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int r = 4 * it + (ln >> 4), j = jw + u * 32 + r;
          const uint4 v = *reinterpret_cast<const uint4 *>(slab + r * 256 + ((ch ^ (r & 15)) << 4));
          // whole row segments past the L2, which keeps its lines for the operands (int8,
          // 131072 rows of [2048 x 768]: 289 us, with ordinary stores 303)
          if (j < tl.j_end && wcol + ch * 8 < a.C) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (size_t)j * a.C + wcol + ch * 8);
            __builtin_nontemporal_store(v.x, &dst->x);
            __builtin_nontemporal_store(v.y, &dst->y);
            __builtin_nontemporal_store(v.z, &dst->z);
            __builtin_nontemporal_store(v.w, &dst->w);
          }
        }
      }
    }
  } else {
    // 4 (columns) x 32 (rows) pieces (s, q) of the wave's 64 columns at f = 32 s + 8 q + 4 h
    // one instantiation a format, so that the blocks below hold no branch; the scale is
    // read here, where registers are free again
    const ActQ aq = load_actq(AFMT, a.ascale);
    auto piece = [&](int u, int s, int q) -> uint2 & {
      const uint32_t row = (uint32_t)(u * 32 + jr), c = (uint32_t)(4 * s + q) ^ (row & 7u);
      return *reinterpret_cast<uint2 *>(slab + row * 128 + c * 16 + h * 8);
    };
    if constexpr (KIND == GATED_BWD) {  // dA has landed
      if (next_w < 0) wait_vm<0>();
      else if (grp_b) wait_vm<kDmaB>();
      else wait_vm<kDmaA>();
    }
    if (live) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float sx = I8 ? g_scale[BT + wj * 64 + u * 32 + jr] : 1.0f;
        uint2 ku[KIND == GATED_BWD ? 8 : 1], ka[KIND == GATED_BWD ? 8 : 1];  // dU, FQ_a(a)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // a 16-block of columns: 8 here, 8 in lane ^ 32
            // (the backward works in small steps: side by side they would spill, and a
            // reload behind the output stores waits for them)
            constexpr bool BWD = KIND == GATED_BWD;
            auto sum = [&](int half, int k) {  // g (0) or u (1) of element k
              const int at = 8 * b + k;
              if constexpr (I8) {
                const int p = wi * 128 + s * 32 + 16 * b + 8 * (k >> 2) + 4 * h + (k & 3);
                return ((float)acc[s + 2 * half][u][at] * sx) * g_scale[p + 64 * half];
              } else {
                return acc[s + 2 * half][u][at];
              }
            };
            auto grads = [&](int q, uint32_t m, const float *sig) {
              // dA's pieces lie where dG's go, lane by lane
              uint2 &pc = piece(u, s, 2 * b + q);
              const uint2 dp = pc;
              const float d[4] = {lo_bf16(dp.x), hi_bf16(dp.x), lo_bf16(dp.y), hi_bf16(dp.y)};
              float dg[4], du[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                swiglu_grad((m >> k) & 1u ? d[k] : 0.0f, sum(0, 4 * q + k), sum(1, 4 * q + k), sig[k], dg[k],
                            du[k]);
              pc = make_uint2(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]));
              ku[4 * s + 2 * b + q] = make_uint2(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]));
              __builtin_amdgcn_sched_barrier(0);
            };
            if constexpr (!BWD || AFMT == FQ_FMT_NVFP4) {
              float sig[8], v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float g = sum(0, k);
                sig[k] = sigmoid_hw(g);
                v[k] = bf16_to_f32(f32_to_bf16((g * sig[k]) * sum(1, k)));
              }
              if constexpr (BWD) __builtin_amdgcn_sched_barrier(0);
              const uint32_t m = act_fq8_pair<32>(aq, v);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint2 pk = make_uint2(pack_bf16(v[4 * q], v[4 * q + 1]),
                                            pack_bf16(v[4 * q + 2], v[4 * q + 3]));
                if constexpr (BWD) {
                  ka[4 * s + 2 * b + q] = pk;
                  __builtin_amdgcn_sched_barrier(0);
                  grads(q, m >> (4 * q), sig + 4 * q);
                } else {
                  piece(u, s, 2 * b + q) = pk;
                }
              }
            } else {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                float sig[4], v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float g = sum(0, 4 * q + k);
                  sig[k] = sigmoid_hw(g);
                  v[k] = bf16_to_f32(f32_to_bf16((g * sig[k]) * sum(1, 4 * q + k)));
                }
                __builtin_amdgcn_sched_barrier(0);
                const uint32_t m = act_fq4(aq, v);
                ka[4 * s + 2 * b + q] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
                __builtin_amdgcn_sched_barrier(0);
                grads(q, m, sig);
              }
            }
          }
        const char *half = slab + u * 4096;
        const int ju = jw + u * 32;
        if constexpr (KIND == GATED) {
          store_slab32(half, a.out, a.C, wcol, a.C, ju, tl.j_end, ln);
        } else {
          auto put_kept = [&](const uint2 (&k)[8]) {
            wait_lgkm0();  // the half slab has been read back
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
              for (int q = 0; q < 4; ++q) piece(u, s, q) = k[4 * s + q];
          };
          store_slab32(half, a.out, 2 * (size_t)a.C, wcol, a.C, ju, tl.j_end, ln);
          put_kept(ku);
          store_slab32(half, a.out + a.C, 2 * (size_t)a.C, wcol, a.C, ju, tl.j_end, ln);
          if (a.aq) {
            put_kept(ka);
            store_slab32(half, a.aq, a.C, wcol, a.C, ju, tl.j_end, ln);
          }
        }
      }
    }
  }
  wait_lgkm0();  // the slab and the scales are read back before they are written again
  block_barrier();
  if (next_w < 0) return 0;
  if (ld.nk < 2) return 1;
  ld.template issue<1>(a, 1, wave, lane);
  return 2;
}

// Persistent grid, one block a CU: each XCD (block b runs on XCD b % 8) owns a
// contiguous eighth of the tiles, dealt round-robin to its blocks, so that the tiles
// in flight there share operand panels in its L2.
template <int KIND, bool I8, int AFMT>
__global__ __launch_bounds__(NT) void k_tile_product(ProdArgs a, int n_it, int gm) {
  __shared__ int tile_start[kMaxExperts + 1];
  build_tile_prefix(a.seg, a.E, BT, 0, tile_start);
  const int total = __builtin_amdgcn_readfirstlane(tile_start[a.E]) * n_it;
  const int nslot = gridDim.x >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int chunk = (total + 7) >> 3;
  const int w_end = min((xcd + 1) * chunk, total);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int w = xcd * chunk + slot;
  if (w >= w_end) return;  // the whole block
  Streams<KIND> ld;
  ld.template init<I8>(a, decode<KIND>(a, tile_start, n_it, gm, w), wave, lane);
  int pre = 0;
  for (; w < w_end; w += nslot) {
    const PTile tl = decode<KIND>(a, tile_start, n_it, gm, w);
    pre = run_tile<KIND, I8, AFMT>(a, tile_start, n_it, gm, tl, ld, pre, w + nslot < w_end ? w + nslot : -1);
  }
}

template <int KIND, bool I8, int AFMT = FQ_FMT_NONE>
void launch(const ProdArgs &a, int R_max, hipStream_t st) {
  const int n_it = ceil_div(a.C, kCols<KIND>);
  // row tiles, at most: m non-empty experts hold 256 (q - 1) + 1 rows or more for q tiles
  const int m = a.E < R_max ? a.E : R_max;
  const size_t units = ((size_t)((R_max - m) / BT) + (size_t)m) * (size_t)n_it;
  const int cus = device_cus();
  const size_t up8 = (units + 7) / 8 * 8;
  const int grid = (int)(up8 < (size_t)cus ? up8 : (size_t)cus);
  hipLaunchKernelGGL((k_tile_product<KIND, I8, AFMT>), dim3(grid), dim3(NT), 0, st, a, n_it,
                     tile_group(cus / 8, n_it, ceil_div(R_max, (long)BT * a.E)));
}

template <int KIND>
void launch_bf16(const ProdArgs &a, int R_max, hipStream_t st) {
  switch (a.afmt) {
    case FQ_FMT_NONE: launch<KIND, false, FQ_FMT_NONE>(a, R_max, st); break;
    case FQ_FMT_INT8: launch<KIND, false, FQ_FMT_INT8>(a, R_max, st); break;
    case FQ_FMT_FP8_E4M3: launch<KIND, false, FQ_FMT_FP8_E4M3>(a, R_max, st); break;
    default: launch<KIND, false, FQ_FMT_NVFP4>(a, R_max, st); break;
  }
}

}  // namespace

void launch_tile_product(const ProdArgs &a, int kind, bool i8, int R_max, hipStream_t st) {
  if (kind == PLAIN) launch<PLAIN, true>(a, R_max, st);
  else if (kind == GATED && i8) launch<GATED, true>(a, R_max, st);
  else if (kind == GATED) launch_bf16<GATED>(a, R_max, st);
  else launch_bf16<GATED_BWD>(a, R_max, st);
}

}  // namespace fq
