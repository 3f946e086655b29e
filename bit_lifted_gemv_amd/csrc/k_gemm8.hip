// Product of 8-bit weights (e4m3, a scale per 128 x 128 block) with many rows of
// 8-bit activations (a power of two per 128 positions), on the matrix cores, with
// the epilogue of lq_gemm8 and the ragged expert runs of lq_gemm8_grouped.
//
// Tile.  WT x WW waves, each 16 FT tokens x 16 FW rows of weights in tiles of 16 x 16:
// v_mfma_scale_f32_16x16x128_f8f6f4 takes a whole block of 128 positions, rows of weights
// as operand A, so that a lane's four sums are four rows of one token: one 8- or
// 16-byte piece of the output.  The exponents of both sides are the instruction's
// scales; a float32 scale costs four multiply-adds per product.  The instruction adds
// eight products at a time and cuts them off 13 places below the largest sum of two
// factors' exponents: 2^-16 of a typical result, 2^-14.5 with outlying positions, where the
// 16-bit results round by up to 2^-11 or 2^-8.  For float32 results (PREC) the operands become
// bfloat16 (exact) and v_mfma_f32_16x16x32_bf16 keeps 24 bits, at half the rate or less.
//
// Operands come to LDS by loads that write it directly, in stages of 128 positions (a
// ring of S); 16-byte piece c of row r lies at piece c ^ (r / 2 % 8), so that 16 lanes
// reading one piece of 16 rows touch every bank once.  Rows of 128 bytes are what such
// loads move best: rows of 64 bytes took twice as long per byte.
//
// A wave holds a stage's rows and a ring of four token tiles; each is refilled from
// LDS as soon as its last product has been issued.  Where the refills pass to the
// next stage, one barrier says both that it has landed and that this one's place
// in the ring may be loaded again.
//
// The waits are counted by hand (the compiler would drain the loads before every
// read of LDS): every wave issues the same number of loads per stage.
//
// Bound by the matrix instructions: 256 x 256 tiles of 4096 x 4096 -> 2 x 14336 take
// 397 us (2.4 PF); per 1024 positions 85 us (2.8 PF, what a large library product of
// the same types reaches on the same card), the rest is the tiles' beginnings (25 us, the
// first loads) and ends (some 50 us, half of them the output's 117 MB).
#include "f6_epilogue.h"
#include "f6_product.h"
#include "f8.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;
using namespace f8;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 64 lanes x 16 (or 4) bytes from resource r at voff + soff to LDS at `lds` (bytes).
// m0 is the compiler's own and never allocated (it warns of it among the clobbers): each load sets it,
// and no other instruction of the kernel reads it.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voff, const i32x4& r, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}
__device__ __forceinline__ void load_word_to_lds(uint32_t lds, uint32_t voff, const i32x4& r, uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t at, int offset) {
  const auto* base = reinterpret_cast<const __attribute__((address_space(3))) char*>(at);
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(base + offset);
}

template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ i32x4 resource(const void* p, int64_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = uniform(static_cast<int>(u));
  r[1] = uniform(static_cast<int>(u >> 32) & 0xFFFF);
  r[2] = uniform(static_cast<int>(bytes > 0xFFFFFFFF ? 0xFFFFFFFF : bytes));
  r[3] = 0x00020000;
  return r;
}

template <int WT, int WW, int WK, int FT, int FW>
struct Tile {
  static constexpr int GROUP = WT * WW, NW = GROUP * WK;        // waves
  static constexpr int TOK = 16 * FT * WT, ROWS = 16 * FW * WW;
  static constexpr int IL = TOK / 8 / GROUP, WL = ROWS / 8 / GROUP;   // 1 KB loads per wave and stage
  static constexpr int LOADS = IL + WL + 1;
  // a stage: tokens, rows and the rows' scales; behind the ring the tokens' exponents, whose words
  // hold four blocks (two of them, in turn), and a place that nobody reads
  static constexpr int ROWS_AT = TOK * 128, SCALES_AT = ROWS_AT + ROWS * 128, STAGE = SCALES_AT + ROWS * 4;
  static constexpr int BEHIND = 2 * TOK * 4 + 256;
  static constexpr int PER_SIMD = 2;                            // waves, of up to 256 registers
  static constexpr int MAX_LDS = 163840 / (PER_SIMD * 4 / NW);  // workgroups of a compute unit
  static constexpr int RING = (MAX_LDS / WK - BEHIND) / STAGE, S = RING > 4 ? 4 : RING;
  static constexpr int PART = S * STAGE + BEHIND, LDS = WK * PART;   // of a group, of all
  static constexpr int PITCH = 16 * FW + 4, AT_ONCE = 8 / FW;   // of the sums on their way out
  static_assert(NW * AT_ONCE * 16 * PITCH * 4 <= LDS);
  static_assert(WK <= 2 && S >= 2 && TOK >= 64 && ROWS >= 64 && FT >= 4 && S * LOADS < 64);
  static_assert(TOK / 64 + ROWS / 64 <= GROUP);                 // one wave for each 64 exponents or scales
  static_assert(WK == 1 || GROUP * FT * FW * 1024 <= LDS);           // the groups' sums change hands there
  // a word of exponents is loaded S WK blocks ahead, over one whose blocks are behind: not more than four
  static_assert(S * WK <= 4);
};

template <int AK, bool FS, bool PREC, int WT, int WW, int WK, int FT, int FW>
__global__ void __launch_bounds__(64 * WT * WW * WK, (Tile<WT, WW, WK, FT, FW>::PER_SIMD))
gemm8_kernel(F8Product p) {
  using P = Tile<WT, WW, WK, FT, FW>;
  constexpr int TOK = P::TOK, ROWS = P::ROWS, GROUP = P::GROUP, S = P::S;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = uniform(tid >> 6), wk = wave / GROUP, wg = wave % GROUP, wt = wg % WT, ww = wg / WT;

  // ---- which tile: token tiles in fours, the rows inside, so that the
  // workgroups of an XCD (every eighth block) share both operands in its L2
  int tiles = p.token_tiles;
  Runs runs{};
  if (p.offsets) {
    tiles = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      runs = load_runs(p, e0, tiles, TOK, lane);
      tiles = uniform(__shfl(runs.upto, 63));
    }
  }
  const int RT = p.row_blocks, total = tiles * RT * p.slices, chunk = (total + 7) / 8;
  const int block = p.block0 + static_cast<int>(blockIdx.x);
  if (block >> 3 >= chunk) return;
  const int at = (block & 7) * chunk + (block >> 3);
  if (at >= total) return;
  const int slice = p.slices == 1 ? 0 : at / (tiles * RT), here = at - slice * tiles * RT;
  const int four = here / (4 * RT), in = here - four * 4 * RT, wide4 = min(4, tiles - 4 * four);
  const int tile = 4 * four + in % wide4, rt = in / wide4;
  int expert = 0, row0 = tile * TOK, row_end = p.R;
  if (p.offsets) {
    const bool found = p.E <= 64 ? find_in(runs, 0, tile, TOK, expert, row0, row_end)
                                 : find_run(p, tile, TOK, lane, expert, row0, row_end);
    if (!found) return;
  }
  const int tokens = min(TOK, row_end - row0);
  const int half = p.m / 2, out_m = p.gated ? half : p.m;
  const int out0 = rt * (p.gated ? ROWS / 2 : ROWS);

  // ---- sources of this wave's loads.  Of a wave's FW row tiles the first half are the
  // gate's and the others the up rows of the same outputs.
  auto weight_row = [&](int lr) {
    if (!p.gated) return min(out0 + lr, p.m - 1);
    const int w = lr / (16 * FW), j = lr / 16 % FW;
    return min(out0 + w * (16 / 2) * FW + j % (FW / 2) * 16 + lr % 16, half - 1) + (j < FW / 2 ? 0 : half);
  };
  auto token_row = [&](int lt) {
    int r = row0 + min(lt, tokens - 1);
    if (p.rows) {
      r = p.rows[r];
      r = r < 0 || r >= p.a_rows ? 0 : r;                // its sums are dropped below
    }
    return r;
  };
  const int64_t strips = (p.m + 127) / 128;
  const i32x4 ares = resource(p.a, p.a_rows * p.lda), eres = resource(p.exps, p.a_rows * p.lde);
  const i32x4 wres = resource(p.w + expert * p.w_matrix, p.w_matrix);
  const i32x4 sres = resource(static_cast<const uint8_t*>(p.scales) + expert * p.scales_matrix * (FS ? 4 : 1),
                              strips * p.lds * (FS ? 4 : 1));
  uint32_t a_src[P::IL], w_src[P::WL];
  // where piece x of row r of a tile lies, 16 lanes reading one piece of 16 rows apart
  auto place = [](int r, int x) { return x ^ (r >> 1 & 7); };
#pragma unroll
  for (int i = 0; i < P::IL; ++i) {
    const int lt = 8 * (wg + GROUP * i) + lane / 8;
    a_src[i] = static_cast<uint32_t>(token_row(lt)) * static_cast<uint32_t>(p.lda) + 16 * place(lt, lane % 8);
  }
#pragma unroll
  for (int i = 0; i < P::WL; ++i) {
    const int lr = 8 * (wg + GROUP * i) + lane / 8;
    w_src[i] = static_cast<uint32_t>(weight_row(lr)) * static_cast<uint32_t>(p.ldw) + 16 * place(lr, lane % 8);
  }
  // wave w of a group loads the exponents of 64 tokens, the scales of 64 rows, or nothing
  constexpr int EW = TOK / 64, SW = ROWS / 64;
  const uint32_t small_src =
      wg < EW ? static_cast<uint32_t>(token_row(64 * wg + lane)) * static_cast<uint32_t>(p.lde)
      : wg < EW + SW ? static_cast<uint32_t>(weight_row(64 * (wg - EW) + lane) / 128) *
                           static_cast<uint32_t>(p.lds) * (FS ? 4u : 1u)
                     : 0u;
  // this group's stages: every WK-th from wk of the slice's
  const int step0 = slice * p.slice_steps, steps = min(p.slice_steps, p.steps - step0);
  const int most = (steps + WK - 1) / WK, mine = (steps + WK - 1 - wk) / WK;
  const uint32_t lds0 = lds_address(lds) + wk * P::PART;
  auto step_of = [&](int n) { return step0 + min(n * WK + wk, steps - 1); };
  // past the end: the last one again, into a place that nobody reads
  auto issue = [&](int n, int slot) {
    const int q = step_of(n);
    const uint32_t base = lds0 + slot * P::STAGE;
#pragma unroll
    for (int i = 0; i < P::IL; ++i)
      load_to_lds(base + (wg + GROUP * i) * 1024, a_src[i], ares, q * 128);
#pragma unroll
    for (int i = 0; i < P::WL; ++i)
      load_to_lds(base + P::ROWS_AT + (wg + GROUP * i) * 1024, w_src[i], wres, q * 128);
    // every lane of an exponent load touches a line of its own: only when a new word begins
    const bool scales = wg >= EW && wg < EW + SW;
    const bool fresh = n == 0 || q >> 2 != (q - WK) >> 2;
    const uint32_t to = scales ? base + P::SCALES_AT + (wg - EW) * 256
                        : wg < EW && fresh ? lds0 + S * P::STAGE + (q >> 2 & 1) * TOK * 4 + wg * 256
                                           : lds0 + S * P::STAGE + 2 * TOK * 4;
    if (scales) load_word_to_lds(to, small_src, sres, FS ? q * 4 : q & ~3);
    else load_word_to_lds(to, wg < EW && fresh ? small_src : 0u, eres, q & ~3);
  };

  // ---- operands: all row tiles, and a ring of four token tiles
  f32x4 acc[FT][FW] = {};
  i32x8 a[4], b[FW];
  uint32_t ea[4], sb[FW];                                // exponents, still in words
  f32x4 sf[FS ? FW : 1];                                 // float32 scales of a lane's four rows
  // A lane's places in LDS; those of the ring move on with the stage that is read,
  // tiles are immediate offsets from them.
  uint32_t a_at[2], b_at[2], s_at, e_at;
  {
    const uint32_t at = c * 128 + 16 * place(c, g);
    a_at[0] = lds0 + wt * 16 * FT * 128 + at;
    b_at[0] = lds0 + P::ROWS_AT + ww * 16 * FW * 128 + at;
    a_at[1] = a_at[0] ^ 64;                               // (every other part is a multiple of 128)
    b_at[1] = b_at[0] ^ 64;
    s_at = lds0 + P::SCALES_AT + (ww * 16 * FW + (FS ? 4 * g : c)) * 4;
  }
  const uint32_t e0_at = lds0 + S * P::STAGE + (wt * 16 * FT + c) * 4;
  auto exponents_of = [&](int n) { e_at = e0_at + (step_of(n) >> 2 & 1) * TOK * 4; };
  auto a_moves = [&](uint32_t by) { a_at[0] += by; a_at[1] += by; };
  auto b_moves = [&](uint32_t by) { b_at[0] += by; b_at[1] += by; s_at += by; };
  auto read_tile = [&](const uint32_t (&at)[2], int offset, i32x8& v) {
    const i32x4 lo = lds_read<i32x4>(at[0], offset), hi = lds_read<i32x4>(at[1], offset);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = lo[2]; v[3] = lo[3];
    v[4] = hi[0]; v[5] = hi[1]; v[6] = hi[2]; v[7] = hi[3];
  };
  auto read_a = [&](int f) {
    read_tile(a_at, f * 16 * 128, a[f % 4]);
    ea[f % 4] = lds_read<uint32_t>(e_at, f * 16 * 4);
  };
  auto read_b = [&](int f) {
    read_tile(b_at, f * 16 * 128, b[f]);
    if constexpr (FS) sf[f] = lds_read<f32x4>(s_at, f * 16 * 4);
    else sb[f] = lds_read<uint32_t>(s_at, f * 16 * 4);
  };
  bf16x8 wb[PREC ? FW : 1][4];
  // a stage's exponents of the rows out of their words, and its rows in bfloat16
  auto begin = [&](int shift) {
    if constexpr (!FS) {
#pragma unroll
      for (int j = 0; j < FW; ++j) sb[j] >>= shift;
    }
    if constexpr (PREC) {
#pragma unroll
      for (int j = 0; j < FW; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wb[j][i] = widen8<LQ_E4M3>(b[j][2 * i], b[j][2 * i + 1],
                                     FS ? 1.f : power_of_two(sb[j] & 255));
    }
  };
  // The products of token tile t; `after(j)` follows that with row tile j.
  auto products = [&](int t, int shift, auto&& after) {
    const uint32_t e = ea[t % 4] >> shift;
    bf16x8 wa[4];
    if constexpr (PREC) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        wa[i] = widen8<AK>(a[t % 4][2 * i], a[t % 4][2 * i + 1], power_of_two(e & 255));
    }
#pragma unroll
    for (int j = 0; j < FW; ++j) {
      f32x4& to = acc[t][j];
      constexpr int B = AK == LQ_E5M2 ? 1 : 0;
      if constexpr (PREC) {
        f32x4 z = FS ? f32x4{} : to;
#pragma unroll
        for (int i = 0; i < 4; ++i) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][i], wa[i], z, 0, 0, 0);
        to = FS ? to + z * sf[j] : z;
      } else if constexpr (FS) {
        const f32x4 z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[t % 4], f32x4{}, 0, B, 0, 127, 0, e);
        to += z * sf[j];
      } else {
        to = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[t % 4], to, 0, B, 0, sb[j], 0, e);
      }
      after(j);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

#pragma unroll
  for (int i = 0; i < S; ++i) issue(i, i);
  wait_and_barrier<(S - 1) * P::LOADS>();
  exponents_of(0);
#pragma unroll
  for (int i = 0; i < FW; ++i) read_b(i);
#pragma unroll
  for (int i = 0; i < 4; ++i) read_a(i);
  // The scheduling barriers keep the order: a token tile's products, then the reads
  // that refill its place, four tiles ahead of their use.  The last stage refills
  // nothing; a group without one skips it.
  int slot = 0;
  for (int n = 0; n + 1 < most; ++n) {
    const int next = slot + 1 == S ? 0 : slot + 1, shift = 8 * (step_of(n) & 3);
    const uint32_t on = static_cast<uint32_t>((next - slot) * P::STAGE);
    begin(shift);
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      products(t, shift, [&](int j) {
        if (t == FT - 1) {
          __builtin_amdgcn_sched_barrier(0);
          read_b(j);
        }
      });
      if (t == FT - 4) {
        // the next stage has landed and nobody reads this one's place any more
        wait_and_barrier<(S - 2) * P::LOADS>();
        issue(n + S, slot);
        a_moves(on);
        b_moves(on);
        exponents_of(n + 1);
      }
      read_a((t + 4) % FT);
      __builtin_amdgcn_sched_barrier(0);
    }
    slot = next;
  }
  if (WK == 1 || mine == most) {
    const int shift = 8 * (step_of(most - 1) & 3);
    begin(shift);
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      products(t, shift, [](int) {});
      if (t + 4 < FT) read_a(t + 4);
    }
  }

  // ---- the groups' halves change hands: each finishes half of the token tiles
  constexpr int LAST = WK == 1 ? FT : FT / 2;
  if constexpr (WK == 2) {
    wait_and_barrier<0>();
    f32x4* ex = reinterpret_cast<f32x4*>(lds) + lane;
    auto slot_of = [&](int group, int t, int j) { return ((group * GROUP + wg) * LAST + t) * FW + j; };
#pragma unroll
    for (int t = 0; t < LAST; ++t)
#pragma unroll
      for (int j = 0; j < FW; ++j)
        ex[slot_of(1 - wk, t, j) * 64] = wk ? acc[t][j] : acc[LAST + t][j];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < LAST; ++t)
#pragma unroll
      for (int j = 0; j < FW; ++j) {
        const f32x4 other = ex[slot_of(wk, t, j) * 64];
        acc[t][j] = wk ? other + acc[LAST + t][j] : acc[t][j] + other;
      }
  }

  // ---- the end: AT_ONCE token tiles at a time through the wave's own part of LDS, [token][row],
  // so that its stores are whole runs and its code short (unrolled over all the sums it would be
  // 100 KB, fetched once per tile: 15 us of each).  Without a residual no load stands between
  // the stores: a wait for one is a wait for the stores before it.  Tiles of 256 rows store past
  // the caches, which their operands need: outputs from 12 MB, the smallest that take these tiles
  // (1664 x 4096 -> 4096, 14 MB: 37.2 us, plain stores 38.4; 512 tokens to 8 of 64 experts 84 and
  // 90; 4096 x 4096 -> 28672, 235 MB: 434 and 443), also where lq_quant8 reads the output next
  // (both calls: 40.7 and 41.4; 93 and 96; 495 and 502; nothing at 117 MB, 447 and 446).
  constexpr bool STREAM = ROWS > 128;
  constexpr int PITCH = P::PITCH, AT_ONCE = P::AT_ONCE, MASKS = (LAST + 3) / 4, G = 4;
  const int wave_token = wt * 16 * FT + (WK == 2 && wk ? 16 * LAST : 0);
  uint64_t live[MASKS];                                  // of the wave's tokens: whether their index is one
#pragma unroll
  for (int i = 0; i < MASKS; ++i) {
    const int token = wave_token + 64 * i + lane;
    int r = 0;
    if (p.rows && token < tokens) r = p.rows[row0 + token];
    live[i] = __ballot(r >= 0 && r < p.a_rows);
  }
  // a lane keeps its four columns and goes through the tokens
  const int shift = (FW == 4 ? 4 : 3) - (p.gated ? 1 : 0), apart = 64 >> shift, first = lane >> shift;
  const int o_in = (lane & ((1 << shift) - 1)) * 4, o = out0 + ww * (p.gated ? 16 * FW / 2 : 16 * FW) + o_in;
  const int n = min(4, out_m - o);
  float bias[4] = {}, bias_up[4] = {};
  if (p.bias && slice == 0) {
    const float* from = p.bias + static_cast<int64_t>(expert) * p.m + o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < n) bias[i] = from[i];
      if (i < n && p.gated) bias_up[i] = from[half + i];
    }
  }
  // (they have arrived before the stores begin)
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(bias[i]), "+v"(bias_up[i]));
  if constexpr (WK == 1) wait_and_barrier<0>();
  else __syncthreads();
  float* ex = reinterpret_cast<float*>(lds) + wave * AT_ONCE * 16 * PITCH;
#pragma unroll
  for (int f0 = 0; f0 < LAST; f0 += AT_ONCE) {
#pragma unroll
    for (int t = 0; t < AT_ONCE; ++t)
#pragma unroll
      for (int j = 0; j < FW; ++j)
        *reinterpret_cast<f32x4*>(ex + (16 * t + c) * PITCH + 16 * j + 4 * g) = acc[f0 + t][j];
    const uint64_t alive = live[f0 / 4] >> (16 * (f0 % 4));
#pragma unroll 1
    for (int at0 = first; at0 < AT_ONCE * 16; at0 += G * apart) {
      const int token0 = wave_token + 16 * f0 + at0;
      auto inside = [&](int i) { return token0 + i * apart < tokens ? n : 0; };
      Residual res[G];
      if (p.residual) {
#pragma unroll
        for (int i = 0; i < G; ++i)
          res[i] = load_residual(inside(i), p.out_dt, p.residual,
                                 static_cast<int64_t>(row0 + token0 + i * apart) * p.ldr + o);
      }
      auto finished = [&](int column, const float (&b)[4], float (&y)[4 * G]) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const f32x4 z = *reinterpret_cast<const f32x4*>(ex + (at0 + i * apart) * PITCH + column);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[4 * i + j] = z[j];
        }
        if (p.rows) {
#pragma unroll
          for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[4 * i + j] = alive >> (at0 + i * apart) & 1 ? y[4 * i + j] : 0.f;
        }
        if (p.bias) {
#pragma unroll
          for (int i = 0; i < 4 * G; ++i) y[i] += b[i % 4];
        }
      };
      float y[4 * G];
      finished(o_in, bias, y);
      activate(y, p.act);
      if (p.gated) {
        float up[4 * G];
        finished(o_in + 16 * FW / 2, bias_up, up);
#pragma unroll
        for (int i = 0; i < 4 * G; ++i) y[i] *= up[i];
      }
      float y4[G][4];
#pragma unroll
      for (int i = 0; i < 4 * G; ++i) y4[i / 4][i % 4] = y[i];
      if (p.residual) {
#pragma unroll
        for (int i = 0; i < G; ++i) add_residual(y4[i], p.out_dt, res[i]);
      }
      const int64_t to = (row0 + token0 + static_cast<int64_t>(slice) * p.R) * p.ldo + o;
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (inside(i) > 0) store4<STREAM>(y4[i], n, p.out_dt, p.out, to + i * apart * p.ldo);
    }
  }
}

template <int AK, bool FS, bool PREC, int WT, int WW, int WK, int FT, int FW>
hipError_t launch(const F8Product& in, hipStream_t st) {
  using P = Tile<WT, WW, WK, FT, FW>;
  F8Product p = in;
  const int64_t outs = p.gated ? P::ROWS / 2 : P::ROWS, out_m = p.gated ? p.m / 2 : p.m;
  p.row_blocks = static_cast<int>((out_m + outs - 1) / outs);
  int64_t tiles = (p.R + P::TOK - 1) / P::TOK;
  if (p.offsets) tiles = p.R / P::TOK + (p.E < p.R ? p.E : p.R);
  p.token_tiles = static_cast<int>(tiles);
  const int64_t grid = (tiles * p.row_blocks * p.slices + 7) / 8 * 8;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  auto* k = gemm8_kernel<AK, FS, PREC, WT, WW, WK, FT, FW>;
  // per call: the attribute belongs to the current device
  const hipError_t big = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, P::LDS);
  if (big != hipSuccess) return big;
  // a launch has fewer than 2^32 threads
  constexpr int64_t kMost = (int64_t{1} << 31) / (64 * P::NW);
  for (int64_t b = 0; b < grid; b += kMost) {
    p.block0 = static_cast<int>(b);
    k<<<static_cast<uint32_t>(grid - b < kMost ? grid - b : kMost), 64 * P::NW, P::LDS, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int AK, bool FS, bool PREC>
hipError_t by_shape(const F8Product& p, int shape, hipStream_t st) {
  if constexpr (!FS && !PREC) {
    if (shape == kSquare) return launch<AK, FS, PREC, 2, 4, 1, 8, 4>(p, st);
    if (shape == kTall) return launch<AK, FS, PREC, 2, 4, 1, 4, 4>(p, st);
  }
  if (shape == kPair) return launch<AK, FS, PREC, 2, 2, 1, 4, 4>(p, st);
  // larger pieces of the tile where a wave works on each operand it reads (float32 results
  // convert it, float32 scales multiply its sums)
  if constexpr (PREC || FS) return launch<AK, FS, PREC, 2, 2, 2, 4, 4>(p, st);
  else return launch<AK, FS, PREC, 2, 4, 1, 4, 2>(p, st);
}

template <int AK>
hipError_t by_scales(const F8Product& p, int shape, bool precise, hipStream_t st) {
  if (precise) return p.float_scales ? by_shape<AK, true, true>(p, shape, st) : by_shape<AK, false, true>(p, shape, st);
  return p.float_scales ? by_shape<AK, true, false>(p, shape, st) : by_shape<AK, false, false>(p, shape, st);
}

}  // namespace

F8ManyPlan many_f8_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, bool grouped,
                        bool float_scales, bool precise) {
  F8ManyPlan p{};
  const int64_t cus = num_cus(), steps = (K + 127) / 128;
  const int64_t runs = grouped ? (E < R ? E : R) : 1, out_m = gated ? m / 2 : m;
  auto count = [&](int tok, int rows) {
    const int64_t outs = gated ? rows / 2 : rows;
    const int64_t tiles = grouped ? R / tok + (runs + 1) / 2 : (R + tok - 1) / tok;
    return tiles * ((out_m + outs - 1) / outs);
  };
  // Tiles of tokens x rows, measured on each side.  Where exponents alone are applied by the
  // matrix instruction: 256 x 256 and 128 x 256 in eight waves, one workgroup on a unit, or 128
  // x 128 in four, two of them (4096 x 4096 -> 2 x 14336: 397 us, 465, 456; 2048 x 8192 -> 8192:
  // 131, 154, 147; of 2100 rows 199, 176, 156).  Of one matrix the fewest rounds of the units'
  // tiles decide, priced by these rates, a last round of single workgroups 1.4 of 2.3 (700 x
  // 4096 -> 14336: 128 x 256 66, 128 x 128 58).  Of runs, whose tiles are only estimated, 256 x
  // 256 if they are long (64 experts, 2048 -> 2 x 1408, 512 rows each: 270, 128 x 256 306; 256
  // rows each: 186, 173, 128 x 128 190). Float32 scales or results: 128 x 128 in four waves, two
  // workgroups on a unit (4096 x 4096 -> 2 x 14336 with float32 scales 524, 128 x 256 561; to
  // float32 811, 867).  Where no unit has more than one such tile (520 x 8192 -> 8192, 320 of
  // them: 64, one at a time 82), eight waves share it, 64 x 32 each (512 x 8192 -> 8192: 41; 64
  // x 64 in four waves 46); for float32 scales or results 64 x 64, four waves for every other
  // block of positions (the same with float32 scales 44, 64 x 32 each 48, four waves 55; to
  // float32 64; 77; 77).
  const bool quick = !float_scales && !precise;
  auto rounds = [&](int64_t n) { return (n + cus - 1) / cus; };
  const int64_t square = rounds(count(256, 256)) * 40, tall = rounds(count(128, 256)) * 23;
  const int64_t pairs = count(128, 128), rest = pairs % (2 * cus);
  const int64_t pair = pairs / (2 * cus) * 23 + (rest > cus ? 23 : rest ? 14 : 0);
  if (quick && !grouped && count(128, 256) * 5 >= cus * 4)
    p.shape = square <= tall && square <= pair ? kSquare : tall <= pair ? kTall : kPair;
  else if (quick && grouped && count(256, 256) >= cus && R >= 512 * runs) p.shape = kSquare;
  else if (quick && count(128, 256) * 5 >= cus * 4) p.shape = kTall;
  else if (pairs > cus) p.shape = kPair;
  else p.shape = kOne;
  // Where tiles leave units without one, the positions are split, down to 1024 a
  // slice (777 x 5125 -> 1281: one 28, three 22; 64 x 14336 -> 4096: one 67, eight 22).
  p.slices = 1;
  const int64_t tiles = count(128, 128);
  if (p.shape == kOne && tiles < cus) {
    p.slices = static_cast<int>(cus / tiles);
    if (p.slices > steps / 8) p.slices = static_cast<int>(steps / 8);
    if (p.slices > 16) p.slices = 16;
    if (p.slices < 1) p.slices = 1;
  }
  p.slice_steps = static_cast<int>((steps + p.slices - 1) / p.slices);
  p.slices = static_cast<int>((steps + p.slice_steps - 1) / p.slice_steps);
  return p;
}

hipError_t launch_gemm8(const F8Product& p, int a_type, const F8ManyPlan& plan, bool precise, hipStream_t st) {
  return a_type == LQ_E5M2 ? by_scales<LQ_E5M2>(p, plan.shape, precise, st)
                           : by_scales<LQ_E4M3>(p, plan.shape, precise, st);
}

}  // namespace lq
