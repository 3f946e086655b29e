// Product of 1-bit weights with 16-bit lifted activations for many tokens,
// on the matrix cores in float4 (signs) x float6 (activation parts,
// f6_parts.h), with the epilogue of lq_gemm_ep and the ragged expert runs of
// lq_gemm_grouped.
//
// Tile.  A workgroup of WR WK waves takes 128 WR rows of the weights and 32 TT
// tokens; the weights cost 1/8 byte per position and the parts 2.4 to 3.9, so the
// tile is tall.  WK waves share each 128-row strip and split the positions of
// a stage; every wave holds 128 rows x 32 TT tokens of sums (4 TT tiles of
// 32 x 32) and uses each operand it reads from LDS four times.  Operands come
// to LDS by loads that write it directly (buffer_load ... lds, 16 bytes per
// lane): the tokens' parts in stages of SEC groups of 128 positions (a ring
// of S), the signs in units of 256 positions, 32 bytes per row (two units; a
// 16-byte piece per row and stage would ask L2 for the same lines twice as
// often).  A wave reads an operand of the next step into the registers of the
// one it has just used, so the only wait in the loop is the stage barrier,
// which sits behind the first products of a step.  Workgroups of four waves
// use half a compute unit's LDS, so that two of them share it and one's
// barriers, first loads and epilogue are covered by the other's products.
//
// The loads to LDS are inline assembly (they have no output register) so
// that the waits on them can be counted by hand: the compiler would drain
// them before every read of LDS.  Every wave issues the same number per
// stage (the last ones repeat a chunk).
//
// Measured (MI355X, kernel trace, least and median): 4096 x 8192 -> 2 x 14336
// gated, three parts, 1114 and 1144 us, 1.73 PFLOP/s of lifted product; 16384
// rows of 64 experts, 4096 -> 2 x 1408, 298 and 317, 1.27; 512 x 20480 -> 8192 to
// float16, four parts, 157 and 180, 1.09 (three took 127); 3000 rows of 8
// experts, 28672 -> 4096, four parts, 682 and 709, 1.03.  Bound by power: the
// matrix cores are busy 72 % of the cycles at 1.5 GHz; the instruction alone on
// random operands gives 2.0 to 2.1 with three parts.
//
// End.  The tiles go through LDS, 32 tokens at a time, where the WK partial
// sums are added in a fixed order and rows become consecutive, so stores are
// whole runs.
#include "f6_epilogue.h"
#include "f6_parts.h"
#include "f6_product.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

constexpr uint32_t kRsrcWord3 = 0x00020000u;

__device__ __forceinline__ f32x16 mfma(const i32x8& a, const i32x8& b, const f32x16& c, int scale) {
  // A: E2M1 (cbsz 4), scale 2^0; B: E2M3 (blgp 2), scale 2^(scale - 127)
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 2, 0, 127, 0, scale);
}

// 64 lanes x 16 bytes from resource r at voff + soff to LDS at `lds` (bytes).
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voff, const i32x4& r,
                                            uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(r), "s"(soff)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

__device__ __forceinline__ i32x4 resource(const void* p, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(u));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32) & 0xFFFF);
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  r[3] = static_cast<int>(kRsrcWord3);
  return r;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int NP, int WR, int WK, int TT, bool ONE>
struct Shape {
  static constexpr int NW = WR * WK;                   // waves
  static constexpr int SEC = WK == 4 ? 2 : 1;          // groups per stage
  static constexpr int NU = 2 * SEC / WK;              // steps of a wave per stage
  static constexpr int UNIT = 2 / SEC;                 // stages per unit of signs
  static constexpr int TOK = 32 * TT;
  static constexpr int ROWS = 128 * WR;
  static constexpr int GB = group_bytes(2, NP);
  static constexpr int CH = GB / 16;
  static constexpr int IMG_CHUNKS = SEC * TOK * CH;
  static constexpr int IMG_LOADS = (IMG_CHUNKS + 63) / 64;
  static constexpr int IL = (IMG_LOADS + NW - 1) / NW;  // loads of parts per wave and stage
  static constexpr int WL = ROWS / 32 / NW;             // loads of signs per wave and unit
  static constexpr int STAGE = IMG_LOADS * 1024;
  static constexpr int SIGNS = ROWS * 32;               // a unit of signs
  // a workgroup to itself on a compute unit, or two of four waves
  static constexpr int MAX_LDS = ONE ? 163840 : 81920;
  static constexpr int RING = UNIT == 1 ? MAX_LDS / (STAGE + SIGNS) : (MAX_LDS - 2 * SIGNS) / STAGE;
  static constexpr int S_MOST = UNIT == 1 ? 6 : 4;
  static constexpr int S = RING > S_MOST ? S_MOST : RING;
  static constexpr int SR = UNIT == 1 ? S : 2;         // units of signs in LDS
  // loads that may still be on their way when the next stage and its signs
  // must have landed: those of the stages behind it
  static constexpr int WAIT = (S - 2) * (UNIT == 1 ? IL + WL : IL);
  static constexpr int PITCH = 132;                    // floats per token in the final exchange
  static constexpr int EXCHANGE = NW * 32 * PITCH * 4;
  static constexpr int OPERANDS = S * STAGE + SR * SIGNS;
  static constexpr int LDS = OPERANDS > EXCHANGE ? OPERANDS : EXCHANGE;
  static_assert(S >= 2 && LDS <= MAX_LDS && NU >= 1 && WL >= 1);
  static_assert((S - 1) * (IL + WL) + WL < 64);
};

template <int NP, int WR, int WK, int TT, bool ONE>
__global__ void __launch_bounds__(64 * WR * WK, 2) gemm_f6_kernel(F6Product a) {
  using P = Shape<NP, WR, WK, TT, ONE>;
  constexpr int SEC = P::SEC, NU = P::NU, TOK = P::TOK, ROWS = P::ROWS, NW = P::NW;
  extern __shared__ __align__(1024) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wr = wave % WR, wk = wave / WR;

  // ---- which tile: token tiles in pairs, the rows inside, so that the
  // workgroups of an XCD (every eighth block) share parts and signs in its L2
  const int RT = a.row_tiles;
  int tiles = a.token_tiles;
  Runs runs{};                           // of the last 64 experts: all of them up to 64
  if (a.offsets) {
    tiles = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      runs = load_runs(a, e0, tiles, TOK, lane);
      tiles = uniform(__shfl(runs.upto, 63));
    }
  }
  const int total = tiles * RT * a.slices;
  const int chunk = (total + 7) / 8;
  const int block = a.block0 + static_cast<int>(blockIdx.x);
  if (block >> 3 >= chunk) return;
  const int at = (block & 7) * chunk + (block >> 3);
  if (at >= total) return;
  const int slice = a.slices == 1 ? 0 : at / (tiles * RT), here = at - slice * tiles * RT;
  const int pair = here / (2 * RT), in = here - pair * 2 * RT;
  const int wide = min(2, tiles - 2 * pair);
  int tile = 2 * pair + in % wide;
  const int rt = in / wide;
  int expert = 0, row0, row_end = a.R;
  if (a.offsets) {
    const bool found = a.E <= 64 ? find_in(runs, 0, tile, TOK, expert, row0, row_end)
                                 : find_run(a, tile, TOK, lane, expert, row0, row_end);
    if (!found) return;
  } else {
    row0 = tile * TOK;
  }
  const int tokens = min(TOK, row_end - row0);

  const uint32_t* w = a.w + static_cast<int64_t>(expert) * a.m * a.ldw;
  const float* s = a.s + static_cast<int64_t>(expert) * a.m;
  const float* bias = a.bias && slice == 0 ? a.bias + static_cast<int64_t>(expert) * a.m : nullptr;
  const int half_m = a.m / 2;
  const int outs = a.gated ? ROWS / 2 : ROWS;          // outputs of the tile
  const int out0 = rt * outs;
  const int out_m = a.gated ? half_m : a.m;

  // ---- sources of this wave's loads: loads wave, wave + NW, ... of a stage
  // (past the last one: the last again) and of a unit of signs
  const i32x4 ires = resource(a.img, a.img_bytes);
  const i32x4 wres = resource(w, static_cast<uint32_t>(a.m) * a.ldw * 4u);
  uint32_t part_src[P::IL], sign_src[P::WL];
#pragma unroll
  for (int i = 0; i < P::IL; ++i) {
    const int c = min(min(wave + NW * i, P::IMG_LOADS - 1) * 64 + lane, P::IMG_CHUNKS - 1);
    const int sec = c / (TOK * P::CH), t = c / P::CH % TOK, ch = c % P::CH;
    int r = row0 + min(t, tokens - 1);
    if (a.rows) {
      r = a.rows[r];
      r = r < 0 || r >= a.src_rows ? a.src_rows : r;   // the image's row of zeros
    }
    part_src[i] = static_cast<uint32_t>(r) * a.img_row_bytes + sec * P::GB + ch * 16;
  }
#pragma unroll
  for (int i = 0; i < P::WL; ++i) {
    const int c = (wave + NW * i) * 64 + lane, lr = c / 2;
    int row;
    if (a.gated)
      row = min(out0 + lr / 128 * 64 + (lr & 63), half_m - 1) + ((lr >> 6) & 1) * half_m;
    else
      row = min(out0 + lr, a.m - 1);
    sign_src[i] = static_cast<uint32_t>(row) * a.ldw * 4u + (c & 1) * 16;
  }
  // this slice's units of 256 positions
  const int unit0 = slice * a.slice_units, units = min(a.slice_units, a.groups / 2 - unit0);
  const int stages = units * P::UNIT, stage0 = unit0 * P::UNIT;
  const uint32_t lds0 = lds_address(lds);
  constexpr int SIGNS_AT = P::S * P::STAGE;
  // past the end: the last one again, into a slot nobody reads
  auto issue_parts = [&](int stage, int slot) {
    const uint32_t off = (stage0 + min(stage, stages - 1)) * SEC * P::GB;
#pragma unroll
    for (int i = 0; i < P::IL; ++i)
      load_to_lds(lds0 + slot * P::STAGE + min(wave + NW * i, P::IMG_LOADS - 1) * 1024,
                  part_src[i], ires, off);
  };
  auto issue_signs = [&](int unit, int slot) {
    const uint32_t off = (unit0 + min(unit, units - 1)) * 32;
#pragma unroll
    for (int i = 0; i < P::WL; ++i)
      load_to_lds(lds0 + SIGNS_AT + slot * P::SIGNS + (wave + NW * i) * 1024, sign_src[i],
                  wres, off);
  };

  // ---- operands
  const int i32 = lane & 31, h = lane >> 5;
  const uint32_t two = held(0x22222222u);
  f32x16 acc[4][TT] = {};
  i32x8 b[TT][NP], sign[4];
  uint32_t word[4][NU], ex[TT];            // of a stage: every step of the wave
  int scale[TT][NP];
  auto step_group = [&](int) { return SEC == 2 ? wk >> 1 : 0; };
  auto step_u = [&](int u) { return SEC == 2 ? wk & 1 : wk * NU + u; };
  auto read_part = [&](int slot, int u, int t, int p) {
    const uint8_t* g = lds + slot * P::STAGE + step_group(u) * TOK * P::GB +
                       (32 * t + i32) * P::GB;
    const int at2 = (step_u(u) * NP + p) * 2 + h;
    const int4 lo = *reinterpret_cast<const int4*>(g + 16 * at2);
    const int2 hi = *reinterpret_cast<const int2*>(g + tail_offset(2, NP) + 8 * at2);
    b[t][p][0] = lo.x; b[t][p][1] = lo.y; b[t][p][2] = lo.z; b[t][p][3] = lo.w;
    b[t][p][4] = hi.x; b[t][p][5] = hi.y; b[t][p][6] = 0; b[t][p][7] = 0;
  };
  auto read_exponents = [&](int slot) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
      ex[t] = *reinterpret_cast<const uint32_t*>(
          lds + slot * P::STAGE + step_group(0) * TOK * P::GB + (32 * t + i32) * P::GB +
          exp_offset(2, NP));
  };
  auto set_scales = [&](int u) {
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int p = 0; p < NP; ++p)
        scale[t][p] = static_cast<int>(ex[t] >> (16 * h + 8 * step_u(u)) & 255u) - part_shift(p);
  };
  // j: group of the pair that the unit covers; one step's word, or both
  auto read_words = [&](int slot, int j) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint8_t* at = lds + SIGNS_AT + slot * P::SIGNS + (wr * 128 + 32 * q + i32) * 32 +
                          h * 16 + 8 * (j + step_group(0));
      if constexpr (NU == 2) {
        const uint2 w2 = *reinterpret_cast<const uint2*>(at);
        word[q][0] = w2.x;
        word[q][1] = w2.y;
      } else {
        word[q][0] = *reinterpret_cast<const uint32_t*>(at + 4 * step_u(0));
      }
    }
  };

#pragma unroll
  for (int i = 0; i < P::S; ++i) {
    if (i < P::SR) issue_signs(i, i);
    issue_parts(i, i);
  }
  wait_and_barrier<(P::SR - 1) * P::WL + (P::S - 1) * P::IL>();
  read_words(0, 0);
  read_exponents(0);
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int p = 0; p < NP; ++p) read_part(0, 0, t, p);
#pragma unroll
  for (int q = 0; q < 4; ++q) sign[q] = expand_signs(word[q][0], two);
  set_scales(0);

  // The order below is kept by the scheduling barriers: four products, then
  // the reads that refill their operand; the next step's signs are expanded
  // between the step's last products, each as its operand is free.
  int slot = 0, sign_slot = 0;
  for (int unit = 0; unit < units; ++unit) {
    const int next_sign = sign_slot + 1 == P::SR ? 0 : sign_slot + 1;
#pragma unroll
    for (int j = 0; j < P::UNIT; ++j) {
      const int next = slot + 1 == P::S ? 0 : slot + 1;
      const bool unit_ends = j == P::UNIT - 1;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const bool last = u == NU - 1;
        const int nslot = last ? next : slot, nu = last ? 0 : u + 1;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bool refill = t == TT - 1 && p == NP - 1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[q][t] = mfma(sign[q], b[t][p], acc[q][t], scale[t][p]);
              if (refill) {
                __builtin_amdgcn_sched_barrier(0);
                sign[q] = expand_signs(word[q][nu], two);
              }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (t == 0 && p == 0) {
              if (last) {
                // the next stage has landed and nobody reads this one any more
                wait_and_barrier<P::WAIT>();
                if (unit_ends) issue_signs(unit + P::SR, sign_slot);
                issue_parts(unit * P::UNIT + j + P::S, slot);
                if (unit_ends) read_words(next_sign, 0);
                else read_words(sign_slot, j + 1);
                read_exponents(nslot);
              }
            }
            read_part(nslot, nu, t, p);
            if (refill) set_scales(nu);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      slot = next;
    }
    sign_slot = next_sign;
  }
  wait_and_barrier<0>();

  // ---- the exchange: [wave][token][row], 32 tokens at a time.  A thread
  // keeps its four output columns and takes every (512 / quads)-th token, so
  // scales, bias and column offsets are its own for the whole tile.
  float* ex32 = reinterpret_cast<float*>(lds);
  const int shift = __builtin_ctz(ROWS / 4) - (a.gated ? 1 : 0);   // log2 of the quads of a row
  const int o = (tid & ((1 << shift) - 1)) * 4, tk0 = tid >> shift, tk_step = 64 * NW >> shift;
  const int n = min(4, out_m - (out0 + o));
  const int strip = a.gated ? o / 64 : o / 128;
  const float* z0 = ex32 + strip * 32 * P::PITCH + (a.gated ? o % 64 : o % 128);
  const OutputTypes types = output_types(a.out, a.ldo, a.residual, a.ldr, a.out_dt);
  const RowScales rs = row_scales(s, bias, out0 + o, a.m);
  RowScales up = rs;
  if (a.gated) up = row_scales(s, bias, half_m + out0 + o, a.m);
  const int64_t slice_row = row0 + static_cast<int64_t>(slice) * a.R;
  // a chunk of tokens: their residuals are on their way before the sums are added
  constexpr int CHUNK = 16 / WK < 4 ? 16 / WK : 4;
  auto load_chunk = [&](int t, int tk, Residual (&r)[CHUNK]) {
#pragma unroll
    for (int c = 0; c < CHUNK; ++c) {
      const int token = 32 * t + tk + c * tk_step;
      const bool live = tk + c * tk_step < 32 && token < tokens;
      r[c] = load_residual(live ? n : 0, types, a.residual, (slice_row + token) * a.ldr + out0 + o);
    }
  };
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    Residual r[CHUNK];
    load_chunk(t, tk0, r);
    if (t) __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4)
        *reinterpret_cast<float4*>(ex32 + (wave * 32 + i32) * P::PITCH + 32 * q + 8 * r4 + 4 * h) =
            make_float4(acc[q][t][4 * r4], acc[q][t][4 * r4 + 1], acc[q][t][4 * r4 + 2],
                        acc[q][t][4 * r4 + 3]);
    __syncthreads();
    const int stop = n > 0 ? min(32, tokens - 32 * t) : 0;
    for (int tk = tk0; tk < stop; tk += CHUNK * tk_step) {
      Residual next[CHUNK];
      load_chunk(t, tk + CHUNK * tk_step, next);
#pragma unroll
      for (int c = 0; c < CHUNK; ++c) {
        const int token = tk + c * tk_step;
        if (token >= stop) break;
        const float* z = z0 + token * P::PITCH;
        auto sum = [&](const float* from) {            // the WK partial sums, in order
          float4 v = *reinterpret_cast<const float4*>(from);
#pragma unroll
          for (int k = 1; k < WK; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(from + k * WR * 32 * P::PITCH);
            v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
          }
          return v;
        };
        float y[4];
        scaled(sum(z), rs, y);
        activate4(y, a.act);
        if (a.gated) {
          float g[4];
          scaled(sum(z + 64), up, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] *= g[j];
        }
        store4(y, n, types, r[c], a.residual != nullptr, a.out,
               (slice_row + 32 * t + token) * a.ldo + out0 + o);
      }
#pragma unroll
      for (int c = 0; c < CHUNK; ++c) r[c] = next[c];
    }
  }
}

template <int NP, int WR, int WK, int TT, bool ONE>
hipError_t launch(const F6Product& p, hipStream_t st) {
  using P = Shape<NP, WR, WK, TT, ONE>;
  F6Product a = p;
  const int64_t outs = a.gated ? P::ROWS / 2 : P::ROWS;
  const int64_t out_m = a.gated ? a.m / 2 : a.m;
  a.row_tiles = static_cast<int>((out_m + outs - 1) / outs);
  int64_t tiles = (a.R + P::TOK - 1) / P::TOK;
  if (a.offsets) tiles = a.R / P::TOK + (a.E < a.R ? a.E : a.R);
  a.token_tiles = static_cast<int>(tiles);
  const int64_t grid = (tiles * a.row_tiles * a.slices + 7) / 8 * 8;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  auto* k = gemm_f6_kernel<NP, WR, WK, TT, ONE>;
  // per call: the attribute belongs to the current device
  const hipError_t big = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, P::LDS);
  if (big != hipSuccess) return big;
  // a launch has fewer than 2^32 threads: more workgroups go in several
  constexpr int64_t kMost = (int64_t{1} << 31) / (64 * P::NW);
  for (int64_t b = 0; b < grid; b += kMost) {
    a.block0 = static_cast<int>(b);
    k<<<dim3(static_cast<uint32_t>(grid - b < kMost ? grid - b : kMost)), 64 * P::NW, P::LDS, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int NP>
hipError_t by_shape(const F6Product& p, int shape, hipStream_t st) {
  switch (shape) {
    case 4120: if constexpr (NP == 3) return launch<NP, 4, 1, 2, false>(p, st); break;
    case 2421: return launch<NP, 2, 4, 2, true>(p, st);
    case 2220: if constexpr (NP == 4) return launch<NP, 2, 2, 2, false>(p, st); break;
    case 4221: if constexpr (NP <= 4) return launch<NP, 4, 2, 2, true>(p, st); break;
    case 4110: return launch<NP, 4, 1, 1, false>(p, st);
    case 2210: return launch<NP, 2, 2, 1, false>(p, st);
    case 2411: return launch<NP, 2, 4, 1, true>(p, st);
    case 1410: return launch<NP, 1, 4, 1, false>(p, st);
    default: break;
  }
  return hipErrorInvalidValue;
}

}  // namespace

F6ManyPlan many_f6_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                        bool grouped) {
  F6ManyPlan p{};
  const int64_t cus = num_cus(), units = padded_positions(K) / 256;
  const int64_t runs = grouped ? (E < R ? E : R) : 1;
  const int64_t out_m = gated ? m / 2 : m;
  const bool two = R > 32 * runs;
  // tiles of 128 WR rows and 32 TT tokens; of runs, half end inside a tile
  auto count = [&](int WR, int TT) {
    const int64_t outs = (gated ? 64 : 128) * WR, tok = 32 * TT;
    const int64_t tiles = grouped ? R / tok + (runs + 1) / 2 : (R + tok - 1) / tok;
    return tiles * ((out_m + outs - 1) / outs);
  };
  auto up = [&](int64_t n) { return (n + cus - 1) / cus * cus; };
  // The tallest tile that fills the compute units, measured on each side, with
  // three parts where nothing else is said:
  // 512 x 64 in two workgroups of four waves per unit (4096 x 8192 -> 28672:
  // 1175 us; 256 x 64 in eight waves 1400), or in one of eight where there is
  // one tile each (1024 x 19456 -> 8192: 231 against 243); 256 x 64 (512 x
  // 20480 -> 8192: 135; 512 x 64 in eight waves 174, 256 x 32 152); 256 x 32 in
  // eight waves for one tile each (64 x 8192 -> 28672: 36; four waves 39).
  // Where 128 x 32 tiles leave units empty, the positions are split into
  // slices (64 x 10240 -> 4096: 4 slices 20, one 31), down to 512 positions
  // each, or 8192 to put two workgroups on a unit (24 x 68096 -> 8192: 8
  // slices 46, 4 slices 51).  Of four parts a 64-token stage leaves no room for
  // two workgroups of 512 rows: 512 x 64 in one of eight waves (4096 x 8192 ->
  // 28672: 1615; 256 x 64 in two of four 1637), or the latter where the last
  // round of the former would be filled below 9/10 (4096 x 4096 -> 2816: 118
  // against 135; 1024 x 8192 -> 28672: 430 against 448).  Of runs the last
  // round is not known here, and the latter's second workgroup covers the ends
  // of a tile: up to 8192 positions the latter (16384 rows of 64 experts, 4096
  // -> 2 x 1408: 397 against 431; 8192 of 8, 4096 -> 2 x 14336: 1751 against
  // 1738), past that the former (3000 of 8, 28672 -> 4096: 766 against 829).
  p.slices = 1;
  if (NP == 3 && two && count(4, 2) > cus) p.shape = 4120;
  else if (NP == 4 && two && count(4, 2) > cus &&
           (grouped ? units <= 32 : count(4, 2) * 10 < up(count(4, 2)) * 9)) p.shape = 2220;
  else if (NP <= 4 && two && count(4, 2) * 5 >= cus * 4) p.shape = 4221;
  else if (two && count(2, 2) * 5 >= cus * 4) p.shape = 2421;
  else if (count(4, 1) >= 2 * cus) p.shape = 4110;
  else if (count(2, 1) > cus) p.shape = 2210;
  else if (count(2, 1) * 4 >= cus * 3) p.shape = 2411;
  else {
    p.shape = 1410;
    const int64_t tiles = count(1, 1);
    const int64_t one = cus / tiles, both = 2 * cus / tiles;
    p.slices = static_cast<int>(units / (both < 1 ? 1 : both) >= 32 ? both : one);
    if (p.slices > units / 2) p.slices = static_cast<int>(units / 2);
    if (p.slices > 16) p.slices = 16;
    if (p.slices < 1) p.slices = 1;
  }
  p.slice_units = static_cast<int>((units + p.slices - 1) / p.slices);
  p.slices = static_cast<int>((units + p.slice_units - 1) / p.slice_units);
  p.ldz = (m + 3) / 4 * 4;
  p.sums_bytes = p.slices > 1 ? static_cast<size_t>(p.slices) * R * p.ldz * 4 : 0;
  return p;
}

hipError_t launch_gemm_f6(const F6Product& p, int shape, int NP, hipStream_t st) {
  return NP == 3 ? by_shape<3>(p, shape, st) : NP == 4 ? by_shape<4>(p, shape, st) : by_shape<5>(p, shape, st);
}

}  // namespace lq
