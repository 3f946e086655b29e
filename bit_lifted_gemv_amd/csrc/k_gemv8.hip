// Product of 8-bit weights (e4m3, a scale per 128 x 128 block) with few rows of
// activations (lq_gemm8, lq_gemm8_grouped), on the matrix cores:
//   z[t][i] = sum_q sw[i / 128][q] 2^(ea[t][q] - 127) sum_{k in block q} w[i][k] a[t][k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 covers one block of 128 positions: operand A
// 16 tokens, scaled by the power of two of its lane's token; operand B 16 rows of
// weights, scaled by theirs (a float32 scale multiplies the block's sum: a lane's four
// sums are of one row).  The instruction adds eight products at a time and cuts them off
// 13 places below the largest sum of two factors' exponents: 2^-16 of a typical result,
// 2^-14.5 with outlying positions, where the 16-bit results round by up to 2^-11 or 2^-8.
// For float32 results (PREC) the operands become bfloat16 (exact, and the powers of two
// go in) and v_mfma_f32_16x16x32_bf16 keeps 24 bits; for 16-bit results too that would cost
// 0 to 4 % (x 4096 -> 2 x 14336: one token 25.5 and 26.5 us, 16 tokens 28.1 and 28.8; 4096 x
// 4096 11.2 and 11.2) for an error that their rounding hides.
//
// Bound by reading the weights: nothing of them passes through LDS.  A wave
// takes WF x 16 rows and up to 16 tokens, each lane loads two 16-byte pieces of
// its row's block (the two halves of 64 bytes, so that a load covers whole
// 64-byte runs of 16 rows; activations are read in the same order), and U blocks
// are on their way at once.  The waves of a workgroup share the rows and split
// the positions; their sums meet in LDS.
//
// HELD: 16-bit activations of few tokens are quantized on the way to LDS (lq_quant8's
// result bit for bit), behind the first loads of weights, which saves the launch that
// does it (about 4.7 us): 4096 x 4096, one token, 9.3 us (8-bit ones straight from memory
// 7.5), four tokens 12.8 (8.2); 28672 positions of one token would cost 51 (42).
#include "f6_epilogue.h"
#include "f6_product.h"
#include "f8.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;
using namespace f8;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewTokens = 16;

__device__ __forceinline__ void wait_lds_and_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
}

// FS: float32 scales, where activations are held (one bfloat16 token x 4096 -> 8192 11.4 us, 12.4 where the
// kernel asks p.float_scales; four x 4096 -> 1024 10.6 and 11.4; one x 8192 -> 8192 22.2 and 21.6).  Others ask:
// the branch keeps a block's loads behind the products before them (one e4m3 token x 8192 -> 8192 19.9 us, 20.9
// without it; x 28672 47.5 and 49.2; x 4096 -> 28672 25.6 and 25.8).
template <int AK, bool FS, bool PREC, int WF>
__global__ void __launch_bounds__(512) gemv8_kernel(F8Product p) {
  constexpr bool HELD = AK == LQ_F16 || AK == LQ_BF16;   // 16-bit activations
  constexpr int AT = HELD ? LQ_E4M3 : AK;                // of the operand
  const bool float_scales = HELD ? FS : p.float_scales;
  constexpr int TOK = kFewTokens, ROWS = 16 * WF, PITCH = ROWS + 4;
  constexpr int U = WF == 1 ? (HELD ? 8 : 4) : WF == 2 || HELD ? 4 : 2;   // blocks of positions on their way
  extern __shared__ __align__(16) float lds[];
  const int tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;

  // ---- tile, block of rows, slice
  const int block = p.block0 + static_cast<int>(blockIdx.x);
  const int slice = block % p.slices, rest = block / p.slices;
  const int rb = rest % p.row_blocks, tile = rest / p.row_blocks;
  int expert = 0, row0 = tile * TOK, row_end = p.R;
  if (p.offsets && !find_run(p, tile, TOK, lane, expert, row0, row_end)) return;
  const int tokens = min(TOK, row_end - row0);
  const int half = p.m / 2, out_m = p.gated ? half : p.m;
  const int outs = p.gated ? ROWS / 2 : ROWS, out0 = rb * outs;

  // ---- sources
  const uint8_t* wrow[WF];
  const uint8_t* srow[WF];
#pragma unroll
  for (int f = 0; f < WF; ++f) {
    int row;
    if (p.gated) {
      constexpr int H = WF > 1 ? WF / 2 : 1;
      row = min(out0 + (f % H) * 16 + c16, half - 1) + (f / H) * half;
    } else {
      row = min(out0 + f * 16 + c16, p.m - 1);
    }
    wrow[f] = p.w + expert * p.w_matrix + row * p.ldw + 16 * g;
    srow[f] = static_cast<const uint8_t*>(p.scales) +
              (expert * p.scales_matrix + row / 128 * p.lds) * (float_scales ? 4 : 1);
  }
  auto source_row = [&](int token) {
    int r = row0 + min(token, tokens - 1);
    if (p.rows) {
      r = p.rows[r];
      r = r < 0 || r >= p.a_rows ? 0 : r;                // its sums are dropped below
    }
    return static_cast<int64_t>(r);
  };
  const uint8_t* arow = nullptr;
  const uint8_t* erow = nullptr;
  if constexpr (!HELD) {
    const int64_t r = source_row(c16);
    arow = static_cast<const uint8_t*>(p.a) + r * p.lda + 16 * g;
    erow = p.exps + r * p.lde;
  }

  // ---- this wave's blocks of 128 positions
  const int s_end = min((slice + 1) * p.slice_steps, p.steps), s_begin = slice * p.slice_steps;
  const int per = (s_end - s_begin + waves - 1) / waves;
  const int begin = s_begin + wave * per, end = min(begin + per, s_end);

  uint4 wv[U][WF][2], av[HELD ? 1 : U][2];
  uint32_t sv[U][WF], ev[HELD ? 1 : U];
  auto load = [&](int u, int step) {
    const int64_t at = min(step, end - 1);
#pragma unroll
    for (int f = 0; f < WF; ++f) {
      const uint4* from = reinterpret_cast<const uint4*>(wrow[f] + at * 128);
      wv[u][f][0] = from[0];
      wv[u][f][1] = from[4];
      sv[u][f] = float_scales ? reinterpret_cast<const uint32_t*>(srow[f])[at] : srow[f][at];
    }
    if constexpr (!HELD) {
      const uint4* from = reinterpret_cast<const uint4*>(arow + at * 128);
      av[u][0] = from[0];
      av[u][1] = from[4];
      ev[u] = erow[at];
    }
  };
  auto words = [](const uint4& lo, const uint4& hi) {
    i32x8 v;
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    return v;
  };
  if (begin < end) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, begin + u);
  }

  // ---- HELD: [token][positions of the slice], then their exponents in words
  const int blocks = s_end - s_begin, held_pitch = blocks * 128 + 32;
  uint8_t* held = reinterpret_cast<uint8_t*>(lds);
  uint32_t* held_exps = reinterpret_cast<uint32_t*>(held + tokens * held_pitch);
  if constexpr (HELD) {
    const int l16 = tid & 15;                            // 16 lanes a block, eight values each
    for (int x = tid >> 4; x < tokens * blocks; x += blockDim.x >> 4) {
      const int token = x / blocks, block = x - token * blocks;
      const int k = (s_begin + block) * 128 + l16 * 8;
      const uint16_t* from = static_cast<const uint16_t*>(p.a) + source_row(token) * p.lda + k;
      uint32_t w[4] = {0, 0, 0, 0};
      if (p.pieces) {                                    // rows are whole 16-byte pieces
        if (k < p.K) {
          const uint4 v = *reinterpret_cast<const uint4*>(from);
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < p.K) w[i / 2] |= static_cast<uint32_t>(from[i]) << (16 * (i % 2));
      }
      const int byte = block16<AK, 4, 1, 8>(w);
      const float scale = power_of_two(byte);
      *reinterpret_cast<int2*>(held + token * held_pitch + block * 128 + l16 * 8) =
          make_int2(round16<AK>(w[0], w[1], scale), round16<AK>(w[2], w[3], scale));
      if (l16 == 0) held_exps[token * blocks + block] = byte;
    }
    wait_lds_and_barrier();
  }
  const int my_token = min(c16, tokens - 1);
  const uint8_t* my_held = held + my_token * held_pitch + 16 * g;

  f32x4 acc[WF] = {};
  auto step = [&](int u, int s) {
    i32x8 a;
    int e;
    if constexpr (HELD) {
      const uint4* from = reinterpret_cast<const uint4*>(my_held + (s - s_begin) * 128);
      a = words(from[0], from[4]);
      e = static_cast<int>(held_exps[my_token * blocks + s - s_begin]);
    } else {
      a = words(av[u][0], av[u][1]);
      e = static_cast<int>(ev[u]);
    }
    bf16x8 wide[4];
    if constexpr (PREC) {
#pragma unroll
      for (int i = 0; i < 4; ++i) wide[i] = widen8<AT>(a[2 * i], a[2 * i + 1], power_of_two(e));
    }
#pragma unroll
    for (int f = 0; f < WF; ++f) {
      const i32x8 b = words(wv[u][f][0], wv[u][f][1]);
      // a power of two goes into the products (a block's sum without it may leave float32's range)
      const float scale = float_scales ? __uint_as_float(sv[u][f]) : 1.f;
      f32x4 z = {};
      if constexpr (PREC) {
        const float power = float_scales ? 1.f : power_of_two(sv[u][f]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              wide[i], widen8<LQ_E4M3>(b[2 * i], b[2 * i + 1], power), z, 0, 0, 0);
      } else {
        const int byte = float_scales ? 127 : static_cast<int>(sv[u][f]);
        z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, AT == LQ_E5M2 ? 1 : 0, 0, 0, e, 0, byte);
      }
      acc[f] += z * scale;
    }
  };
  for (int s = begin; s < end; s += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u < end) {
        step(u, s + u);
        load(u, s + u + U);
      }
    }
  }

  // ---- the waves' sums, [wave][token][row], added in order
  if constexpr (HELD) wait_lds_and_barrier();            // nobody reads the activations any more
#pragma unroll
  for (int f = 0; f < WF; ++f)
#pragma unroll
    for (int i = 0; i < 4; ++i) lds[(wave * TOK + 4 * g + i) * PITCH + 16 * f + c16] = acc[f][i];
  __syncthreads();
  const int quads = outs / 4;
  const float* bias = p.bias && slice == 0 ? p.bias + static_cast<int64_t>(expert) * p.m : nullptr;
  for (int x = tid; x < quads * tokens; x += blockDim.x) {
    const int token = x / quads, o = (x - token * quads) * 4, n = min(4, out_m - (out0 + o));
    if (n <= 0) continue;
    const int64_t row = row0 + token;
    bool live = true;
    if (p.rows) {
      const int r = p.rows[row];
      live = r >= 0 && r < p.a_rows;
    }
    auto sum = [&](int at, int column, float (&y)[4]) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < waves; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(lds + (w * TOK + token) * PITCH + at);
        v.x += z.x; v.y += z.y; v.z += z.z; v.w += z.w;
      }
      const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[i] = (live ? z[i] : 0.f) + (bias && i < n ? bias[column + i] : 0.f);
    };
    float y[4], up[4];
    sum(o, out0 + o, y);
    if (p.gated) sum(outs + o, half + out0 + o, up);
    if (p.sums) {
      float* to = p.sums + (slice * static_cast<int64_t>(p.R) + row) * p.ldz;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < n) {
          to[out0 + o + i] = y[i];
          if (p.gated) to[half + out0 + o + i] = up[i];
        }
      }
      continue;
    }
    activate(y, p.act);
    if (p.gated) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] *= up[i];
    }
    finish4(y, n, p.out_dt, p.residual, row * p.ldr + out0 + o, p.out, row * p.ldo + out0 + o);
  }
}

template <int AK, bool FS, bool PREC, int WF>
hipError_t launch(const F8Product& in, const F8FewPlan& plan, hipStream_t st) {
  F8Product p = in;
  const int64_t tok = kFewTokens, outs = p.gated ? 8 * WF : 16 * WF, out_m = p.gated ? p.m / 2 : p.m;
  p.row_blocks = static_cast<int>((out_m + outs - 1) / outs);
  int64_t tiles = (p.R + tok - 1) / tok;
  if (p.offsets) tiles = p.R / tok + (p.E < p.R ? p.E : p.R);
  const int64_t blocks = tiles * p.row_blocks * p.slices;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const int threads = 64 * plan.waves;
  // the sums, in the place of the held activations: at most 34 KB of eight waves, and 17 KB
  int64_t bytes = plan.waves * tok * (16 * WF + 4) * 4;
  if ((AK == LQ_F16 || AK == LQ_BF16) && plan.held_bytes > bytes) bytes = plan.held_bytes;
  auto* k = gemv8_kernel<AK, FS, PREC, WF>;
  // a launch has fewer than 2^32 threads
  const int64_t most = (int64_t{1} << 31) / threads;
  for (int64_t b = 0; b < blocks; b += most) {
    p.block0 = static_cast<int>(b);
    k<<<static_cast<uint32_t>(blocks - b < most ? blocks - b : most), threads, static_cast<uint32_t>(bytes), st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int AK, bool FS, bool PREC>
hipError_t by_shape(const F8Product& p, const F8FewPlan& plan, hipStream_t st) {
  return plan.wf == 1   ? launch<AK, FS, PREC, 1>(p, plan, st)
         : plan.wf == 2 ? launch<AK, FS, PREC, 2>(p, plan, st)
                        : launch<AK, FS, PREC, 4>(p, plan, st);
}

template <int AK>
hipError_t by_scales(const F8Product& p, const F8FewPlan& plan, bool precise, hipStream_t st) {
  if constexpr (AK == LQ_F16 || AK == LQ_BF16) {
    if (p.float_scales) return precise ? by_shape<AK, true, true>(p, plan, st) : by_shape<AK, true, false>(p, plan, st);
  }
  return precise ? by_shape<AK, false, true>(p, plan, st) : by_shape<AK, false, false>(p, plan, st);
}

}  // namespace

F8FewPlan few_f8_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, bool grouped) {
  F8FewPlan p{};
  const int64_t cus = num_cus(), steps = (K + 127) / 128;
  const int64_t runs = grouped ? (E < R ? E : R) : 1;
  const int64_t out_m = gated ? m / 2 : m;
  auto blocks = [&](int wf) {
    const int64_t outs = gated ? 8 * wf : 16 * wf;
    return (out_m + outs - 1) / outs * runs;
  };
  // The tallest block that leaves no compute unit without one (16 tokens x 4096 ->
  // 2 x 14336: 64 rows 28 us, 32 rows 36; one token x 4096 -> 4096: 16 rows 8.8 us,
  // 32 rows 10.1), and waves of 8 blocks of positions or more (the same: 4 waves 8.8 us,
  // 8 waves 9.7; 28672 -> 8192: 8 waves 46, 4 waves 55), 16 where there are
  // workgroups enough (16 tokens: 2 waves 28 us, 4 waves 32).
  p.wf = blocks(4) >= cus ? 4 : gated || blocks(2) >= cus ? 2 : 1;
  const int64_t have = blocks(p.wf), each = have * 2 >= cus * 3 ? 16 : 8;
  p.waves = static_cast<int>(steps >= 8 * each ? 8 : steps < each ? 1 : steps / each);
  p.slices = 1;
  p.slice_steps = static_cast<int>(steps);
  if (have < cus) {
    int64_t s = cus / have;
    if (s > steps / 64) s = steps / 64;
    if (s > 16) s = 16;
    if (s < 1) s = 1;
    p.slice_steps = static_cast<int>((steps + s - 1) / s);
    p.slices = static_cast<int>((steps + p.slice_steps - 1) / p.slice_steps);
  }
  // 16-bit activations; of runs the host knows only that none is longer than R
  p.held = R <= 4 && R * p.slice_steps <= 128;
  p.held_bytes = p.held ? R * (p.slice_steps * 132 + 32) : 0;
  return p;
}

hipError_t launch_gemv8(const F8Product& p, int a_type, const F8FewPlan& plan, bool precise,
                        hipStream_t st) {
  switch (a_type) {
    case LQ_E4M3: return by_scales<LQ_E4M3>(p, plan, precise, st);
    case LQ_E5M2: return by_scales<LQ_E5M2>(p, plan, precise, st);
    case LQ_F16: return by_scales<LQ_F16>(p, plan, precise, st);
    default: return by_scales<LQ_BF16>(p, plan, precise, st);
  }
}

}  // namespace lq
