// Product of 8-bit weights (e4m3, a scale per 128 x 128 block) with few rows of
// activations (lq_gemm8, lq_gemm8_grouped), on the matrix cores:
//   z[t][i] = sum_q sw[i / 128][q] 2^(ea[t][q] - 127) sum_{k in block q} w[i][k] a[t][k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 covers one block of 128 positions: operand A
// 16 tokens, scaled by the power of two of its lane's token; operand B 16 rows of
// weights, whose scale multiplies the block's sum (a lane's four sums are of one
// row).  The instruction adds eight products at a time and cuts them off 13 bits
// below the largest one's power of two: some 2^-17 of a typical result, which
// 16-bit results do not show.  For float32 results (PREC) the operands become
// bfloat16 (exact, and the token's power of two goes in) and
// v_mfma_f32_16x16x32_bf16 keeps 24 bits.
//
// Bound by reading the weights: nothing of them passes through LDS.  A wave
// takes WF x 16 rows and TF x 16 tokens, each lane loads two 16-byte pieces of
// its row's block (the two halves of 64 bytes, so that a load covers whole
// 64-byte runs of 16 rows; activations are read in the same order), and U blocks
// are on their way at once.  The waves of a workgroup share the rows and split
// the positions; their sums meet in LDS.  16-bit activations are quantized
// in registers on the way (lq_quant8's result bit for bit).
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

template <int AK, bool PREC, int TF, int WF>
__global__ void __launch_bounds__(512) gemv8_kernel(F8Product p) {
  constexpr bool WIDE = AK == LQ_F16 || AK == LQ_BF16;   // 16-bit activations
  constexpr int TOK = 16 * TF, ROWS = 16 * WF, PITCH = ROWS + 4;
  constexpr int U = TF * (WIDE ? 2 : 1) + WF <= 4 ? 4 : 2;
  constexpr int AP = WIDE ? 4 : 2;                       // 16-byte pieces of a lane's activations
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
              (expert * p.scales_matrix + row / 128 * p.lds) * (p.float_scales ? 4 : 1);
  }
  const uint8_t* arow[TF];
  const uint8_t* erow[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    int r = row0 + min(16 * f + c16, tokens - 1);
    if (p.rows) {
      r = p.rows[r];
      r = r < 0 || r >= p.a_rows ? 0 : r;                // its sums are dropped below
    }
    arow[f] = static_cast<const uint8_t*>(p.a) + static_cast<int64_t>(r) * p.lda * (WIDE ? 2 : 1) +
              (WIDE ? 32 : 16) * g;
    erow[f] = WIDE ? nullptr : p.exps + r * p.lde;
  }

  // ---- this wave's blocks of 128 positions
  const int s_end = min((slice + 1) * p.slice_steps, p.steps), s_begin = slice * p.slice_steps;
  const int per = (s_end - s_begin + waves - 1) / waves;
  const int begin = s_begin + wave * per, end = min(begin + per, s_end);

  uint4 wv[U][WF][2], av[U][TF][AP];
  uint32_t sv[U][WF], ev[U][TF];
  auto load = [&](int u, int step) {
    const int64_t at = min(step, end - 1);
#pragma unroll
    for (int f = 0; f < WF; ++f) {
      const uint4* from = reinterpret_cast<const uint4*>(wrow[f] + at * 128);
      wv[u][f][0] = from[0];
      wv[u][f][1] = from[4];
      sv[u][f] = p.float_scales ? reinterpret_cast<const uint32_t*>(srow[f])[at] : srow[f][at];
    }
#pragma unroll
    for (int f = 0; f < TF; ++f) {
      const uint4* from = reinterpret_cast<const uint4*>(arow[f] + at * (WIDE ? 256 : 128));
      if (WIDE) {
        // rows hold whole 16-byte pieces: those past the end are zeros
        const int k = static_cast<int>(at) * 128 + 16 * g;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        av[u][f][0] = k < p.K ? from[0] : zero;
        av[u][f][1] = k + 8 < p.K ? from[1] : zero;
        av[u][f][AP - 2] = k + 64 < p.K ? from[8] : zero;
        av[u][f][AP - 1] = k + 72 < p.K ? from[9] : zero;
        ev[u][f] = 0;
      } else {
        av[u][f][0] = from[0];
        av[u][f][1] = from[4];
        ev[u][f] = erow[f][at];
      }
    }
  };
  auto words = [](const uint4& lo, const uint4& hi) {
    i32x8 v;
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    return v;
  };

  f32x4 acc[TF][WF] = {};
  auto step = [&](int u) {
    i32x8 a[TF];
    int ea[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) {
      if (WIDE) {
        float v[32], largest = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = av[u][f][i % AP];
          const uint32_t w4[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = low16<AK>(w4[j]);
            v[8 * i + 2 * j + 1] = high16<AK>(w4[j]);
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) largest = fmaxf(largest, finite_magnitude(v[i]));
        largest = fmaxf(largest, __shfl_xor(largest, 16));
        largest = fmaxf(largest, __shfl_xor(largest, 32));
        ea[f] = block_exponent<LQ_E4M3>(largest);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          a[f][i] = static_cast<int>(round4<LQ_E4M3>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], ea[f]));
      } else {
        a[f] = words(av[u][f][0], av[u][f][1]);
        ea[f] = static_cast<int>(ev[u][f]);
      }
    }
    bf16x8 wide[PREC ? TF : 1][4];
    if (PREC) {
#pragma unroll
      for (int t = 0; t < TF; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          wide[t][i] = widen8<AK>(a[t][2 * i], a[t][2 * i + 1], power_of_two(ea[t]));
    }
#pragma unroll
    for (int f = 0; f < WF; ++f) {
      const i32x8 b = words(wv[u][f][0], wv[u][f][1]);
      const float scale = p.float_scales ? __uint_as_float(sv[u][f]) : power_of_two(sv[u][f]);
      bf16x8 wb[4];
      if (PREC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) wb[i] = widen8<LQ_E4M3>(b[2 * i], b[2 * i + 1], 1.f);
      }
#pragma unroll
      for (int t = 0; t < TF; ++t) {
        f32x4 z = {};
        if (PREC) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide[t][i], wb[i], z, 0, 0, 0);
        } else {
          constexpr int A = AK == LQ_E5M2 ? 1 : 0;
          z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[t], b, z, A, 0, 0, ea[t], 0, 127);
        }
        acc[t][f] += z * scale;
      }
    }
  };
  if (begin < end) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, begin + u);
    for (int s = begin; s < end; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (s + u < end) {
          step(u);
          load(u, s + u + U);
        }
      }
    }
  }

  // ---- the waves' sums, [wave][token][row], added in order
#pragma unroll
  for (int t = 0; t < TF; ++t)
#pragma unroll
    for (int f = 0; f < WF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lds[(wave * TOK + 16 * t + 4 * g + i) * PITCH + 16 * f + c16] = acc[t][f][i];
  __syncthreads();
  const int quads = outs / 4;
  const OutputTypes types = output_types(p.out, p.ldo, p.residual, p.ldr, p.out_dt);
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
    finish4(y, n, types, p.residual, row * p.ldr + out0 + o, p.out, row * p.ldo + out0 + o);
  }
}

template <int AK, bool PREC, int TF, int WF>
hipError_t launch(const F8Product& in, const F8FewPlan& plan, hipStream_t st) {
  F8Product p = in;
  const int64_t tok = 16 * TF, outs = p.gated ? 8 * WF : 16 * WF, out_m = p.gated ? p.m / 2 : p.m;
  p.row_blocks = static_cast<int>((out_m + outs - 1) / outs);
  int64_t tiles = (p.R + tok - 1) / tok;
  if (p.offsets) tiles = p.R / tok + (p.E < p.R ? p.E : p.R);
  const int64_t blocks = tiles * p.row_blocks * p.slices;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const int threads = 64 * plan.waves;
  const int bytes = static_cast<int>(plan.waves * tok * (16 * WF + 4) * 4);
  auto* k = gemv8_kernel<AK, PREC, TF, WF>;
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  // a launch has fewer than 2^32 threads
  const int64_t most = (int64_t{1} << 31) / threads;
  for (int64_t b = 0; b < blocks; b += most) {
    p.block0 = static_cast<int>(b);
    k<<<static_cast<uint32_t>(blocks - b < most ? blocks - b : most), threads, bytes, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int AK, bool PREC>
hipError_t by_shape(const F8Product& p, const F8FewPlan& plan, hipStream_t st) {
  if (plan.wf == 1) return launch<AK, PREC, 1, 1>(p, plan, st);
  switch (plan.tf) {
    case 1: return launch<AK, PREC, 1, 2>(p, plan, st);
    case 2: return launch<AK, PREC, 2, 2>(p, plan, st);
    default: return launch<AK, PREC, 4, 2>(p, plan, st);
  }
}

template <int AK>
hipError_t by_precision(const F8Product& p, const F8FewPlan& plan, bool precise, hipStream_t st) {
  return precise ? by_shape<AK, true>(p, plan, st) : by_shape<AK, false>(p, plan, st);
}

}  // namespace

F8FewPlan few_f8_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, bool grouped) {
  F8FewPlan p{};
  const int64_t cus = num_cus(), steps = (K + 127) / 128;
  const int64_t runs = grouped ? (E < R ? E : R) : 1, rows = (R + runs - 1) / runs;
  p.tf = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const int64_t out_m = gated ? m / 2 : m;
  auto blocks = [&](int wf) {
    const int64_t outs = gated ? 8 * wf : 16 * wf;
    return (out_m + outs - 1) / outs * runs;
  };
  p.wf = p.tf > 1 || gated || blocks(2) >= 2 * cus ? 2 : 1;
  p.waves = static_cast<int>(steps >= 32 ? 8 : steps >= 8 ? 4 : steps >= 2 ? 2 : 1);
  p.slices = 1;
  p.slice_steps = static_cast<int>(steps);
  const int64_t have = blocks(p.wf);
  if (have < cus) {
    int64_t s = (cus + have - 1) / have;
    const int64_t most = steps / (4 * p.waves) > 1 ? steps / (4 * p.waves) : 1;
    if (s > most) s = most;
    if (s > 16) s = 16;
    p.slice_steps = static_cast<int>((steps + s - 1) / s);
    p.slices = static_cast<int>((steps + p.slice_steps - 1) / p.slice_steps);
  }
  return p;
}

hipError_t launch_gemv8(const F8Product& p, int a_type, const F8FewPlan& plan, bool precise,
                        hipStream_t st) {
  switch (a_type) {
    case LQ_E4M3: return by_precision<LQ_E4M3>(p, plan, precise, st);
    case LQ_E5M2: return by_precision<LQ_E5M2>(p, plan, precise, st);
    case LQ_F16: return by_precision<LQ_F16>(p, plan, precise, st);
    default: return by_precision<LQ_BF16>(p, plan, precise, st);
  }
}

}  // namespace lq
