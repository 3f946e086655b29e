// Product of 1-bit weights with 16-bit lifted activations for at most 16 rows
// per matrix (one token to sixteen, or the few rows of an expert), on the
// 16 x 16 x 128 matrix instruction in float4 (signs) x float6 (activation
// parts, f6_parts.h), with the epilogue of lq_gemm_ep.
//
// A workgroup of 8 waves takes up to 16 tokens, a slice of the positions and a
// run of row blocks.  It first splits its slice of the tokens into float6
// parts, into LDS (no launch of its own: spread over the workgroups it costs
// less than one), then streams the signs from HBM straight into registers, 16
// bytes per lane and 16-row tile of 512 positions, DEPTH of them ahead.  A
// wave works on a unit of T tiles (each operand read from LDS serves T
// products), alone (KV = 1) or with KV - 1 others on interleaved groups of
// the slice where there are too few rows to fill the chip; those add their
// sums through LDS in wave order.  Gated: the first half of a unit's tiles
// are gate rows, the second half the same outputs' up rows.
//
// One slice: the epilogue follows at once, a lane holding four consecutive
// outputs of a token.  More (activations longer than LDS, or few rows): each
// slice's float32 sums go to the workspace and a reduction adds them in order
// (k_gemv_f6's second kernel, or the join).  Bound by reading the signs once.
#include "f6_epilogue.h"
#include "f6_parts.h"
#include "f6_product.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kFar = 0x40000000u;     // past every weight range (<= 2^30 bytes), also twice
constexpr int kWaves = 8;
constexpr int kTok = 16;

template <int U>
__device__ __forceinline__ f32x4 mfma(const i32x8& a, const i32x8& b, const f32x4& c, int scale) {
  // A: E2M1 (cbsz 4), scale 2^0; B: E2M3 (blgp 2), scale 2^(byte U of scale - 127)
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 2, 0, 127, U, scale);
}

// The sums of a unit: the steps of one group for T tiles.
template <int NP, int T>
__device__ __forceinline__ void group_products(const uint8_t* g, int gl, const uint4 (&w)[T],
                                               uint32_t two, f32x4 (&acc)[T]) {
  const uint32_t ex = *reinterpret_cast<const uint32_t*>(g + exp_offset(4, NP) + 4 * gl);
  uint32_t words[T][4];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    words[t][0] = w[t].x;
    words[t][1] = w[t].y;
    words[t][2] = w[t].z;
    words[t][3] = w[t].w;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    i32x8 b[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int at = (u * NP + p) * 4 + gl;
      const int4 lo = *reinterpret_cast<const int4*>(g + 16 * at);
      const int2 hi = *reinterpret_cast<const int2*>(g + tail_offset(4, NP) + 8 * at);
      b[p][0] = lo.x; b[p][1] = lo.y; b[p][2] = lo.z; b[p][3] = lo.w;
      b[p][4] = hi.x; b[p][5] = hi.y; b[p][6] = 0; b[p][7] = 0;
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const i32x8 s = expand_signs(words[t][u], two);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int scale = static_cast<int>(ex - 0x04040404u * p);
        if (u == 0) acc[t] = mfma<0>(s, b[p], acc[t], scale);
        if (u == 1) acc[t] = mfma<1>(s, b[p], acc[t], scale);
        if (u == 2) acc[t] = mfma<2>(s, b[p], acc[t], scale);
        if (u == 3) acc[t] = mfma<3>(s, b[p], acc[t], scale);
      }
    }
  }
}

template <int NP, int T, int DEPTH>
__global__ void __launch_bounds__(64 * kWaves, 2) gemv_f6_kernel(F6Few f) {
  extern __shared__ __align__(256) uint8_t lds[];
  const F6Product& a = f.p;
  constexpr int GB = group_bytes(4, NP);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- which tokens, slice and row blocks
  int tile = blockIdx.z, expert = 0, row0 = tile * kTok, row_end = a.R;
  if (a.offsets) {
    int tiles = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64)
      tiles += __builtin_amdgcn_readfirstlane(wave_total(run_tiles(a, e0 + lane, kTok)));
    if (tile >= tiles) return;
    find_run(a, tile, kTok, lane, expert, row0, row_end);
  }
  const int tokens = min(kTok, row_end - row0);
  const int slice = blockIdx.y;
  const int g0 = slice * f.slice_groups, ng = min(f.slice_groups, a.groups - g0);

  // ---- the slice's parts into LDS: [group][token][GB]
  {
    const auto* src = static_cast<const uint16_t*>(f.a);
    const int blocks = ng * 16;
    for (int i = tid; i < tokens * blocks; i += 64 * kWaves) {
      const int t = i / blocks, b = i - t * blocks;
      int r = row0 + t;
      bool live = true;
      if (a.rows) {
        r = a.rows[r];
        live = r >= 0 && r < a.src_rows;
      }
      const int k0 = (g0 * 16 + b) * 32;
      float x[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && k0 + 8 * j < f.K)
          v = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(r) * f.lda + k0 + 8 * j);
        unpack8(v, f.a_dt == LQ_BF16, x + 8 * j);
      }
      const uint32_t e = block_exponent(largest_bits(x));
      u32x6 part[NP];
      split_block<NP>(x, e, part);
      const int gl = b / 4 % 4, u = b % 4;
      uint8_t* g = lds + (b / 16 * tokens + t) * GB;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int at = (u * NP + p) * 4 + gl;
        *reinterpret_cast<uint4*>(g + 16 * at) =
            make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
        *reinterpret_cast<uint2*>(g + tail_offset(4, NP) + 8 * at) =
            make_uint2(part[p][4], part[p][5]);
      }
      g[exp_offset(4, NP) + 4 * gl + u] = static_cast<uint8_t>(e);
    }
  }
  __syncthreads();

  // ---- units
  const int KV = f.kv, part = wave % KV, sub = wave / KV, subs = kWaves / KV;
  const int i16 = lane & 15, gl = lane >> 4;
  const uint32_t* w = a.w + static_cast<int64_t>(expert) * a.m * a.ldw;
  const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(w), (short)0,
      static_cast<int>(static_cast<uint32_t>(a.m) * a.ldw * 4u), kRsrcWord3);
  const float* s = a.s + static_cast<int64_t>(expert) * a.m;
  const float* bias = a.bias ? a.bias + static_cast<int64_t>(expert) * a.m : nullptr;
  const int half_m = a.m / 2, out_m = a.gated ? half_m : a.m;
  const int unit_outs = a.gated ? 8 * T : 16 * T;
  const uint32_t two = held(0x22222222u);
  const uint8_t* mine = lds + min(i16, tokens - 1) * GB;
  const int n = (ng - part + KV - 1) / KV;      // this wave's groups: part, part + KV, ...
  f32x4* exchange = reinterpret_cast<f32x4*>(lds + f.exchange_at);
  const OutputTypes types = output_types(a.out, a.ldo, a.residual, a.ldr, a.out_dt);

  uint32_t at[T];                               // byte offsets of the unit's rows
  uint4 ring[DEPTH][T];
  auto aim = [&](int block) {
    const int out0 = (block * subs + sub) * unit_outs;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      int row;
      if (a.gated) {
        const int o = out0 + (t % (T > 1 ? T / 2 : 1)) * 16 + i16;
        row = o < half_m ? o + (t >= T / 2 ? half_m : 0) : -1;
      } else {
        const int o = out0 + t * 16 + i16;
        row = o < a.m ? o : -1;
      }
      at[t] = row < 0 ? kFar : static_cast<uint32_t>(row) * a.ldw * 4u + (g0 * 16 + 4 * gl) * 4u;
    }
  };
  auto load = [&](int d, int j) {               // group j of this wave into slot d
    const int so = j < n ? (part + j * KV) * 64 : static_cast<int>(kFar);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const auto r = __builtin_amdgcn_raw_buffer_load_b128(wres, at[t], so, 0);
      __builtin_memcpy(&ring[d][t], &r, 16);
    }
  };

  const int b0 = blockIdx.x * f.blocks_per, b1 = min(b0 + f.blocks_per, f.row_blocks);
  aim(b0);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, d);
  for (int block = b0; block < b1; ++block) {
    f32x4 acc[T] = {};
    for (int j = 0; j < n; j += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (j + d < n)
          group_products<NP, T>(mine + (part + (j + d) * KV) * tokens * GB, gl, ring[d], two, acc);
        load(d, j + d + DEPTH);
      }
    }
    const int out0 = (block * subs + sub) * unit_outs;
    if (block + 1 < b1) {
      aim(block + 1);
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) load(d, d);
    }
    if (KV > 1) {
      if (block > b0) __syncthreads();
#pragma unroll
      for (int t = 0; t < T; ++t) exchange[(wave * T + t) * 64 + lane] = acc[t];
      __syncthreads();
      if (part != 0) continue;
#pragma unroll
      for (int t = 0; t < T; ++t)
        for (int q = 1; q < KV; ++q) acc[t] += exchange[((wave + q) * T + t) * 64 + lane];
    }
    if (i16 >= tokens) continue;
    const int64_t row = row0 + i16;
    if (f.slices > 1) {
      // sums of this slice: [slice][row][m]
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int o = out0 + (a.gated && T > 1 ? t % (T / 2) : t) * 16 + 4 * gl;
        const int zr = a.gated && t >= T / 2 ? half_m + o : o;
        float* z = f.sums + (slice * static_cast<int64_t>(a.R) + row) * f.ldz + zr;
        const int left = out_m - o;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < left) z[c] = acc[t][c];
      }
      continue;
    }
#pragma unroll
    for (int t = 0; t < (T > 1 ? T : 1); ++t) {
      if (a.gated && t >= T / 2) break;
      const int o = out0 + t * 16 + 4 * gl;
      const int left = min(4, out_m - o);
      if (left <= 0) continue;
      float y[4];
      scaled(make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]),
             row_scales(s, bias, o, left), y);
      activate4(y, a.act);
      if (a.gated) {
        float g[4];
        const f32x4& v = acc[T > 1 ? t + T / 2 < T ? t + T / 2 : t : 0];
        scaled(make_float4(v[0], v[1], v[2], v[3]), row_scales(s, bias, half_m + o, left), g);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] *= g[c];
      }
      finish4(y, left, types, a.residual, row * a.ldr + o, a.out, row * a.ldo + o);
    }
  }
}

// The slices' sums added in order, and the epilogue: a thread per row and
// four outputs.
__global__ void __launch_bounds__(256) gemv_f6_reduce_kernel(F6Few f) {
  const F6Product& a = f.p;
  const int half_m = a.m / 2, out_m = a.gated ? half_m : a.m;
  const int o = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int n = min(4, out_m - o);
  const int row = blockIdx.y;
  if (n <= 0) return;
  int expert = 0;
  if (a.offsets) {
    // the last run that begins at or before this row; outside every run the
    // row is left as it was
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.offsets[mid] <= row) lo = mid;
      else hi = mid;
    }
    if (a.offsets[lo] > row || a.offsets[lo + 1] <= row) return;
    expert = lo;
  }
  const float* s = a.s + static_cast<int64_t>(expert) * a.m;
  const float* bias = a.bias ? a.bias + static_cast<int64_t>(expert) * a.m : nullptr;
  auto sum = [&](int col) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const float* z = f.sums + static_cast<int64_t>(row) * f.ldz + col;
    const int64_t step = static_cast<int64_t>(a.R) * f.ldz;
    for (int q = 0; q < f.slices; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] += z[q * step + min(c, n - 1)];
    return make_float4(v[0], v[1], v[2], v[3]);
  };
  float y[4];
  scaled(sum(o), row_scales(s, bias, o, n), y);
  activate4(y, a.act);
  if (a.gated) {
    float g[4];
    scaled(sum(half_m + o), row_scales(s, bias, half_m + o, n), g);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] *= g[c];
  }
  const OutputTypes types = output_types(a.out, a.ldo, a.residual, a.ldr, a.out_dt);
  const int64_t r = row;
  finish4(y, n, types, a.residual, r * a.ldr + o, a.out, r * a.ldo + o);
}

template <int NP, int T, int DEPTH>
hipError_t launch(const F6Few& f, int tiles, hipStream_t st) {
  auto* k = gemv_f6_kernel<NP, T, DEPTH>;
  static const hipError_t big = hipFuncSetAttribute(
      reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, 163840);
  if (big != hipSuccess) return big;
  const dim3 grid((f.row_blocks + f.blocks_per - 1) / f.blocks_per, f.slices, tiles);
  const int lds = f.exchange_at + (f.kv > 1 ? kWaves * T * 1024 : 0);
  k<<<grid, 64 * kWaves, lds, st>>>(f);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && f.slices > 1) {
    const int out_m = f.p.gated ? f.p.m / 2 : f.p.m;
    gemv_f6_reduce_kernel<<<dim3((out_m + 1023) / 1024, f.p.R), 256, 0, st>>>(f);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// Slices, units and workgroups: every choice from the sizes.
F6FewPlan few_f6_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                      bool grouped) {
  F6FewPlan p{};
  const int64_t runs = grouped ? (E < R ? E : R) : 1;
  p.groups = static_cast<int>(padded_positions(K) / 512);
  p.tiles = static_cast<int>(grouped ? R / kTok + runs : (R + kTok - 1) / kTok);
  const int tokens = static_cast<int>(R < kTok ? R : kTok);
  // LDS holds a slice of up to `tokens` tokens; 8 KB per tile of a unit stay for the exchange
  const int fit = (163840 - 4 * kWaves * 1024) / (group_bytes(4, NP) * tokens);
  p.slices = (p.groups + fit - 1) / fit;
  const int64_t tiles16 = (m + 15) / 16;
  const int64_t waves = static_cast<int64_t>(num_cus()) * kWaves;
  auto units = [&](int T) { return (tiles16 + T - 1) / T * p.slices * runs; };
  p.T = 1;
  for (int T : {4, 2})
    if (p.T == 1 && units(T) * 2 >= waves) p.T = T;
  if (gated && p.T == 1) p.T = 2;
  p.kv = 1;
  while (p.kv < 8 && units(p.T) * p.kv * 2 <= waves && p.kv * p.slices * 2 <= p.groups) p.kv *= 2;
  p.slice_groups = (p.groups + p.slices - 1) / p.slices;
  p.slices = (p.groups + p.slice_groups - 1) / p.slice_groups;
  const int64_t unit_rows = 16 * p.T * (kWaves / p.kv);
  p.row_blocks = static_cast<int>((m + unit_rows - 1) / unit_rows);
  // enough workgroups for every compute unit, and no more conversions than that
  const int64_t all = static_cast<int64_t>(p.row_blocks) * p.slices * runs;
  const int64_t per = all / (2 * num_cus());
  p.blocks_per = static_cast<int>(per < 1 ? 1 : per > p.row_blocks ? p.row_blocks : per);
  p.exchange_at = (tokens * p.slice_groups * group_bytes(4, NP) + 255) / 256 * 256;
  p.ldz = (m + 3) / 4 * 4;
  p.sums_bytes = p.slices > 1 ? static_cast<size_t>(p.slices) * R * p.ldz * 4 : 0;
  return p;
}

hipError_t launch_gemv_f6(const F6Few& f, const F6FewPlan& plan, int NP, hipStream_t st) {
#define LQ_FEW(np, t, d) \
  if (NP == np && plan.T == t) return launch<np, t, d>(f, plan.tiles, st)
  LQ_FEW(3, 1, 6);
  LQ_FEW(3, 2, 4);
  LQ_FEW(3, 4, 2);
  LQ_FEW(4, 1, 6);
  LQ_FEW(4, 2, 4);
  LQ_FEW(4, 4, 2);
#undef LQ_FEW
  return hipErrorInvalidValue;
}

}  // namespace lq
