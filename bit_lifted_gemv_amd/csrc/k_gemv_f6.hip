// Product of 1-bit weights with 16-bit lifted activations for at most 16 rows
// per matrix (one token to sixteen, or the few rows of an expert), on the
// 16 x 16 x 128 matrix instruction in float4 (signs) x float6 (activation
// parts, f6_parts.h), with the epilogue of lq_gemm_ep.
//
// A workgroup of 8 waves takes up to 16 tokens, a slice of the positions and a
// run of row blocks.  It first splits its slice of the tokens into float6
// parts, into LDS (its own, so no launch for them; the signs' first loads are
// behind the activations' meanwhile), then streams the signs from HBM
// straight into registers, 16 bytes per lane and 16-row tile of 512
// positions, DEPTH of them ahead.  A wave works on a unit of T tiles (each
// operand read from LDS serves T products), alone (KV = 1) or with KV - 1
// others on interleaved groups of the slice where there are too few rows to
// fill the chip; those add their sums through LDS in wave order.  Gated: the
// first half of a unit's tiles are gate rows, the second half the same
// outputs' up rows.
//
// One slice: the epilogue follows at once, a lane holding four consecutive
// outputs of a token.  More: each slice's float32 sums, scaled (and the first
// with the bias), go to the workspace and a second kernel adds them in order
// and finishes (k_f6_reduce.hip; the join adds them itself).  A workgroup of many rows and few
// positions converts little for the signs it streams, one of few rows and
// many positions needs no second launch: few_f6_plan weighs the two.  Bound
// by reading the signs once, and by latency for the smallest calls.
//
// Measured (MI355X, medians of a kernel trace): 1 x 10240 -> 4096 in 6.2 us (by
// clocks read in the kernel: activations there after 1 us, split after 2.3,
// signs done after 4.1, stored after 5.1); 5 x 68096 -> 8192 to float16 25.1 here
// and 4.8 in the reduction (of three parts 22.8; the 70 MB of signs come from
// the 256 MB cache where calls on a few matrices repeat, faster than a copy of
// 5.1 TB/s); 16 x 8192 -> 2 x 14336 gated 13.8 and 4.7; one token to 8 experts
// of 2816 x 4096: 9.5.
#include "f6_epilogue.h"
#include "f6_parts.h"
#include "f6_product.h"
#include "lq_internal.h"

#include <cstring>

namespace lq {
namespace {

using namespace f6;

constexpr uint32_t kRsrcWord3 = 0x00020000u;
constexpr uint32_t kFar = 0x40000000u;     // past every weight range (<= 2^30 bytes), also twice
constexpr int kWaves = 8;

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
        const int scale = static_cast<int>(ex - 0x01010101u * part_shift(p));
        if (u == 0) acc[t] = mfma<0>(s, b[p], acc[t], scale);
        if (u == 1) acc[t] = mfma<1>(s, b[p], acc[t], scale);
        if (u == 2) acc[t] = mfma<2>(s, b[p], acc[t], scale);
        if (u == 3) acc[t] = mfma<3>(s, b[p], acc[t], scale);
      }
    }
  }
}

// One block of 32 positions of a token: 64 bytes of 16-bit values, zeros past
// K and for an index out of range.
struct Block {
  uint4 v[4];
};
__device__ __forceinline__ Block load_block(const F6Few& f, int row, int k0) {
  Block b;
  const F6Product& a = f.p;
  bool live = true;
  if (a.rows) {
    row = a.rows[row];
    live = row >= 0 && row < a.src_rows;
  }
  const auto* src = static_cast<const uint16_t*>(f.a) + static_cast<int64_t>(live ? row : 0) * f.lda;
#pragma unroll
  for (int j = 0; j < 4; ++j) b.v[j] = make_uint4(0, 0, 0, 0);
  if (live && k0 + 32 <= f.K) {
#pragma unroll
    for (int j = 0; j < 4; ++j) b.v[j] = *reinterpret_cast<const uint4*>(src + k0 + 8 * j);
  } else if (live) {                            // the last block of a row
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (k0 + 8 * j < f.K) b.v[j] = *reinterpret_cast<const uint4*>(src + k0 + 8 * j);
  }
  return b;
}

template <int NP, bool bf16>
__device__ __forceinline__ void store_block(const Block& b, int place, uint8_t* g) {
  float x[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack8(b.v[j], bf16, x + 8 * j);
  const uint32_t e = block_exponent(largest_bits(b.v, bf16));
  u32x6 part[NP];
  split_block<NP>(x, e, part);
  const int gl = place / 4, u = place % 4;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = (u * NP + p) * 4 + gl;
    *reinterpret_cast<uint4*>(g + 16 * at) =
        make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
    *reinterpret_cast<uint2*>(g + tail_offset(4, NP) + 8 * at) = make_uint2(part[p][4], part[p][5]);
  }
  g[exp_offset(4, NP) + place] = static_cast<uint8_t>(e);
}

template <int NP, int T, int DEPTH, bool BF16>
__global__ void __launch_bounds__(64 * kWaves, 2) gemv_f6_kernel(F6Few f) {
  extern __shared__ __align__(256) uint8_t lds[];
  const F6Product& a = f.p;
  constexpr int GB = group_bytes(4, NP);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // ---- which tokens, slice and row blocks
  int tile = f.tile0 + blockIdx.z, expert = 0, row0 = tile * f.tok, row_end = a.R;
  if (a.offsets && !find_run(a, tile, f.tok, lane, expert, row0, row_end)) return;
  const int tokens = min(f.tok, row_end - row0);
  const int slice = blockIdx.y;
  const int g0 = slice * f.slice_groups, ng = min(f.slice_groups, a.groups - g0);

  // ---- the slice's parts into LDS, [group][token][GB]: all but each thread's
  // last block here, the next one on its way while one is split
  const int blocks = ng * 16, all = tokens * blocks;
  int i = tid, t_now = i / blocks, b_now = i - t_now * blocks;
  Block now{};
  if (i < all) now = load_block(f, row0 + t_now, (g0 * 16 + b_now) * 32);
  auto split_now = [&]() {
    if (i < all)
      store_block<NP, BF16>(now, b_now % 16, lds + (b_now / 16 * tokens + t_now) * GB);
  };
  for (int left = all; left > 64 * kWaves; left -= 64 * kWaves) {
    const int next = i + 64 * kWaves;
    int t = t_now, b = b_now + 64 * kWaves;
    while (b >= blocks) {
      b -= blocks;
      ++t;
    }
    Block ahead{};
    if (next < all) ahead = load_block(f, row0 + t, (g0 * 16 + b) * 32);
    split_now();
    now = ahead;
    i = next;
    t_now = t;
    b_now = b;
  }

  // ---- units, and their first signs
  const int KV = f.kv, part = wave % KV, sub = wave / KV, subs = kWaves / KV;
  const int i16 = lane & 15, gl = lane >> 4;
  const uint32_t* w = a.w + static_cast<int64_t>(expert) * a.m * a.ldw;
  const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(w), (short)0,
      static_cast<int>(static_cast<uint32_t>(a.m) * a.ldw * 4u), kRsrcWord3);
  const int half_m = a.m / 2, out_m = a.gated ? half_m : a.m;
  const int unit_outs = a.gated ? 8 * T : 16 * T;
  const int n = (ng - part + KV - 1) / KV;      // this wave's groups: part, part + KV, ...
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
  // scales of a block's outputs (gated: rows), loaded with its first signs
  const float* s = a.s + static_cast<int64_t>(expert) * a.m;
  const float* bias = a.bias && slice == 0 ? a.bias + static_cast<int64_t>(expert) * a.m : nullptr;
  RowScales scales[T];
  auto column = [&](int block, int t) {
    return (block * subs + sub) * unit_outs + (a.gated ? t % (T > 1 ? T / 2 : 1) : t) * 16 + 4 * gl;
  };
  auto load_scales = [&](int block) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int o = column(block, t);
      scales[t] = row_scales(s, bias, a.gated && t >= T / 2 ? half_m + o : o, a.m);
    }
  };
  const int b0 = blockIdx.x * f.blocks_per, b1 = min(b0 + f.blocks_per, f.row_blocks);
  aim(b0);
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(d, d);
  load_scales(b0);
  __builtin_amdgcn_sched_barrier(0);

  split_now();
  __syncthreads();

  const uint32_t two = held(0x22222222u);
  const uint8_t* mine = lds + min(i16, tokens - 1) * GB;
  f32x4* exchange = reinterpret_cast<f32x4*>(lds + f.exchange_at);
  const OutputTypes types = output_types(a.out, a.ldo, a.residual, a.ldr, a.out_dt);

  for (int rb = b0; rb < b1; ++rb) {
    f32x4 acc[T] = {};
    for (int j = 0; j < n; j += DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        if (j + d < n)
          group_products<NP, T>(mine + (part + (j + d) * KV) * tokens * GB, gl, ring[d], two, acc);
        load(d, j + d + DEPTH);
      }
    }
    RowScales its[T];
#pragma unroll
    for (int t = 0; t < T; ++t) its[t] = scales[t];
    if (rb + 1 < b1) {
      aim(rb + 1);
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) load(d, d);
      load_scales(rb + 1);
    }
    if (KV > 1) {
      if (rb > b0) __syncthreads();
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
    const bool whole = a.sums == nullptr;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const int o = column(rb, t), left = min(4, out_m - o);
      const int col = a.gated && t >= T / 2 ? half_m + o : o;
      float z[4];
      scaled(make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]), its[t], z);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[t][c] = z[c];
      if (!whole) {
        float* to = a.sums + (slice * static_cast<int64_t>(a.R) + row) * a.ldz + col;
        if (left == 4 && col % 4 == 0) *reinterpret_cast<f32x4*>(to) = acc[t];
        else
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < left) to[c] = z[c];
      }
    }
    if (!whole) continue;
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (a.gated && t >= T / 2) break;
      const int o = column(rb, t), left = min(4, out_m - o);
      if (left <= 0) continue;
      float y[4] = {acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
      activate4(y, a.act);
      if (a.gated) {
        const f32x4& up = acc[t + T / 2 < T ? t + T / 2 : t];
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] *= up[c];
      }
      finish4(y, left, types, a.residual, row * a.ldr + o, a.out, row * a.ldo + o);
    }
  }
}

template <int NP, int T, int DEPTH, bool BF16>
hipError_t launch(const F6Few& args, int tiles, hipStream_t st) {
  auto* k = gemv_f6_kernel<NP, T, DEPTH, BF16>;
  F6Few f = args;
  const int lds = f.exchange_at + (f.kv > 1 ? kWaves * T * 1024 : 0);
  if (lds > 64 * 1024) {                   // per call: the attribute belongs to the current device
    const hipError_t big = hipFuncSetAttribute(reinterpret_cast<const void*>(k),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (big != hipSuccess) return big;
  }
  // a grid's z ends at 65535: small matrices with more tiles take several launches
  for (f.tile0 = 0; f.tile0 < tiles; f.tile0 += 65535) {
    const dim3 grid((f.row_blocks + f.blocks_per - 1) / f.blocks_per, f.p.slices,
                    tiles - f.tile0 < 65535 ? tiles - f.tile0 : 65535);
    k<<<grid, 64 * kWaves, lds, st>>>(f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Every choice from the sizes: tokens per tile, the rows of a workgroup and
// its slice of the positions, by an estimate of the time.  Measured: a
// workgroup's conversions 2.5 us and 1.7 us per 512 blocks of 32 positions
// (0.7 of it the conversions alone); a compute unit's share of the HBM rate
// 21 KB per us (16 with T = 1, where reading the operands from LDS is the
// limit); a second launch 3 us (the join has one anyway) and its sums at
// about 4 TB/s.  Of one matrix the first 16 tokens are planned, tiles of more
// tokens run the same.
static F6FewPlan find_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                           bool grouped, bool join, int64_t cus) {
  F6FewPlan p{};
  const int64_t runs = grouped ? (E < R ? E : R) : 1;
  p.groups = static_cast<int>(padded_positions(K) / 512);
  // a tile holds twice the average run, so that few runs need a second one
  const int64_t average = (R + runs - 1) / runs;
  p.tok = !grouped ? static_cast<int>(R < 16 ? R : 16) : average <= 2 ? 4 : average <= 4 ? 8 : 16;
  p.tiles = static_cast<int>(grouped ? R / p.tok + runs : (R + p.tok - 1) / p.tok);
  const int gb = group_bytes(4, NP);
  const int fit = (163840 - kWaves * 1024 * 4) / (gb * p.tok);
  double best = 1e30;
  for (int T = gated ? 2 : 1; T <= 4; T *= 2)
    for (int kv = 1; kv <= 8; kv *= 2)
      for (int per = 1; per <= 4; per *= 2) {
        const int64_t unit_rows = 16 * T * (kWaves / kv);
        const int64_t row_blocks = (m + unit_rows - 1) / unit_rows;
        if (per > row_blocks) break;
        const int64_t wgs = (row_blocks + per - 1) / per * runs;
        // slices: as many as LDS needs, and the next counts that fill whole rounds of compute units
        int last = 0;
        for (int want = 0; want <= 4; ++want) {
          int64_t slices = want == 0 ? 1 : want * cus / wgs;
          const int64_t least = (p.groups + fit - 1) / fit;
          if (slices < least) slices = least;
          if (slices > p.groups) slices = p.groups;
          const int sg = static_cast<int>((p.groups + slices - 1) / slices);
          slices = (p.groups + sg - 1) / sg;
          if (slices == last || sg < kv) continue;
          last = static_cast<int>(slices);
          const int64_t rounds = (wgs * slices + cus - 1) / cus;
          const double convert = 2.5 + 1.7 * ((average < p.tok ? average : p.tok) * sg * 16) / 512.0;
          const double stream = per * (unit_rows * sg * 64 / (T == 1 ? 16e3 : 21e3) + 0.3);
          double us = rounds * (convert + stream);
          if (slices > 1)
            us += (join ? 0.0 : 3.0) + static_cast<double>(slices) * R * m * 8 / 4e6;
          if (us < best * 0.999) {
            best = us;
            p.T = T;
            p.kv = kv;
            p.blocks_per = per;
            p.row_blocks = static_cast<int>(row_blocks);
            p.slice_groups = sg;
            p.slices = static_cast<int>(slices);
          }
        }
      }
  p.exchange_at = (p.tok * p.slice_groups * gb + 255) / 256 * 256;
  p.ldz = (m + 3) / 4 * 4;
  p.sums_bytes = p.slices > 1 ? static_cast<size_t>(p.slices) * R * p.ldz * 4 : 0;
  return p;
}

// The search takes some microseconds: each thread keeps the plans of the
// shapes it met last (they follow from the sizes alone).
F6FewPlan few_f6_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                      bool grouped, bool join) {
  struct Entry {
    int64_t key[6] = {-1, -1, -1, -1, -1, -1};
    F6FewPlan plan;
  };
  constexpr int kKept = 64;
  thread_local Entry kept[kKept];
  const int64_t cus = num_cus();
  const int64_t key[6] = {E, m, K, R, cus, NP * 8 + gated * 4 + grouped * 2 + join};
  uint64_t hash = 0;
  for (int64_t k : key) hash = (hash + static_cast<uint64_t>(k)) * 0x9E3779B97F4A7C15ull;
  Entry& e = kept[hash >> 58];
  if (std::memcmp(e.key, key, sizeof key)) {
    e.plan = find_plan(E, m, K, R, gated, NP, grouped, join, cus);
    std::memcpy(e.key, key, sizeof key);
  }
  return e.plan;
}

hipError_t launch_gemv_f6(const F6Few& f, const F6FewPlan& plan, int NP, hipStream_t st) {
#define LQ_FEW(np, t, d) \
  if (NP == np && plan.T == t)                                       \
  return f.a_dt == LQ_BF16 ? launch<np, t, d, true>(f, plan.tiles, st) \
                           : launch<np, t, d, false>(f, plan.tiles, st)
  LQ_FEW(3, 1, 6);
  LQ_FEW(3, 2, 4);
  LQ_FEW(3, 4, 2);
  LQ_FEW(4, 1, 6);
  LQ_FEW(4, 2, 4);
  LQ_FEW(4, 4, 2);
  LQ_FEW(5, 1, 6);
  LQ_FEW(5, 2, 4);
  LQ_FEW(5, 4, 2);
#undef LQ_FEW
  return hipErrorInvalidValue;
}

}  // namespace lq
