// The rows of a mixture-of-experts layer on their way to the experts and back
// (positions, tokens and weights as lq_route gives them):
//   lq_sort_rows       out[r] = x[rows[r]], zeros for an index outside [0, T)
//   lq_join_rows       out[t] = residual[t] + sum_j weight[t][j] z[pos[t][j]]
//   lq_join_rows_grad  dz[pos[t][j]] = weight[t][j] dy[t],
//                      dweight[t][j] = sum_i dy[t][i] z[pos[t][j]][i]
// All are bound by memory: each value is read once and written once.  Sums are
// float32, in a fixed order.
#include "f6_epilogue.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

// 16 bytes at any address (global memory takes them), aligned or not.
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

// ------------------------------------------------------------------ sort
// A wave per row, 16 bytes per lane, kAhead of them on their way, the rest of a
// row byte by byte.  Stores past the caches, which leaves those to the tokens' rows, each
// read k times: 32768 rows of 4 KB 37.0 us, plain stores 38.9; 65536 75 and 79, and with lq_quant8
// reading them next 146 and 166; 8192 rows 9.7 and 10.1 (22.2 and 21.3), fewer no difference.
constexpr int kAhead = 4;

__global__ void __launch_bounds__(256) sort_rows_kernel(const uint8_t* __restrict__ x, int T,
                                                        int64_t row_bytes, int64_t x_pitch,
                                                        const int* __restrict__ rows, int R,
                                                        uint8_t* __restrict__ out, int64_t out_pitch) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = static_cast<int64_t>(gridDim.x) * 4;
  const int64_t pieces = row_bytes / 16, tail = pieces * 16 + lane;
  for (int64_t r = blockIdx.x * int64_t{4} + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); r < R; r += waves) {
    const int t = rows[r];
    const bool live = t >= 0 && t < T;
    const uint8_t* from = x + (live ? t : 0) * x_pitch;
    uint8_t* to = out + r * out_pitch;
    for (int64_t p0 = lane; p0 < pieces; p0 += 64 * kAhead) {
      i32x4 v[kAhead] = {};
      if (live) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          v[i] = *reinterpret_cast<const i32x4_any*>(from + min(p0 + 64 * i, pieces - 1) * 16);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (p0 + 64 * i < pieces)
          __builtin_nontemporal_store(v[i], reinterpret_cast<i32x4_any*>(to + (p0 + 64 * i) * 16));
    }
    if (tail < row_bytes) to[tail] = live ? from[tail] : 0;
  }
}

// ------------------------------------------------------------------ values
// W = 8 consecutive columns of a row, or one (the last n % 8 columns go one by one),
// as they lie in memory: their conversion waits for their arrival.
template <int DT, int W>
struct Columns {
  static constexpr int WORDS = W == 1 ? 1 : DT == LQ_F32 ? 8 : 4;
  int w[WORDS];
};
template <int DT, int W>
__device__ __forceinline__ void load(const void* row, int64_t at, Columns<DT, W>& v) {
  constexpr int SIZE = DT == LQ_F32 ? 4 : 2;
  const uint8_t* p = static_cast<const uint8_t*>(row) + at * SIZE;
  if constexpr (W == 1) {
    v.w[0] = SIZE == 4 ? *reinterpret_cast<const int*>(p) : *reinterpret_cast<const uint16_t*>(p);
  } else {
#pragma unroll
    for (int x = 0; x < v.WORDS / 4; ++x) {
      const i32x4 y = *reinterpret_cast<const i32x4_any*>(p + 16 * x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[4 * x + i] = y[i];
    }
  }
}
template <int DT, int W>
__device__ __forceinline__ float value(const Columns<DT, W>& v, int i) {
  return DT == LQ_F32 ? __int_as_float(v.w[i]) : value16(static_cast<uint32_t>(v.w[i / 2]) >> (16 * (i % 2)), DT);
}
template <int DT, int W>
__device__ __forceinline__ void load(const void* row, int64_t at, float (&v)[W]) {
  Columns<DT, W> c;
  load(row, at, c);
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = value(c, i);
}

template <int W>
__device__ __forceinline__ void load_any(const void* row, int64_t at, int dt, float (&v)[W]) {
  if (dt == LQ_F32) load<LQ_F32>(row, at, v);
  else if (dt == LQ_F16) load<LQ_F16>(row, at, v);
  else load<LQ_BF16>(row, at, v);
}

template <int W>
__device__ __forceinline__ void store(const float (&v)[W], int dt, void* row, int64_t at) {
  if constexpr (W == 1) {
    if (dt == LQ_F32) static_cast<float*>(row)[at] = v[0];
    else static_cast<uint16_t*>(row)[at] = static_cast<uint16_t>(round16x2(v[0], 0.f, dt));
  } else if (dt == LQ_F32) {
    float* p = static_cast<float*>(row) + at;
    *reinterpret_cast<i32x4_any*>(p) = i32x4{__float_as_int(v[0]), __float_as_int(v[1]),
                                             __float_as_int(v[2]), __float_as_int(v[3])};
    *reinterpret_cast<i32x4_any*>(p + 4) = i32x4{__float_as_int(v[4]), __float_as_int(v[5]),
                                                 __float_as_int(v[6]), __float_as_int(v[7])};
  } else {
    i32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = static_cast<int>(round16x2(v[2 * i], v[2 * i + 1], dt));
    *reinterpret_cast<i32x4_any*>(static_cast<uint16_t*>(row) + at) = w;
  }
}

// ------------------------------------------------------------------ join
// A wave takes 512 columns of a token, eight per lane, so that the positions and
// weights are the wave's own; AHEAD rows' loads are on their way at once.
struct Join {
  const void* z;
  int64_t ldz;
  int R, n;
  const int* pos;
  const float* weight;         // or null
  int T, k;
  const void* residual;        // or null
  int64_t ldr;
  void* out;
  int64_t ldo;
  int out_dt;
};

template <int DT, int AHEAD, int W>
__device__ __forceinline__ void join_columns(const Join& a, int64_t t, int o) {
  float y[W] = {}, sum[W] = {};
  if (a.residual) load_any(a.residual, t * a.ldr + o, a.out_dt, y);
  for (int j0 = 0; j0 < a.k; j0 += AHEAD) {
    Columns<DT, W> v[AHEAD] = {};
    float w[AHEAD];
#pragma unroll
    for (int c = 0; c < AHEAD; ++c) {
      const int64_t at = t * a.k + min(j0 + c, a.k - 1);
      const int p = a.pos[at];
      const bool live = j0 + c < a.k && p >= 0 && p < a.R;
      w[c] = live ? (a.weight ? a.weight[at] : 1.f) : 0.f;
      if (live) load(a.z, p * a.ldz + o, v[c]);
    }
#pragma unroll
    for (int c = 0; c < AHEAD; ++c)
#pragma unroll
      for (int i = 0; i < W; ++i) sum[i] += w[c] * value(v[c], i);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) y[i] += sum[i];
  store(y, a.out_dt, a.out, t * a.ldo + o);
}

template <int DT, int AHEAD>
__global__ void __launch_bounds__(256) join_rows_kernel(Join a) {
  const int lane = threadIdx.x & 63, parts = (a.n + 511) / 512;
  const int64_t units = static_cast<int64_t>(a.T) * parts, waves = static_cast<int64_t>(gridDim.x) * 4;
  for (int64_t u = blockIdx.x * int64_t{4} + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units; u += waves) {
    const int64_t t = u / parts;
    const int o0 = static_cast<int>(u - t * parts) * 512, whole = a.n / 8 * 8;
    if (o0 + lane * 8 < whole) join_columns<DT, AHEAD, 8>(a, t, o0 + lane * 8);
    if (o0 + 512 > whole && whole + lane < a.n) join_columns<DT, AHEAD, 1>(a, t, whole + lane);
  }
}

// ------------------------------------------------------------------ gradient of the join
// A workgroup per token: dy[t] is read once per C choices; the dot products
// go through the waves and LDS.  The workgroups behind the tokens' clear
// the rows of dz that no token has (rows[r] outside [0, T)).
struct JoinGrad {
  const void* dy;
  int64_t ldy;
  const void* z;
  int64_t ldz;
  int R, n;
  const int* pos;
  const float* weight;
  int T, k;
  const int* rows;             // or null
  void* dz;
  int64_t lddz;
  float* dweight;
  int token_groups;
};

template <int DT, int C, int W>
__device__ __forceinline__ void grad_columns(const JoinGrad& a, int64_t t, int o, const int (&p)[C],
                                             const float (&w)[C], float (&dot)[C]) {
  Columns<DT, W> raw, v[C] = {};
  load(a.dy, t * a.ldy + o, raw);
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (p[c] >= 0) load(a.z, p[c] * a.ldz + o, v[c]);
  float g[W];
#pragma unroll
  for (int i = 0; i < W; ++i) g[i] = value(raw, i);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (p[c] < 0) continue;
    float d[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      dot[c] += g[i] * value(v[c], i);
      d[i] = w[c] * g[i];
    }
    store(d, DT, a.dz, p[c] * a.lddz + o);
  }
}

template <int DT, int C>
__global__ void __launch_bounds__(256) join_grad_kernel(JoinGrad a) {
  __shared__ float part[4][C];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, whole = a.n / 8 * 8;
  if (static_cast<int>(blockIdx.x) >= a.token_groups) {
    const int groups = gridDim.x - a.token_groups;
    const float zero[8] = {}, nought[1] = {};
    for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) - a.token_groups) * 256 + wave * 64; r0 < a.R;
         r0 += static_cast<int64_t>(groups) * 256) {
      const int t = r0 + lane < a.R ? a.rows[r0 + lane] : 0;
      uint64_t none = __ballot(r0 + lane < a.R && (t < 0 || t >= a.T));
      while (none) {
        const int64_t r = r0 + __builtin_ctzll(none);
        none &= none - 1;
        for (int o = lane * 8; o < whole; o += 512) store(zero, DT, a.dz, r * a.lddz + o);
        if (whole + lane < a.n) store(nought, DT, a.dz, r * a.lddz + whole + lane);
      }
    }
    return;
  }
  for (int64_t t = blockIdx.x; t < a.T; t += a.token_groups) {
    for (int j0 = 0; j0 < a.k; j0 += C) {
      int p[C];
      float w[C], dot[C] = {};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t at = t * a.k + min(j0 + c, a.k - 1);
        p[c] = a.pos[at];
        w[c] = a.weight[at];
        if (j0 + c >= a.k || p[c] >= a.R) p[c] = -1;
      }
      for (int o = tid * 8; o < whole; o += 2048) grad_columns<DT, C, 8>(a, t, o, p, w, dot);
      if (whole + tid < a.n) grad_columns<DT, C, 1>(a, t, whole + tid, p, w, dot);
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int s = 1; s < 64; s *= 2) dot[c] += __shfl_xor(dot[c], s);
      }
      if (j0 || t != blockIdx.x) __syncthreads();          // the last sums have been read
      if (lane == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) part[wave][c] = dot[c];
      }
      __syncthreads();
      if (tid < C && j0 + tid < a.k)
        a.dweight[t * a.k + j0 + tid] = part[0][tid] + part[1][tid] + (part[2][tid] + part[3][tid]);
    }
  }
}

template <int DT>
auto* grad_kernel(int k) {
  return k <= 2 ? join_grad_kernel<DT, 2> : k <= 4 ? join_grad_kernel<DT, 4> : join_grad_kernel<DT, 8>;
}

template <int DT>
auto* join_kernel(int k) {
  return k <= 2 ? join_rows_kernel<DT, 2> : k <= 4 ? join_rows_kernel<DT, 4> : join_rows_kernel<DT, 8>;
}

}  // namespace

hipError_t launch_sort_rows(const void* x, int size, int64_t T, int64_t n, int64_t ldx,
                            const int* rows, int64_t R, void* out, int64_t ldo, hipStream_t st) {
  const int64_t groups = (R + 3) / 4, most = int64_t{1} << 20;
  sort_rows_kernel<<<static_cast<uint32_t>(groups < most ? groups : most), 256, 0, st>>>(
      static_cast<const uint8_t*>(x), static_cast<int>(T), n * size, ldx * size, rows,
      static_cast<int>(R), static_cast<uint8_t*>(out), ldo * size);
  return hipGetLastError();
}

hipError_t launch_join_rows(const void* z, lq_dtype dt, int64_t R, int64_t n, int64_t ldz,
                            const int* pos, const float* weight, int64_t T, int k,
                            const void* residual, int64_t ldr, void* out, lq_dtype out_dt,
                            int64_t ldo, hipStream_t st) {
  const int64_t groups = (T * ((n + 511) / 512) + 3) / 4, most = int64_t{1} << 20;
  auto* kernel = dt == LQ_F32 ? join_kernel<LQ_F32>(k) : dt == LQ_F16 ? join_kernel<LQ_F16>(k) : join_kernel<LQ_BF16>(k);
  kernel<<<static_cast<uint32_t>(groups < most ? groups : most), 256, 0, st>>>(
      Join{z, ldz, static_cast<int>(R), static_cast<int>(n), pos, weight, static_cast<int>(T), k, residual,
           ldr, out, ldo, out_dt});
  return hipGetLastError();
}

hipError_t launch_join_rows_grad(const void* dy, lq_dtype dt, int64_t ldy, const void* z, int64_t ldz,
                                 int64_t R, int64_t n, const int* pos, const float* weight, int64_t T,
                                 int k, const int* rows, void* dz, int64_t lddz, float* dweight,
                                 hipStream_t st) {
  const int64_t most = int64_t{1} << 20;
  const int tokens = static_cast<int>(T < most ? T : most);
  int64_t clears = rows ? (R + 255) / 256 : 0;
  if (clears > 4096) clears = 4096;
  if (tokens + clears == 0) return hipSuccess;
  auto* kernel = dt == LQ_F32 ? grad_kernel<LQ_F32>(k) : dt == LQ_F16 ? grad_kernel<LQ_F16>(k) : grad_kernel<LQ_BF16>(k);
  kernel<<<static_cast<uint32_t>(tokens + clears), 256, 0, st>>>(
      JoinGrad{dy, ldy, z, ldz, static_cast<int>(R), static_cast<int>(n), pos, weight, static_cast<int>(T), k,
               rows, dz, lddz, dweight, tokens});
  return hipGetLastError();
}

}  // namespace lq
