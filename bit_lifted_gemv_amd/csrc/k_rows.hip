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

// ------------------------------------------------------------------ sort
// A wave per row, pieces of V bytes per lane, AHEAD of them on their way.
constexpr int kAhead = 4;

template <class V>
__global__ void __launch_bounds__(256) sort_rows_kernel(const uint8_t* __restrict__ x, int T,
                                                        int64_t row_bytes, int64_t x_pitch,
                                                        const int* __restrict__ rows, int R,
                                                        uint8_t* __restrict__ out, int64_t out_pitch) {
  const int lane = threadIdx.x & 63;
  const int waves = gridDim.x * 4;
  const int pieces = static_cast<int>(row_bytes / sizeof(V));
  for (int64_t r = blockIdx.x * 4 + (threadIdx.x >> 6); r < R; r += waves) {
    const int t = __builtin_amdgcn_readfirstlane(rows[r]);
    const bool live = t >= 0 && t < T;
    const V* from = reinterpret_cast<const V*>(x + (live ? t : 0) * x_pitch);
    V* to = reinterpret_cast<V*>(out + r * out_pitch);
    for (int p0 = lane; p0 < pieces; p0 += 64 * kAhead) {
      V v[kAhead] = {};
      if (live) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = from[min(p0 + 64 * i, pieces - 1)];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (p0 + 64 * i < pieces) to[p0 + 64 * i] = v[i];
    }
  }
}

// ------------------------------------------------------------------ values
// Eight columns of a row, the first n of them inside; zeros behind.
template <int DT>
__device__ __forceinline__ void load8(const void* row, int64_t at, int n, bool wide, float (&v)[8]) {
  if (wide && n >= 8) {
    if (DT == LQ_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + at);
      const float4 a = p[0], b = p[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + at);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = value16(u[i / 2] >> (16 * (i % 2)), DT);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < n ? load_as_float<DT>(row, at + i) : 0.f;
}

__device__ __forceinline__ void store8(const float (&v)[8], int dt, void* row, int64_t at, int n,
                                       bool wide) {
  if (wide && n >= 8) {
    if (dt == LQ_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + at) =
          make_uint4(round16x2(v[0], v[1], dt), round16x2(v[2], v[3], dt),
                     round16x2(v[4], v[5], dt), round16x2(v[6], v[7], dt));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= n) break;
    if (dt == LQ_F32) static_cast<float*>(row)[at + i] = v[i];
    else static_cast<uint16_t*>(row)[at + i] = static_cast<uint16_t>(round16x2(v[i], 0.f, dt));
  }
}

// ------------------------------------------------------------------ join
// A thread takes eight columns of a token; its rows' loads go ahead, kRowsAhead
// at a time.
constexpr int kRowsAhead = 8;

template <int DT>
__global__ void __launch_bounds__(256) join_rows_kernel(const void* __restrict__ z, int R, int n,
                                                        int64_t ldz, const int* __restrict__ pos,
                                                        const float* __restrict__ weight, int T, int k,
                                                        const void* residual, int64_t ldr, void* out,
                                                        int64_t ldo, int out_dt, int columns,
                                                        bool wide_z, bool wide_out) {
  // `columns` threads side by side on a token's columns
  const int lane = threadIdx.x % columns, sub = threadIdx.x / columns, per = 256 / columns;
  const int o = (blockIdx.x * columns + lane) * 8, live_n = min(8, n - o);
  if (o >= n) return;
  for (int64_t t = static_cast<int64_t>(blockIdx.y) * per + sub; t < T;
       t += static_cast<int64_t>(gridDim.y) * per) {
    float y[8] = {};
    if (residual) {
      if (out_dt == LQ_F32) load8<LQ_F32>(residual, t * ldr + o, live_n, wide_out, y);
      else if (out_dt == LQ_F16) load8<LQ_F16>(residual, t * ldr + o, live_n, wide_out, y);
      else load8<LQ_BF16>(residual, t * ldr + o, live_n, wide_out, y);
    }
    float sum[8] = {};
    for (int j0 = 0; j0 < k; j0 += kRowsAhead) {
      float v[kRowsAhead][8], w[kRowsAhead];
#pragma unroll
      for (int c = 0; c < kRowsAhead; ++c) {
        const int64_t at = t * k + min(j0 + c, k - 1);
        const int p = pos[at];
        const bool live = j0 + c < k && p >= 0 && p < R;
        w[c] = live ? (weight ? weight[at] : 1.f) : 0.f;
        if (live) {
          load8<DT>(z, p * ldz + o, live_n, wide_z, v[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
        }
      }
#pragma unroll
      for (int c = 0; c < kRowsAhead; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += w[c] * v[c][i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += sum[i];
    store8(y, out_dt, out, t * ldo + o, live_n, wide_out);
  }
}

// ------------------------------------------------------------------ gradient of the join
// A workgroup per token: dy[t] is read once per eight choices; the dot products
// go through the waves and LDS.  The workgroups behind the tokens' clear
// the rows of dz that no token has (rows[r] outside [0, T)).
template <int DT>
__global__ void __launch_bounds__(256) join_grad_kernel(const void* __restrict__ dy, int64_t ldy,
                                                        const void* __restrict__ z, int64_t ldz, int R,
                                                        int n, const int* __restrict__ pos,
                                                        const float* __restrict__ weight, int T, int k,
                                                        const int* __restrict__ rows, void* dz,
                                                        int64_t lddz, float* __restrict__ dweight,
                                                        int token_groups, bool wide) {
  constexpr int C = kRowsAhead;
  __shared__ float part[4][C];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (static_cast<int>(blockIdx.x) >= token_groups) {
    const int groups = gridDim.x - token_groups;
    const float zero[8] = {};
    for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) - token_groups) * 256 + wave * 64; r0 < R;
         r0 += static_cast<int64_t>(groups) * 256) {
      const int t = r0 + lane < R ? rows[r0 + lane] : 0;
      uint64_t none = __ballot(r0 + lane < R && (t < 0 || t >= T));
      while (none) {
        const int64_t r = r0 + __builtin_ctzll(none);
        none &= none - 1;
        for (int o = lane * 8; o < n; o += 512) store8(zero, DT, dz, r * lddz + o, min(8, n - o), wide);
      }
    }
    return;
  }
  for (int64_t t = blockIdx.x; t < T; t += token_groups) {
    for (int j0 = 0; j0 < k; j0 += C) {
      int p[C];
      float w[C], dot[C] = {};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t at = t * k + min(j0 + c, k - 1);
        p[c] = pos[at];
        w[c] = weight[at];
        if (j0 + c >= k || p[c] >= R) p[c] = -1;
      }
      for (int o = tid * 8; o < n; o += 2048) {
        const int live = min(8, n - o);
        float g[8], v[C][8];
        load8<DT>(dy, t * ldy + o, live, wide, g);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (p[c] >= 0) load8<DT>(z, p[c] * ldz + o, live, wide, v[c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (p[c] < 0) continue;
          float d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[c] += g[i] * v[c][i];
            d[i] = w[c] * g[i];
          }
          store8(d, DT, dz, p[c] * lddz + o, live, wide);
        }
      }
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
      if (tid < C && j0 + tid < k)
        dweight[t * k + j0 + tid] = part[0][tid] + part[1][tid] + (part[2][tid] + part[3][tid]);
    }
  }
}

bool on16(const void* p, int64_t pitch_bytes) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(pitch_bytes)) % 16 == 0;
}
int size_of(int dt) { return dt == LQ_F32 ? 4 : 2; }

template <class V>
void sort_rows(const void* x, int64_t T, int64_t bytes, int64_t x_pitch, const int* rows, int64_t R,
               void* out, int64_t out_pitch, hipStream_t st) {
  const int64_t groups = (R + 3) / 4, most = int64_t{1} << 20;
  sort_rows_kernel<V><<<static_cast<uint32_t>(groups < most ? groups : most), 256, 0, st>>>(
      static_cast<const uint8_t*>(x), static_cast<int>(T), bytes, x_pitch, rows, static_cast<int>(R),
      static_cast<uint8_t*>(out), out_pitch);
}

}  // namespace

hipError_t launch_sort_rows(const void* x, int size, int64_t T, int64_t n, int64_t ldx,
                            const int* rows, int64_t R, void* out, int64_t ldo, hipStream_t st) {
  const int64_t bytes = n * size, xp = ldx * size, op = ldo * size;
  // the widest piece that every row's start and length allow
  const uint64_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
                        static_cast<uint64_t>(bytes) | static_cast<uint64_t>(xp) |
                        static_cast<uint64_t>(op);
  if (bits % 16 == 0) sort_rows<uint4>(x, T, bytes, xp, rows, R, out, op, st);
  else if (bits % 4 == 0) sort_rows<uint32_t>(x, T, bytes, xp, rows, R, out, op, st);
  else if (bits % 2 == 0) sort_rows<uint16_t>(x, T, bytes, xp, rows, R, out, op, st);
  else sort_rows<uint8_t>(x, T, bytes, xp, rows, R, out, op, st);
  return hipGetLastError();
}

hipError_t launch_join_rows(const void* z, lq_dtype dt, int64_t R, int64_t n, int64_t ldz,
                            const int* pos, const float* weight, int64_t T, int k,
                            const void* residual, int64_t ldr, void* out, lq_dtype out_dt,
                            int64_t ldo, hipStream_t st) {
  const bool wide_z = on16(z, ldz * size_of(dt));
  const bool wide_out = on16(out, ldo * size_of(out_dt)) &&
                        (!residual || on16(residual, ldr * size_of(out_dt)));
  int columns = 32;
  while (columns < 256 && columns * 8 < n) columns *= 2;
  const int64_t gx = (n + columns * 8 - 1) / (columns * 8), per = 256 / columns;
  const int64_t gy = (T + per - 1) / per;
  const dim3 grid(static_cast<uint32_t>(gx), static_cast<uint32_t>(gy < 65535 ? gy : 65535));
  auto* kernel = dt == LQ_F32 ? join_rows_kernel<LQ_F32>
                 : dt == LQ_F16 ? join_rows_kernel<LQ_F16> : join_rows_kernel<LQ_BF16>;
  kernel<<<grid, 256, 0, st>>>(z, static_cast<int>(R), static_cast<int>(n), ldz, pos, weight,
                               static_cast<int>(T), k, residual, ldr, out, ldo, out_dt, columns,
                               wide_z, wide_out);
  return hipGetLastError();
}

hipError_t launch_join_rows_grad(const void* dy, lq_dtype dt, int64_t ldy, const void* z, int64_t ldz,
                                 int64_t R, int64_t n, const int* pos, const float* weight, int64_t T,
                                 int k, const int* rows, void* dz, int64_t lddz, float* dweight,
                                 hipStream_t st) {
  const int size = size_of(dt);
  const bool wide = on16(dy, ldy * size) && on16(z, ldz * size) && on16(dz, lddz * size);
  const int64_t most = int64_t{1} << 20;
  const int tokens = static_cast<int>(T < most ? T : most);
  int64_t clears = rows ? (R + 255) / 256 : 0;
  if (clears > 4096) clears = 4096;
  if (tokens + clears == 0) return hipSuccess;
  auto* kernel = dt == LQ_F32 ? join_grad_kernel<LQ_F32>
                 : dt == LQ_F16 ? join_grad_kernel<LQ_F16> : join_grad_kernel<LQ_BF16>;
  kernel<<<static_cast<uint32_t>(tokens + clears), 256, 0, st>>>(
      dy, ldy, z, ldz, static_cast<int>(R), static_cast<int>(n), pos, weight, static_cast<int>(T), k,
      rows, dz, lddz, dweight, tokens, wide);
  return hipGetLastError();
}

}  // namespace lq
