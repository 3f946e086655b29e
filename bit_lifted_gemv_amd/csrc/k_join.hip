// The way out of the experts: out[t] = residual[t] + sum_j weight[t][j]
// z[pos[t][j]], z float32 rows in the sorted order (lq_gemm_join), each the
// sum of the product's slices.  A choice with a position outside [0, R) adds
// nothing.  Sums in the order of j, slices within it.  One thread per token
// and four columns, up to eight loads on their way at once; bound by reading
// z once: 1500 tokens of 2 x 4096 in 16 us (3.8 TB/s), 24 of 8 x 2048 in 4.5.
#include "f6_epilogue.h"
#include "lq_internal.h"

namespace lq {
namespace {

constexpr int kAhead = 8;

__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ z, int slices, int R,
                                                   int m, const int* __restrict__ pos,
                                                   const float* __restrict__ weight, int T, int k,
                                                   const void* residual, int64_t ldr, void* out,
                                                   int64_t ldo, int ldz, int out_dt) {
  const int o = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (o >= m) return;
  const int64_t step = static_cast<int64_t>(R) * ldz;
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    const int64_t c0 = static_cast<int64_t>(t) * k;
    for (int i0 = 0; i0 < k * slices; i0 += kAhead) {
      float4 v[kAhead];
      float w[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int i = min(i0 + x, k * slices - 1);
        const int j = slices == 1 ? i : i / slices, q = slices == 1 ? 0 : i - j * slices;
        const int p = pos[c0 + j];
        const bool live = i0 + x < k * slices && p >= 0 && p < R;
        w[x] = live ? weight[c0 + j] : 0.f;
        v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live)
          v[x] = *reinterpret_cast<const float4*>(z + q * step + static_cast<int64_t>(p) * ldz + o);
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        y[0] += w[x] * v[x].x;
        y[1] += w[x] * v[x].y;
        y[2] += w[x] * v[x].z;
        y[3] += w[x] * v[x].w;
      }
    }
    f6::finish4(y, min(4, m - o), out_dt, residual, t * ldr + o, out, t * ldo + o);
  }
}

}  // namespace

hipError_t launch_join(const float* z, int slices, int64_t R, int64_t m, int64_t ldz,
                       const int* pos, const float* weight, int64_t T, int k, const void* residual, int64_t ldr,
                       void* out, int64_t ldo, int dt, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((m + 1023) / 1024),
                  static_cast<uint32_t>(T < 65535 ? T : 65535));
  join_kernel<<<grid, 256, 0, st>>>(z, slices, static_cast<int>(R), static_cast<int>(m), pos, weight,
                                    static_cast<int>(T), k, residual, ldr, out, ldo,
                                    static_cast<int>(ldz),
                                    dt);
  return hipGetLastError();
}

}  // namespace lq
