// The way out of the experts: out[t] = residual[t] + sum_j weight[t][j]
// z[pos[t][j]], z float32 rows in the sorted order (lq_gemm_join).  A choice
// with a position outside [0, R) adds nothing.  Sums in the order of j.
// One thread per token and four columns; bound by reading z once.
#include "f6_epilogue.h"
#include "lq_internal.h"

namespace lq {
namespace {

__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ z, int R, int m,
                                                   const int* __restrict__ pos,
                                                   const float* __restrict__ weight, int T, int k,
                                                   const void* residual, int64_t ldr, void* out,
                                                   int64_t ldo, int ldz, f6::OutputTypes types) {
  const int o = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (o >= m) return;
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; ++j) {
      const int64_t c = static_cast<int64_t>(t) * k + j;
      const int p = pos[c];
      if (p < 0 || p >= R) continue;
      const float w = weight[c];
      const float4 v = *reinterpret_cast<const float4*>(z + static_cast<int64_t>(p) * ldz + o);
      y[0] += w * v.x;
      y[1] += w * v.y;
      y[2] += w * v.z;
      y[3] += w * v.w;
    }
    f6::finish4(y, min(4, m - o), types, residual, t * ldr + o, out, t * ldo + o);
  }
}

}  // namespace

hipError_t launch_join(const float* z, int64_t R, int64_t m, int64_t ldz, const int* pos,
                       const float* weight, int64_t T, int k, const void* residual, int64_t ldr,
                       void* out, int64_t ldo, int dt, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((m + 1023) / 1024),
                  static_cast<uint32_t>(T < 65535 ? T : 65535));
  join_kernel<<<grid, 256, 0, st>>>(z, static_cast<int>(R), static_cast<int>(m), pos, weight,
                                    static_cast<int>(T), k, residual, ldr, out, ldo,
                                    static_cast<int>(ldz),
                                    f6::output_types(out, ldo, residual, ldr, dt));
  return hipGetLastError();
}

}  // namespace lq
