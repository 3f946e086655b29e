// Behind a product on float6 parts whose positions were split into slices
// (k_gemv_f6.hip, k_gemm_f6.hip): sums and epilogue.  Bound by reading the
// sums once, and by its launch.
#include "f6_epilogue.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

// The slices' scaled sums added in order, and the epilogue: a thread per row
// and four outputs, four slices' loads on their way at once.
__global__ void __launch_bounds__(128) f6_reduce_kernel(F6Product a) {
  const int out_m = a.gated ? a.m / 2 : a.m;
  const int o = (blockIdx.y * 128 + threadIdx.x) * 4;
  const int64_t row = blockIdx.x;
  const int n = min(4, out_m - o);
  if (n <= 0) return;
  // rows outside the runs are left as they were
  if (a.offsets && (row < a.offsets[0] || row >= a.offsets[a.E])) return;
  const int64_t step = static_cast<int64_t>(a.R) * a.ldz;
  auto sum = [&](int col, float (&v)[4]) {
    const float* z = a.sums + row * a.ldz + col;
    const bool whole = col % 4 == 0;            // rows are padded to whole fours
    for (int q = 0; q < a.slices; q += 4) {
      float x[4][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float* from = z + min(q + c, a.slices - 1) * step;
        if (whole) {
          const float4 y = *reinterpret_cast<const float4*>(from);
          x[c][0] = y.x; x[c][1] = y.y; x[c][2] = y.z; x[c][3] = y.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[c][j] = from[min(j, n - 1)];
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += q + c < a.slices ? x[c][j] : 0.f;
    }
  };
  float y[4] = {}, up[4] = {};
  sum(o, y);
  if (a.gated) sum(out_m + o, up);
  activate4(y, a.act);
  if (a.gated) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] *= up[j];
  }
  finish4(y, n, output_types(a.out, a.ldo, a.residual, a.ldr, a.out_dt), a.residual,
          row * a.ldr + o, a.out, row * a.ldo + o);
}

}  // namespace

hipError_t launch_f6_reduce(const F6Product& p, hipStream_t st) {
  const int out_m = p.gated ? p.m / 2 : p.m;
  // rows on the grid's x: there may be more than 65535
  f6_reduce_kernel<<<dim3(static_cast<uint32_t>(p.R), (out_m + 511) / 512), 128, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace lq
