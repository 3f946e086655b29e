// What the products on float6 parts share behind the sum: diag(s), bias,
// activation (gated or not), residual and the store in the output's type.
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f6 {

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case LQ_ACT_RELU: return z < 0.f ? 0.f : z;           // a NaN stays one
    case LQ_ACT_SILU: return z / (1.f + expf(-z));
    case LQ_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case LQ_ACT_GELU_TANH:
      return 0.5f * z * (1.f + tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

__device__ __forceinline__ float load_typed(const void* p, int dt, int64_t i) {
  return dt == LQ_F32 ? static_cast<const float*>(p)[i]
                      : dt == LQ_F16 ? f16_bits_to_float(static_cast<const uint16_t*>(p)[i])
                                     : bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}

// Round to nearest even; a NaN stays one.
__device__ __forceinline__ uint16_t round16(float v, int dt) {
  if (dt == LQ_F16) return float_to_f16_bits_rne(v);
  return v != v ? uint16_t{0x7FC0} : float_to_bf16_bits_rne(v);
}

// y[0 .. 3]: the outputs of columns o .. o + 3 of one token, `n` of them
// inside; adds the residual and stores.  `wide`: 4 outputs at o can go in
// one store (and load) of 8 or 16 bytes.
__device__ __forceinline__ void finish4(float (&y)[4], int n, bool wide, const void* residual,
                                        int64_t at_residual, void* out, int64_t at, int dt) {
  if (wide && n == 4) {
    if (dt == LQ_F32) {
      if (residual) {
        const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(residual) + at_residual);
        y[0] += r.x; y[1] += r.y; y[2] += r.z; y[3] += r.w;
      }
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
      if (residual) {
        const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(residual) + at_residual);
        const uint16_t q[4] = {static_cast<uint16_t>(r.x), static_cast<uint16_t>(r.x >> 16),
                               static_cast<uint16_t>(r.y), static_cast<uint16_t>(r.y >> 16)};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] += dt == LQ_F16 ? f16_bits_to_float(q[j]) : bf16_bits_to_float(q[j]);
      }
      uint2 v;
      v.x = round16(y[0], dt) | static_cast<uint32_t>(round16(y[1], dt)) << 16;
      v.y = round16(y[2], dt) | static_cast<uint32_t>(round16(y[3], dt)) << 16;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = v;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= n) break;
    if (residual) y[j] += load_typed(residual, dt, at_residual + j);
    if (dt == LQ_F32) static_cast<float*>(out)[at + j] = y[j];
    else static_cast<uint16_t*>(out)[at + j] = round16(y[j], dt);
  }
}

}  // namespace f6
}  // namespace lq
