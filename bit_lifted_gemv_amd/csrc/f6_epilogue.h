// What the products on float6 parts share behind the sum: diag(s), bias,
// activation (gated or not), residual and the store in the output's type.
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f6 {

// 1 / (1 + exp(-x)) to a few 2^-24 of itself (hardware exponential and
// reciprocal, 1 unit in the last place each); 0 and 1 far out.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

__device__ __forceinline__ void activate4(float (&z)[4], int act) {
  switch (act) {
    case LQ_ACT_RELU:
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] = z[c] < 0.f ? 0.f : z[c];     // a NaN stays one
      break;
    case LQ_ACT_SILU:
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] *= sigmoid(z[c]);
      break;
    case LQ_ACT_GELU:
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] = 0.5f * z[c] * (1.f + erff(z[c] * 0.70710678118654752f));
      break;
    case LQ_ACT_GELU_TANH:                                            // (1 + tanh u) / 2 = sigmoid(2 u)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        z[c] *= sigmoid(1.59576912160573071f * (z[c] + 0.044715f * z[c] * z[c] * z[c]));
      break;
    default: break;
  }
}

// -s and bias of rows row .. row + 3 of m (the tiles hold -sum); 0 past the
// last.  Buffer loads: 16 bytes at any float's address, range checked.
struct RowScales {
  float s[4], b[4];
};
__device__ __forceinline__ RowScales row_scales(const float* s, const float* bias, int row, int m) {
  RowScales r{};
  auto load = [&](const float* p, float (&v)[4]) {
    const __amdgpu_buffer_rsrc_t res = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(p), (short)0, m * 4, 0x00020000);
    const auto x = __builtin_amdgcn_raw_buffer_load_b128(res, row * 4, 0, 0);
    __builtin_memcpy(v, &x, 16);
  };
  load(s, r.s);
  if (bias) load(bias, r.b);
#pragma unroll
  for (int c = 0; c < 4; ++c) r.s[c] = -r.s[c];
  return r;
}
__device__ __forceinline__ void scaled(const float4& v, const RowScales& r, float (&z)[4]) {
  z[0] = v.x * r.s[0] + r.b[0];
  z[1] = v.y * r.s[1] + r.b[1];
  z[2] = v.z * r.s[2] + r.b[2];
  z[3] = v.w * r.s[3] + r.b[3];
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

// `wide`: four consecutive outputs go in one access of 8 or 16 bytes.
struct OutputTypes {
  int dt;
  bool wide;
};
__host__ __device__ __forceinline__ OutputTypes output_types(const void* out, int64_t ldo,
                                                             const void* residual, int64_t ldr,
                                                             int dt) {
  const uint64_t esz = dt == LQ_F32 ? 4 : 2;
  uint64_t bits = reinterpret_cast<uint64_t>(out) | static_cast<uint64_t>(ldo) * esz;
  if (residual) bits |= reinterpret_cast<uint64_t>(residual) | static_cast<uint64_t>(ldr) * esz;
  return {dt, bits % (4 * esz) == 0};
}

// y[0 .. 3]: outputs of four columns of one token, the first n of them
// inside; adds the residual and stores.
__device__ __forceinline__ void finish4(float (&y)[4], int n, const OutputTypes& types,
                                        const void* residual, int64_t at_residual, void* out,
                                        int64_t at) {
  const int dt = types.dt;
  if (types.wide && n == 4) {
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
