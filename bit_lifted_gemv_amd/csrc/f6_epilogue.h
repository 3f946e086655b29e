// What the products on float6 parts share behind the sum: diag(s), bias,
// activation (gated or not), residual and the store in the output's type.
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f6 {

// 1 / (1 + exp(-x)), relatively within 8 + 2 |x| times 2^-24 (hardware
// exponential and reciprocal, 1 unit in the last place each, and the rounding
// of the exponential's argument); 0 and 1 far out.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

// z (1 + erf(z / sqrt 2)) / 2 = z erfc(-z / sqrt 2) / 2, relatively within 16 (1 +
// z^2) 2^-24 for negative z too, where 1 + erf would cancel.  With x = |z| / sqrt
// 2 and t = 1 / (1 + x / 2), erfc(x) = exp(-x^2) (c1 t + ... + c9 t^9): the c of
// least largest relative error over 0 <= x <= 9.45 (2.1e-8, 1.1e-7 as rounded
// here), found by linear programming on exp(x^2) erfc(x) at 1000 points; past
// that the exponential is 0.
__device__ __forceinline__ float gelu(float z) {
  const float t = __builtin_amdgcn_rcpf(1.f + 0.35355339059327376f * fabsf(z));
  float p = -0.0579111204f;
  p = p * t + 0.279627591f;
  p = p * t - 0.478430659f;
  p = p * t + 0.269709527f;
  p = p * t - 0.0219781939f;
  p = p * t + 0.201153696f;
  p = p * t + 0.243395478f;
  p = p * t + 0.28234604f;
  p = p * t + 0.282087624f;
  // exp(-x^2) as 2^(-z^2 log2(e) / 2)
  const float half_erfc = 0.5f * p * t * __builtin_amdgcn_exp2f(-0.72134752044448170f * (z * z));
  return z * (z < 0.f ? half_erfc : 1.f - half_erfc);
}

template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
  switch (act) {
    case LQ_ACT_RELU:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = z[c] < 0.f ? 0.f : z[c];     // a NaN stays one
      break;
    case LQ_ACT_SILU:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] *= sigmoid(z[c]);
      break;
    case LQ_ACT_GELU:
#pragma unroll
      for (int c = 0; c < N; ++c) z[c] = gelu(z[c]);
      break;
    case LQ_ACT_GELU_TANH:                                            // (1 + tanh u) / 2 = sigmoid(2 u)
#pragma unroll
      for (int c = 0; c < N; ++c)
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

// Two values rounded to nearest even, one packed word.
__device__ __forceinline__ uint32_t round16x2(float lo, float hi, int dt) {
  if (dt == LQ_F16)
    return float_to_f16_bits_rne(lo) | static_cast<uint32_t>(float_to_f16_bits_rne(hi)) << 16;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}
__device__ __forceinline__ float value16(uint32_t bits, int dt) {
  const uint16_t b = static_cast<uint16_t>(bits);
  return dt == LQ_F16 ? f16_bits_to_float(b) : bf16_bits_to_float(b);
}

// Four outputs in one access of 8 or 16 bytes, at any address (global memory takes them).
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// The residual of four columns of one token, the first n of them inside, as
// it lies in memory (its conversion waits for its arrival).
struct Residual {
  uint32_t w[4];
};
__device__ __forceinline__ Residual load_residual(int n, int dt,
                                                  const void* residual, int64_t at) {
  Residual r{};
  if (!residual || n <= 0) return r;
  if (dt == LQ_F32) {
    const auto* p = static_cast<const uint32_t*>(residual) + at;
    if (n == 4) {
      const u32x4 v = *reinterpret_cast<const u32x4_any*>(p);
      r.w[0] = v[0]; r.w[1] = v[1]; r.w[2] = v[2]; r.w[3] = v[3];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) r.w[c] = p[c];
    }
  } else {
    const auto* p = static_cast<const uint16_t*>(residual) + at;
    if (n == 4) {
      const u32x2 v = *reinterpret_cast<const u32x2_any*>(p);
      r.w[0] = v[0]; r.w[1] = v[1];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) r.w[c / 2] |= static_cast<uint32_t>(p[c]) << (16 * (c % 2));
    }
  }
  return r;
}

__device__ __forceinline__ void add_residual(float (&y)[4], int dt, const Residual& r) {
  if (dt == LQ_F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] += __uint_as_float(r.w[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] += value16(r.w[c / 2] >> (16 * (c % 2)), dt);
  }
}

// The first n of four outputs; STREAM: whole 16-bit ones past the caches.
template <bool STREAM = false>
__device__ __forceinline__ void store4(const float (&y)[4], int n, int dt, void* out, int64_t at) {
  if (dt == LQ_F32) {
    float* to = static_cast<float*>(out) + at;
    if (n == 4) {
      *reinterpret_cast<u32x4_any*>(to) = u32x4{__float_as_uint(y[0]), __float_as_uint(y[1]),
                                                __float_as_uint(y[2]), __float_as_uint(y[3])};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < n) to[c] = y[c];
    }
    return;
  }
  const u32x2 v = {round16x2(y[0], y[1], dt), round16x2(y[2], y[3], dt)};
  uint16_t* to = static_cast<uint16_t*>(out) + at;
  if (n == 4) {
    if (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(to));
    else *reinterpret_cast<u32x2_any*>(to) = v;
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < n) to[c] = static_cast<uint16_t>(v[c / 2] >> (16 * (c % 2)));
  }
}

// Adds the residual to y and stores the first n of four outputs.
__device__ __forceinline__ void store4(float (&y)[4], int n, int dt,
                                       const Residual& r, bool add, void* out, int64_t at) {
  if (add) add_residual(y, dt, r);
  store4(y, n, dt, out, at);
}

__device__ __forceinline__ void finish4(float (&y)[4], int n, int dt,
                                        const void* residual, int64_t at_residual, void* out,
                                        int64_t at) {
  store4(y, n, dt, load_residual(n, dt, residual, at_residual), residual != nullptr, out, at);
}

}  // namespace f6
}  // namespace lq
