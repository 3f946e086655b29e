// Eight-bit floating point (OCP e4m3, e5m2) with one power of two per 128
// positions: the exponent of a block and the rounding, shared by the kernels
// that quantize (k_quant8.hip, k_gemv8.hip), and the way to bfloat16.
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f8 {

constexpr int kBlock = 128;

template <int T>
constexpr float top() { return T == LQ_E4M3 ? 448.f : 57344.f; }   // 7/8 2^9, 7/8 2^16

// |x|, 0 for infinities and NaN: a block's scale is that of its finite values.
__device__ __forceinline__ float finite_magnitude(float x) {
  const float m = fabsf(x);
  return m < __builtin_inff() ? m : 0.f;
}

// e + 127 with e the smallest integer >= -127 such that largest <= top 2^e; 127
// (scale 1) for a block of zeros.  largest = part 2^x with part in [1/2, 1), and
// top = 7/8 2^9 (2^16), so e = x - 9 (16), one more where part > 7/8.  At most
// 128 - 9 + 1 + 127 = 247.
template <int T>
__device__ __forceinline__ int block_exponent(float largest) {
  const int x = __builtin_amdgcn_frexp_expf(largest);
  const float part = __builtin_amdgcn_frexp_mantf(largest);
  const int e = x - (T == LQ_E4M3 ? 9 : 16) + (part > 0.875f ? 1 : 0) + 127;
  return largest > 0.f ? max(e, 0) : 127;
}

// Four values scaled by 2^(127 - byte) (exact) and rounded once, to nearest
// even, in one word.  Finite ones lie within the type.  e4m3 has no infinity:
// one becomes a NaN, as a NaN does.
template <int T>
__device__ __forceinline__ uint32_t round4(float x0, float x1, float x2, float x3, int byte) {
  float x[4] = {x0, x1, x2, x3};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (T == LQ_E4M3) x[i] = fabsf(x[i]) < __builtin_inff() ? x[i] : __builtin_nanf("");
    x[i] = __builtin_amdgcn_ldexpf(x[i], 127 - byte);
  }
  int w = 0;
  if (T == LQ_E4M3) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(x[0], x[1], w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(x[2], x[3], w, true);
  }
  return static_cast<uint32_t>(w);
}

// 2^(byte - 127) for a byte of an exponent (0: a subnormal); 255 stands for NaN.
__device__ __forceinline__ float power_of_two(uint32_t byte) {
  return __uint_as_float(max(byte << 23, 0x00400000u) | (byte + 1) >> 8 << 22);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight 8-bit values times 2^(byte - 127) in bfloat16.
template <int T>
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x8 v;
  const int w[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bf16x2 a, b;
    if (T == LQ_E5M2) {
      a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w[i], scale, false);
      b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w[i], scale, true);
    } else {
      a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false);
      b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true);
    }
    v[4 * i] = a[0]; v[4 * i + 1] = a[1]; v[4 * i + 2] = b[0]; v[4 * i + 3] = b[1];
  }
  return v;
}

// 2 N 16-bit values of a lane, lanes FIRST .. LAST apart (doubling) sharing a block, to
// e4m3: the same as above by packed maxima and the scaled conversion, which divides
// by a power of two and rounds once.
template <int DT, int N, int FIRST, int LAST>
__device__ __forceinline__ int block16(const uint32_t (&w)[N]) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  constexpr int kInf = DT == LQ_F16 ? 0x7C00 : 0x7F80;
  u16x2 most = {0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
  int m = max(static_cast<int>(most[0]), static_cast<int>(most[1]));
  if (m >= kInf) {                                         // infinities and NaN do not count
    m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int lo = w[i] & 0x7FFF, hi = w[i] >> 16 & 0x7FFF;
      m = max(m, max(lo < kInf ? lo : 0, hi < kInf ? hi : 0));
    }
  }
#pragma unroll
  for (int d = FIRST; d <= LAST; d *= 2) m = max(m, __shfl_xor(m, d));
  return block_exponent<LQ_E4M3>(DT == LQ_F16 ? f16_bits_to_float(static_cast<uint16_t>(m))
                                              : __uint_as_float(static_cast<uint32_t>(m) << 16));
}
template <int DT>
__device__ __forceinline__ int round16(uint32_t lo, uint32_t hi, float scale) {
  typedef short i16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  i16x2 v = {0, 0};
  if (DT == LQ_F16) {
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(v, __builtin_bit_cast(f16x2, lo), scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(v, __builtin_bit_cast(f16x2, hi), scale, true);
  } else {
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, lo), scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, hi), scale, true);
  }
  return __builtin_bit_cast(int, v);
}

// Two 16-bit values of a word
template <int DT>
__device__ __forceinline__ float low16(uint32_t w) {
  return DT == LQ_F16 ? f16_bits_to_float(static_cast<uint16_t>(w)) : __uint_as_float(w << 16);
}
template <int DT>
__device__ __forceinline__ float high16(uint32_t w) {
  return DT == LQ_F16 ? f16_bits_to_float(static_cast<uint16_t>(w >> 16))
                      : __uint_as_float(w & 0xFFFF0000u);
}

}  // namespace f8
}  // namespace lq
