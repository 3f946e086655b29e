// Activations as sums of float6 parts, and 1-bit weights as float4 +-1: the
// operands of v_mfma_scale_f32_*_f8f6f4, which multiplies float4 by float6
// at twice the rate of float8 (measured here 9.2 against 4.9 PFLOP/s with
// independent accumulators, 16-bit operands 2.4).
//
// Parts.  Per block of 32 positions of one token, with f the biased exponent
// of its largest |x| and e = max(f - 2, 20), y = x 2^(127 - e) lies below 8
// in magnitude; p0 = fp6(y), p1 = fp6(16 (y - p0)), p2 = fp6(16 (16 (y - p0)
// - p1)) (E2M3: 4 significant bits up to 7.5, step 1/8 below 2; every
// remainder is exact in float32), and part p carries the power of two
// e - part_shift(p) as its hardware scale, which is what the one exponent
// byte per block holds.  The remainders are at most 1/4, 1/8 and 1/16 of a
// unit of their part's scale (16-bit values above 7.75 come out exactly), so
// the fourth part is taken 64 times finer and not 16, and the fifth, behind a
// remainder of 1/8, 32 times.  The parts NP follow from the result's type, so
// that what they lose stays below its own rounding (shares of the result,
// root mean squares of sums of 8192, Gaussian values / with one position in a
// hundred 20 times the others):
//   bfloat16 results, 1.7e-3: three parts, 2^-14 of the block's largest value
//     (exact for a bfloat16 above 2^-6 or a float16 above 2^-3 of it); lost
//     1.1e-5 / 7.8e-5 of bfloat16 values, 3.2e-5 / 1.3e-4 of float16 ones, 1.4
//     times that through a gate;
//   float16 results, 2.1e-4: four parts, 2^-19; lost below 1e-6 (three would
//     make the error of gated float16 results with such values 2.8e-4);
//   float32 results: five parts, 2^-24, below the sums' own rounding (four lost
//     1.3e-6 of a float16 result with such values).
// The exponent e is at least 20: the last scale, e - 19, stays above 0
// and subtracting it from four packed bytes borrows nothing.  The products with
// +-1 are exact and are summed in float32.  A block with an infinity or a NaN
// has e = 255, which the matrix cores read as NaN: its token's results are
// all NaN.
//
// Image.  A token's positions come in groups of H U blocks: H = 2, U = 2 for
// the 32 x 32 x 64 instruction, H = 4, U = 4 for the 16 x 16 x 128 one.  Per
// token and group:
//   [u][part][h] the first 16 bytes of an operand (24 bytes, 32 x 6 bits),
//   [u][part][h] its last 8, then 16 bytes with the exponents, [h][u].
// A group takes an odd number of 16-byte chunks, so rows of groups in LDS
// start in different banks.  With H = 4, lane group h holds block 4 h + u of
// the group at step u, so that its four sign words are one 16-byte load.
// With H = 2 the same holds over a pair of groups (256 positions): block
// 4 h + 2 j + u of the pair is (h, u) of its group j.  Element 8 q + t of a
// block is its position 4 t + q: the order in which three shifts and four
// bit selects turn a sign word into float4 +-1 (expand_signs).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lq_internal.h"

namespace lq {
namespace f6 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x6 __attribute__((ext_vector_type(6)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

constexpr int kPadPositions = 512;      // images cover whole multiples of this, zero past K

constexpr int part_shift(int p) { return p < 3 ? 4 * p : 5 * p - 1; }

constexpr int group_steps(int H) { return H == 2 ? 2 : 4; }
constexpr int group_positions(int H) { return 32 * H * group_steps(H); }
// Offsets of a group's sections, and its length.
constexpr int tail_offset(int H, int NP) { return 16 * H * group_steps(H) * NP; }
constexpr int exp_offset(int H, int NP) { return 24 * H * group_steps(H) * NP; }
constexpr int group_bytes(int H, int NP) { return exp_offset(H, NP) + 16; }

inline int64_t padded_positions(int64_t K) {
  return (K + kPadPositions - 1) / kPadPositions * kPadPositions;
}
inline int64_t row_bytes(int64_t K, int H, int NP) {
  return padded_positions(K) / group_positions(H) * group_bytes(H, NP);
}

// A per-lane value that the compiler keeps in a vector register.
__device__ __forceinline__ uint32_t held(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// A word of 32 sign bits as float4: a set bit gives -1.0 (0xA), a clear one
// +1.0 (0x2), so products hold -sigma and the epilogue multiplies by -s.
// Three shifts and four bit-field inserts; two = held(0x22222222).
__device__ __forceinline__ i32x8 expand_signs(uint32_t w, uint32_t two) {
  const uint32_t m = 0x88888888u;
  i32x8 a;
  a[0] = static_cast<int>(((w << 3) & m) | (two & ~m));
  a[1] = static_cast<int>(((w << 2) & m) | (two & ~m));
  a[2] = static_cast<int>(((w << 1) & m) | (two & ~m));
  a[3] = static_cast<int>((w & m) | (two & ~m));
  a[4] = a[5] = a[6] = a[7] = 0;         // unused with a float4 operand
  return a;
}

// Scale byte of a block from the bits of its largest |x|.
__device__ __forceinline__ uint32_t block_exponent(uint32_t largest) {
  const int f = static_cast<int>(largest >> 23);
  return f == 255 ? 255u : static_cast<uint32_t>(max(f - 2, 20));
}

// Eight 16-bit values of a 16-byte load.
__device__ __forceinline__ void unpack8(const uint4& v, bool bf16, float* x) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      x[2 * i] = __uint_as_float(q[i] << 16);
      x[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    } else {
      x[2 * i] = f16_bits_to_float(static_cast<uint16_t>(q[i]));
      x[2 * i + 1] = f16_bits_to_float(static_cast<uint16_t>(q[i] >> 16));
    }
  }
}

// Float32 bits of the largest |x| of 16-bit values, two per word (an infinity
// or a NaN counts as larger than any number).
template <int N>
__device__ __forceinline__ uint32_t largest_bits(const uint4 (&v)[N], bool bf16) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 most = {0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, q[j] & 0x7FFF7FFFu));
  }
  const uint16_t m = most[0] > most[1] ? most[0] : most[1];
  return __float_as_uint(bf16 ? bf16_bits_to_float(m) : f16_bits_to_float(m));
}

// The parts of a block of 32 values (x in position order), whose scale byte
// is e.
template <int NP>
__device__ __forceinline__ void split_block(const float (&x)[32], uint32_t e, u32x6 (&part)[NP]) {
  f32x16 even, odd;                      // elements 0, 2, 4, ... and 1, 3, 5, ...
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    even[i] = x[4 * ((2 * i) & 7) + (2 * i) / 8];
    odd[i] = x[4 * ((2 * i + 1) & 7) + (2 * i + 1) / 8];
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const float scale = __uint_as_float((e - part_shift(p)) << 23);
    part[p] = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(even, odd, scale);
    if (p + 1 < NP) {
      const f32x32 back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(part[p], scale);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        even[i] -= back[2 * i];
        odd[i] -= back[2 * i + 1];
      }
    }
  }
}

}  // namespace f6
}  // namespace lq
