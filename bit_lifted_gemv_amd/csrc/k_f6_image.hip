// 16-bit lifted activations into the float6-part operand image of the
// products in k_gemm_f6.hip and k_gemv_f6.hip (layout and arithmetic in
// f6_parts.h).  One thread per (token, block of 32 positions): four 16-byte
// loads, the block's exponent, the parts (one conversion instruction each),
// one 16-byte and one 8-byte store per part.  `zero_row`: one more row of zeros
// follows the last (what a gathered row with an index out of range reads).
#include "f6_parts.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

template <int DT, int H, int NP>
__global__ void __launch_bounds__(256) f6_image_kernel(const uint16_t* __restrict__ a, int64_t rows,
                                                       int64_t zero_row, int K, int64_t lda, int blocks,
                                                       uint8_t* __restrict__ img) {
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = idx / blocks;
  if (row >= rows) return;
  const int b = static_cast<int>(idx - row * blocks);
  uint4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = 32 * b + 8 * j;               // K % 8 == 0: a chunk is all in or out
    v[j] = make_uint4(0, 0, 0, 0);
    if (k < K && row != zero_row) v[j] = *reinterpret_cast<const uint4*>(a + row * lda + k);
  }
  float x[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack8(v[j], DT == LQ_BF16, x + 8 * j);
  const uint32_t e = block_exponent(largest_bits(v, DT == LQ_BF16));
  u32x6 part[NP];
  split_block<NP>(x, e, part);
  constexpr int U = group_steps(H), per = H * U;  // blocks per group
  int c, h, u;                                    // this block's group and place
  if (H == 2) {
    c = b / 8 * 2 + (b >> 1 & 1);
    h = b >> 2 & 1;
    u = b & 1;
  } else {
    c = b / per;
    h = b / U % H;
    u = b % U;
  }
  uint8_t* g = img + (row * (blocks / per) + c) * group_bytes(H, NP);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = (u * NP + p) * H + h;
    *reinterpret_cast<uint4*>(g + 16 * at) =
        make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
    *reinterpret_cast<uint2*>(g + tail_offset(H, NP) + 8 * at) = make_uint2(part[p][4], part[p][5]);
  }
  g[exp_offset(H, NP) + U * h + u] = static_cast<uint8_t>(e);
}

template <int H, int NP>
hipError_t launch(const void* a, lq_dtype dt, int64_t rows, bool zero_row, int64_t K, int64_t lda,
                  void* img, hipStream_t st) {
  const int blocks = static_cast<int>(padded_positions(K) / 32);
  const int64_t all = rows + zero_row;
  const int64_t grid = (all * blocks + 255) / 256;
  const auto* p = static_cast<const uint16_t*>(a);
  if (dt == LQ_BF16)
    f6_image_kernel<LQ_BF16, H, NP><<<dim3(static_cast<uint32_t>(grid)), 256, 0, st>>>(
        p, all, zero_row ? rows : -1, static_cast<int>(K), lda, blocks, static_cast<uint8_t*>(img));
  else
    f6_image_kernel<LQ_F16, H, NP><<<dim3(static_cast<uint32_t>(grid)), 256, 0, st>>>(
        p, all, zero_row ? rows : -1, static_cast<int>(K), lda, blocks, static_cast<uint8_t*>(img));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_f6_image(const void* a, lq_dtype dt, int64_t rows, bool zero_row, int64_t K,
                           int64_t lda, int H, int NP, void* img, hipStream_t st) {
  if (H == 2)
    return NP == 3 ? launch<2, 3>(a, dt, rows, zero_row, K, lda, img, st)
                   : launch<2, 4>(a, dt, rows, zero_row, K, lda, img, st);
  return NP == 3 ? launch<4, 3>(a, dt, rows, zero_row, K, lda, img, st)
                 : launch<4, 4>(a, dt, rows, zero_row, K, lda, img, st);
}

}  // namespace lq
