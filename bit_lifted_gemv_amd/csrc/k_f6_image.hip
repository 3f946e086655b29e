// 16-bit lifted activations into the float6-part operand image of the product
// for many tokens (k_gemm_f6.hip; layout and arithmetic in f6_parts.h, H = 2).
// A wave takes 64 blocks of 32 positions, whose parts are consecutive in the
// image: it loads them with whole lines, turns each lane's block into parts
// (LDS between, both ways) and stores whole lines again.  Bound by the bytes
// read and written (2 and 2.4 per position of three parts, 3.1 of four, 3.9 of
// five): 4096 x 8192 of three in 26 us, 3000 x 28672 of four in 66 (6.7 TB/s),
// and about 8 us at least.  `zero_row`: one more row of zeros follows the last
// (what a gathered row with an index out of range reads).
#include "f6_parts.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f6;

constexpr int kWaves = 4;
constexpr int kInPitch = 80;                    // bytes per block: banks of 16 lanes differ

template <bool BF16, int NP>
__global__ void __launch_bounds__(64 * kWaves) f6_image_kernel(const uint16_t* __restrict__ a,
                                                               int64_t rows, int K, int64_t lda,
                                                               int blocks, int64_t all_blocks,
                                                               uint8_t* __restrict__ img) {
  constexpr int GB = group_bytes(2, NP), kOut = 16 * GB;
  constexpr int kRegion = kOut > 64 * kInPitch ? kOut : 64 * kInPitch;
  __shared__ __align__(16) uint8_t lds[kWaves * kRegion];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* mine = lds + wave * kRegion;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * 64;
  if (first >= all_blocks) return;              // no barrier below: a wave's own region

  // sixteen consecutive blocks are of one row (a row is a multiple of 16)
  int64_t row = first <= UINT32_MAX ? static_cast<uint32_t>(first) / static_cast<uint32_t>(blocks)
                                    : first / blocks;
  int b16 = static_cast<int>(first - row * blocks);
  uint4 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j, b16 += 16) {
    if (b16 >= blocks) {
      b16 -= blocks;
      ++row;
    }
    const int k = b16 * 32 + lane * 8;
    v[j] = make_uint4(0, 0, 0, 0);              // K % 8 == 0: a chunk is all in or out
    if (row < rows && k < K) v[j] = *reinterpret_cast<const uint4*>(a + row * lda + k);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(mine + (16 * j + lane / 4) * kInPitch + lane % 4 * 16) = v[j];
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = *reinterpret_cast<const uint4*>(mine + lane * kInPitch + 16 * j);
  __builtin_amdgcn_wave_barrier();

  float x[32];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack8(v[j], BF16, x + 8 * j);
  const uint32_t e = block_exponent(largest_bits(v, BF16));
  u32x6 part[NP];
  split_block<NP>(x, e, part);
  // block 4 h + 2 j + u of a pair of groups is (h, u) of group j
  const int h = lane >> 2 & 1, u = lane & 1;
  uint8_t* g = mine + (lane / 8 * 2 + (lane >> 1 & 1)) * GB;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = (u * NP + p) * 2 + h;
    *reinterpret_cast<uint4*>(g + 16 * at) =
        make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
    *reinterpret_cast<uint2*>(g + tail_offset(2, NP) + 8 * at) = make_uint2(part[p][4], part[p][5]);
  }
  g[exp_offset(2, NP) + 2 * h + u] = static_cast<uint8_t>(e);
  __builtin_amdgcn_wave_barrier();

  const int64_t left = (all_blocks - first) / 4 * GB;   // image bytes from here on
  uint8_t* out = img + first / 4 * GB;
#pragma unroll
  for (int j = 0; j < (kOut + 1023) / 1024; ++j) {
    const int at = j * 1024 + lane * 16;
    if (at < kOut && at < left)
      *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(mine + at);
  }
}

}  // namespace

hipError_t launch_f6_image(const void* a, lq_dtype dt, int64_t rows, bool zero_row, int64_t K,
                           int64_t lda, int NP, void* img, hipStream_t st) {
  const int blocks = static_cast<int>(padded_positions(K) / 32);
  const int64_t all = (rows + zero_row) * blocks;
  const int64_t grid = (all + 64 * kWaves - 1) / (64 * kWaves);
  auto run = [&](auto* k) {
    k<<<dim3(static_cast<uint32_t>(grid)), 64 * kWaves, 0, st>>>(
        static_cast<const uint16_t*>(a), rows, static_cast<int>(K), lda, blocks, all,
        static_cast<uint8_t*>(img));
    return hipGetLastError();
  };
  if (NP == 3) return dt == LQ_BF16 ? run(f6_image_kernel<true, 3>) : run(f6_image_kernel<false, 3>);
  if (NP == 4) return dt == LQ_BF16 ? run(f6_image_kernel<true, 4>) : run(f6_image_kernel<false, 4>);
  return dt == LQ_BF16 ? run(f6_image_kernel<true, 5>) : run(f6_image_kernel<false, 5>);
}

}  // namespace lq
