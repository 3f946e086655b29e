// Quantization to 8-bit floating point with a power of two per 128 positions
// of a row (lq_quant8) or per 128 x 128 block (lq_quant8_blocks):
//   byte  = 127 + min { e : largest finite |x| of the block <= top 2^e }
//   value = round(x 2^(127 - byte)).
// A power of two costs no accuracy in floating point (only the range below the
// smallest normal value, at most one binade of it), makes the division exact,
// so that results do not depend on how it is carried out, and is what the
// matrix instructions of the product take as a scale.
//
// Bound by memory: each value read once, held in registers between the maximum
// and the rounding.
#include "f8.h"
#include "lq_internal.h"

namespace lq {
namespace {

using namespace f8;

// Eight consecutive values of a row of n from position k, zeros behind it, as they
// lie in memory (16 bytes at any address: global memory takes them).
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

template <int DT>
struct Eight {
  static constexpr int WORDS = DT == LQ_F32 ? 8 : 4;
  uint32_t w[WORDS] = {};
};
template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void* row, int64_t k, int64_t n) {
  Eight<DT> v;
  const uint8_t* p = static_cast<const uint8_t*>(row) + k * (DT == LQ_F32 ? 4 : 2);
  if (k + 8 <= n) {
#pragma unroll
    for (int x = 0; x < v.WORDS / 4; ++x) {
      const i32x4 y = *reinterpret_cast<const i32x4_any*>(p + 16 * x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[4 * x + i] = y[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k + i >= n) break;
      if (DT == LQ_F32) v.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else v.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    }
  }
  return v;
}
template <int DT>
__device__ __forceinline__ void values(const Eight<DT>& e, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = DT == LQ_F32 ? __uint_as_float(e.w[i % Eight<DT>::WORDS])
                        : i % 2 ? high16<DT>(e.w[i / 2]) : low16<DT>(e.w[i / 2]);
}

__device__ __forceinline__ float largest8(const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_magnitude(v[i]));
  return m;
}

template <int T>
__device__ __forceinline__ uint2 round8(const float (&v)[8], int byte) {
  return make_uint2(round4<T>(v[0], v[1], v[2], v[3], byte), round4<T>(v[4], v[5], v[6], v[7], byte));
}

// Rows: 16 lanes per block of 128 positions, so a wave takes 512 positions and
// writes their four exponents as one word (rows of exponents are whole words).
// U such pieces per wave, their loads on the way together.
template <int DT, int T, int U>
__global__ void __launch_bounds__(256) quant8_rows_kernel(const void* __restrict__ x, int64_t units,
                                                          int64_t K, int64_t ld, int per_row,
                                                          uint8_t* __restrict__ q, int64_t ldq,
                                                          uint8_t* __restrict__ exps, int64_t lde) {
  constexpr int ESZ = DT == LQ_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6)) * U;
  Eight<DT> raw[U];
  int64_t row[U];
  int at[U];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int64_t u = min(u0 + c, units - 1);
    row[c] = u / per_row;
    at[c] = static_cast<int>(u - row[c] * per_row);
    raw[c] = load8<DT>(static_cast<const uint8_t*>(x) + row[c] * ld * ESZ, at[c] * int64_t{512} + lane * 8, K);
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    if (u0 + c >= units) return;
    int byte;
    uint2 bits;
    if constexpr (DT != LQ_F32 && T == LQ_E4M3) {          // the same in a third of the instructions
      const auto& w = raw[c].w;
      byte = block16<DT, 4, 1, 8>(w);
      const float scale = power_of_two(byte);
      bits = make_uint2(round16<DT>(w[0], w[1], scale), round16<DT>(w[2], w[3], scale));
    } else {
      float v[8];
      values(raw[c], v);
      float m = largest8(v);
#pragma unroll
      for (int d = 1; d < 16; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
      byte = block_exponent<T>(m);
      bits = round8<T>(v, byte);
    }
    const int64_t k = at[c] * int64_t{512} + lane * 8;
    if (k < (K + 127) / 128 * 128) *reinterpret_cast<uint2*>(q + row[c] * ldq + k) = bits;
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      word |= static_cast<uint32_t>(__builtin_amdgcn_readlane(byte, 16 * b)) << (8 * b);
    if (lane == 0) *reinterpret_cast<uint32_t*>(exps + row[c] * lde + at[c] * 4) = word;
  }
}

// Blocks: a workgroup per 128 x 128 block, eight rows of 16 lanes at a time per
// two waves.  Bound by memory: 28672 x 4096 float32 103 us (5.7 TB/s), bfloat16 67 (5.25), 64
// experts of 2816 x 2048 bfloat16 206 (5.4).
template <int DT>
__global__ void __launch_bounds__(256) quant8_blocks_kernel(const void* __restrict__ w, int m,
                                                            int64_t K, int64_t ld,
                                                            uint8_t* __restrict__ q, int64_t ldq,
                                                            uint8_t* __restrict__ exps, int64_t lde) {
  constexpr int ESZ = DT == LQ_F32 ? 4 : 2;
  __shared__ float part[4];
  const int tid = threadIdx.x, lane = tid & 15, r0 = blockIdx.y * 128 + (tid >> 4);
  const int64_t first = static_cast<int64_t>(blockIdx.z) * m;
  const int64_t k = blockIdx.x * int64_t{128} + lane * 8;
  Eight<DT> raw[8];
  float v[8], largest = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    raw[i] = load8<DT>(static_cast<const uint8_t*>(w) + (first + min(r, m - 1)) * ld * ESZ, k, K);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    values(raw[i], v);
    largest = fmaxf(largest, largest8(v));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) largest = fmaxf(largest, __shfl_xor(largest, d));
  if ((tid & 63) == 0) part[tid >> 6] = largest;
  __syncthreads();
  const int byte = block_exponent<LQ_E4M3>(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    values(raw[i], v);
    if (r < m) *reinterpret_cast<uint2*>(q + (first + r) * ldq + k) = round8<LQ_E4M3>(v, byte);
  }
  if (tid == 0) {
    const int64_t strip = static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
    exps[strip * lde + blockIdx.x] = static_cast<uint8_t>(byte);
  }
}

template <int DT, int T, int U>
hipError_t rows(const void* x, int64_t n, int64_t K, int64_t ld, uint8_t* q, int64_t ldq,
                uint8_t* exps, int64_t lde, hipStream_t st) {
  const int per_row = static_cast<int>((K + 511) / 512);
  constexpr int64_t most = int64_t{1} << 22;                  // workgroups of a launch
  const int64_t rows_per = most * 4 * U / per_row;
  for (int64_t r = 0; r < n; r += rows_per) {
    const int64_t some = n - r < rows_per ? n - r : rows_per;
    const int64_t groups = (some * per_row + 4 * U - 1) / (4 * U);
    quant8_rows_kernel<DT, T, U><<<static_cast<uint32_t>(groups), 256, 0, st>>>(
        static_cast<const uint8_t*>(x) + r * ld * (DT == LQ_F32 ? 4 : 2), some * per_row, K, ld,
        per_row, q + r * ldq, ldq, exps + r * lde, lde);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// One piece a wave where there are few (16 rows of 4096 and their product 32.5 us, two
// pieces 33.2; 4096 rows of 4096 bfloat16 to e5m2 11.3, four 12.1), four of 16-bit values
// where they fill the card many times (4096 rows of 14336 to e4m3: 29 us, 6.0 TB/s; one 35,
// two 33, eight 33; to e5m2 32; one 35.6); of float32 one (48 us; two 49, four 51).
template <int DT, int T>
hipError_t by_size(const void* x, int64_t n, int64_t K, int64_t ld, uint8_t* q, int64_t ldq,
                   uint8_t* exps, int64_t lde, hipStream_t st) {
  if constexpr (DT != LQ_F32) {
    if (n * ((K + 511) / 512) > int64_t{128} * num_cus())
      return rows<DT, T, 4>(x, n, K, ld, q, ldq, exps, lde, st);
  }
  return rows<DT, T, 1>(x, n, K, ld, q, ldq, exps, lde, st);
}

template <int DT>
hipError_t by_type(const void* x, int64_t n, int64_t K, int64_t ld, uint8_t* q, lq_dtype type,
                   int64_t ldq, uint8_t* exps, int64_t lde, hipStream_t st) {
  return type == LQ_E4M3 ? by_size<DT, LQ_E4M3>(x, n, K, ld, q, ldq, exps, lde, st)
                         : by_size<DT, LQ_E5M2>(x, n, K, ld, q, ldq, exps, lde, st);
}

template <int DT>
hipError_t blocks(const void* w, int64_t E, int64_t m, int64_t K, int64_t ld, uint8_t* q,
                  int64_t ldq, uint8_t* exps, int64_t lde, hipStream_t st) {
  const dim3 grid(static_cast<uint32_t>((K + 127) / 128), static_cast<uint32_t>((m + 127) / 128),
                  static_cast<uint32_t>(E));
  quant8_blocks_kernel<DT><<<grid, 256, 0, st>>>(w, static_cast<int>(m), K, ld, q, ldq, exps, lde);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant8(const void* x, lq_dtype dt, int64_t n, int64_t K, int64_t ld, uint8_t* q,
                         lq_dtype type, int64_t ldq, uint8_t* exps, int64_t lde, hipStream_t st) {
  switch (dt) {
    case LQ_F32: return by_type<LQ_F32>(x, n, K, ld, q, type, ldq, exps, lde, st);
    case LQ_F16: return by_type<LQ_F16>(x, n, K, ld, q, type, ldq, exps, lde, st);
    default: return by_type<LQ_BF16>(x, n, K, ld, q, type, ldq, exps, lde, st);
  }
}

hipError_t launch_quant8_blocks(const void* w, lq_dtype dt, int64_t E, int64_t m, int64_t K,
                                int64_t ld, uint8_t* q, int64_t ldq, uint8_t* exps, int64_t lde,
                                hipStream_t st) {
  switch (dt) {
    case LQ_F32: return blocks<LQ_F32>(w, E, m, K, ld, q, ldq, exps, lde, st);
    case LQ_F16: return blocks<LQ_F16>(w, E, m, K, ld, q, ldq, exps, lde, st);
    default: return blocks<LQ_BF16>(w, E, m, K, ld, q, ldq, exps, lde, st);
  }
}

}  // namespace lq
