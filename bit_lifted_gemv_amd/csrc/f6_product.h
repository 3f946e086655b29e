// Arguments of the float4 x float6 products (k_gemm_f6.hip, k_gemv_f6.hip)
// and the search for the expert run that a token tile belongs to.
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f6 {

// Tiles of TOK rows in expert e's run (0 past the last expert).  Offsets come
// from the device unchecked: runs are cut to [0, R].
__device__ __forceinline__ int run_tiles(const F6Product& a, int e, int TOK, int& lo, int& end) {
  lo = end = 0;
  if (e >= a.E) return 0;
  lo = min(max(a.offsets[e], 0), a.R);
  end = min(max(a.offsets[e + 1], lo), a.R);
  return (end - lo + TOK - 1) / TOK;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ int wave_total(int v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// The expert of tile `tile`, its first row and the end of its run; false past
// the last tile.
__device__ __forceinline__ bool find_run(const F6Product& a, int tile, int TOK, int lane,
                                         int& expert, int& row0, int& row_end) {
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    int lo, end;
    const int n = run_tiles(a, e0 + lane, TOK, lo, end);
    const int upto = before + wave_scan(n, lane);
    const uint64_t hit = __ballot(upto > tile);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int first = __shfl(upto - n, l);
      expert = __builtin_amdgcn_readfirstlane(e0 + l);
      row_end = __builtin_amdgcn_readfirstlane(__shfl(end, l));
      row0 = __builtin_amdgcn_readfirstlane(__shfl(lo, l)) + (tile - first) * TOK;
      return true;
    }
    before = __shfl(upto, 63);
  }
  return false;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const void*)p));
}

}  // namespace f6
}  // namespace lq
