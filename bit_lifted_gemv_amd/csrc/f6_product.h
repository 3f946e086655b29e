// The search for the expert run that a token tile belongs to, of the products
// with E matrices (their arguments hold E, R and the offsets).
#pragma once

#include "lq_internal.h"

namespace lq {
namespace f6 {

// Tiles of TOK rows in expert e's run (0 past the last expert).  Offsets come
// from the device unchecked: runs are cut to [0, R].
template <class Product>
__device__ __forceinline__ int run_tiles(const Product& a, int e, int TOK, int& lo, int& end) {
  lo = end = 0;
  if (e >= a.E) return 0;
  lo = min(max(a.offsets[e], 0), a.R);
  end = min(max(a.offsets[e + 1], lo), a.R);
  return end > lo ? 1 + (end - lo - 1) / TOK : 0;
}

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// What a wave knows of 64 experts' runs, lane e of expert e0 + e: bounds, and
// tiles up to and with it.
struct Runs {
  int lo, end, tiles, upto;
};
template <class Product>
__device__ __forceinline__ Runs load_runs(const Product& a, int e0, int before, int TOK, int lane) {
  Runs r;
  r.tiles = run_tiles(a, e0 + lane, TOK, r.lo, r.end);
  r.upto = before + wave_scan(r.tiles, lane);
  return r;
}
// The expert of tile `tile`, its first row and the end of its run, if it is
// one of these 64.
__device__ __forceinline__ bool find_in(const Runs& r, int e0, int tile, int TOK, int& expert,
                                        int& row0, int& row_end) {
  const uint64_t hit = __ballot(r.upto > tile);
  if (!hit) return false;
  const int l = __builtin_ctzll(hit);
  const int first = __shfl(r.upto - r.tiles, l);
  expert = __builtin_amdgcn_readfirstlane(e0 + l);
  row_end = __builtin_amdgcn_readfirstlane(__shfl(r.end, l));
  row0 = __builtin_amdgcn_readfirstlane(__shfl(r.lo, l) + (tile - first) * TOK);
  return true;
}
// The same over all experts; false past the last tile.
template <class Product>
__device__ __forceinline__ bool find_run(const Product& a, int tile, int TOK, int lane,
                                         int& expert, int& row0, int& row_end) {
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const Runs r = load_runs(a, e0, before, TOK, lane);
    if (find_in(r, e0, tile, TOK, expert, row0, row_end)) return true;
    before = __shfl(r.upto, 63);
  }
  return false;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const void*)p));
}

}  // namespace f6
}  // namespace lq
