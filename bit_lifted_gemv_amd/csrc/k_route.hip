// Router of a mixture-of-experts layer: per token the k largest of E logits
// (ties to the lowest expert), their softmax weights, and the stable order
// of the (token, choice) pairs by expert, as offsets, rows and positions.
//
// Two launches (one when a single workgroup holds every token).  A workgroup
// of 16 waves takes runs of 64 tokens; a wave takes one token at a time,
// lane l holding the logits of experts l, l + 64, ... as order-preserving
// integers.  A choice is a maximum over the wave (data-parallel moves within
// and across rows of lanes, no LDS), then the lowest expert among equal
// ones.  A token chooses an expert at most once, so a run's choices are one
// 64-bit mask of tokens per expert in LDS: counts and stable ranks are
// popcounts of it, whatever order the waves set the bits in.  The first
// launch writes the choices and each workgroup's counts per expert; the
// second adds the counts before its own (at most 256 workgroups) and
// scatters.  Bound by launch latency and the E logits per token read once.
#include "lq_internal.h"

namespace lq {
namespace {

constexpr int kRun = 64;                 // tokens per mask
constexpr int kThreads = 1024;
constexpr int kMaxGroups = 256;

// Order-preserving bits of a float; 0 for what is never chosen (NaN, -inf).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u || u == 0xFF800000u) return 0;
  // -0 and +0 are equal logits: both take the bits of +0
  if ((u & 0x7FFFFFFFu) == 0) return 0x80000000u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order_bits(uint32_t b) {
  return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t moved(uint32_t keep, uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      static_cast<int>(keep), static_cast<int>(v), CTRL, ROW_MASK, 0xF, false));
}

// Largest value over the wave, in every lane's hands (a scalar).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<0x111, 0xF>(0, v));   // row_shr 1, 2, 4, 8
  v = max(v, moved<0x112, 0xF>(0, v));
  v = max(v, moved<0x114, 0xF>(0, v));
  v = max(v, moved<0x118, 0xF>(0, v));
  v = max(v, moved<0x142, 0xA>(0, v));   // row_bcast 15
  v = max(v, moved<0x143, 0xC>(0, v));   // row_bcast 31
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

__device__ __forceinline__ float wave_sum(float v) {   // fixed order
  for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}

// The choices of one token by one wave: lane i < k gets choice i.
template <int N>
__device__ __forceinline__ void choose(const void* logits, int dt, int64_t base, int E, int k,
                                       bool renorm, int lane, int& id, float& weight) {
  uint32_t b[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = 64 * j + lane;
    float v = -INFINITY;
    if (e < E)
      v = dt == LQ_F32 ? static_cast<const float*>(logits)[base + e]
          : dt == LQ_F16 ? f16_bits_to_float(static_cast<const uint16_t*>(logits)[base + e])
                         : bf16_bits_to_float(static_cast<const uint16_t*>(logits)[base + e]);
    b[j] = order_bits(v);
  }
  id = -1;
  weight = 0.f;
  float top = 0.f, total = 0.f;
  uint32_t mine = 0;
  for (int i = 0; i < k; ++i) {
    uint32_t best = b[0];
#pragma unroll
    for (int j = 1; j < N; ++j) best = max(best, b[j]);
    const uint32_t largest = wave_max(best);
    if (largest == 0) break;             // nothing left to choose
    uint32_t far = 0;                    // ~expert, so that the largest is the lowest expert
#pragma unroll
    for (int j = N - 1; j >= 0; --j)
      if (b[j] == largest) far = ~static_cast<uint32_t>(64 * j + lane);
    const uint32_t e = ~wave_max(far);
    const float v = from_order_bits(largest);
    if (i == 0) {
      top = v;
      if (!renorm) {
        // softmax over every expert; +inf logits share the whole weight
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (b[j]) {
            const float x = from_order_bits(b[j]);
            t += x == top ? 1.f : expf(x - top);
          }
        total = wave_sum(t);
      }
    }
    const float p = v == top ? 1.f : expf(v - top);
    if (renorm) total += p;
    if (lane == i) {
      id = static_cast<int>(e);
      weight = p;
      mine = largest;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (e == static_cast<uint32_t>(64 * j + lane)) b[j] = 0;
  }
  if (mine) weight /= total;
}

struct RouteArgs {
  const void* logits;
  int dt;
  int64_t ld;
  const uint8_t* valid;
  int T, E, k, renorm;
  int* ids;
  float* weight;
  int* pos;
  int* rows;
  int* offsets;
  int* counts;                           // [groups][E]
  int groups, per;                       // workgroups, runs of 64 tokens per workgroup
};

// Positions of the pairs of run `run` from base[e] (LDS, the next free one
// of each expert) and the run's masks.
__device__ __forceinline__ void scatter(const RouteArgs& a, int run, const uint64_t* mask,
                                        const int* base, int tid) {
  for (int i = tid; i < kRun * a.k; i += kThreads) {
    const int t = run * kRun + i / a.k;
    if (t >= a.T) break;
    const int64_t at = static_cast<int64_t>(t) * a.k + i % a.k;
    const int e = a.ids[at];
    int p = -1;
    if (e >= 0) {
      p = base[e] + __popcll(mask[e] & ((uint64_t{1} << (t % kRun)) - 1));
      a.rows[p] = t;
    }
    a.pos[at] = p;
  }
}

// Exclusive sums of v over the workgroup's threads.
__device__ __forceinline__ int scan_workgroup(int v, int tid, int* part) {
  const int lane = tid & 63;
  int x = v;
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(x, d);
    if (lane >= d) x += o;
  }
  if (lane == 63) part[tid >> 6] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < (tid >> 6); ++w) before += part[w];
  return before + x - v;
}

template <int N, bool ONE>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(RouteArgs a) {
  __shared__ uint64_t mask[64 * N];
  __shared__ int total[64 * N];
  __shared__ int part[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = a.E;
  if (tid < E) total[tid] = 0;
  for (int r = 0; r < a.per; ++r) {
    const int run = blockIdx.x * a.per + r;
    if (tid < E) mask[tid] = 0;
    __syncthreads();
    for (int q = wave; q < kRun; q += 16) {
      const int t = run * kRun + q;
      if (t >= a.T) break;
      int id = -1;
      float weight = 0.f;
      if (!a.valid || a.valid[t])
        choose<N>(a.logits, a.dt, static_cast<int64_t>(t) * a.ld, E, a.k, a.renorm, lane, id,
                  weight);
      if (lane < a.k) {
        a.ids[static_cast<int64_t>(t) * a.k + lane] = id;
        a.weight[static_cast<int64_t>(t) * a.k + lane] = weight;
        if (id >= 0)
          atomicOr(reinterpret_cast<unsigned long long*>(&mask[id]), 1ull << q);
      }
    }
    __syncthreads();
    if (tid < E) total[tid] += __popcll(mask[tid]);
  }
  if (!ONE) {
    if (tid < E) a.counts[static_cast<int64_t>(blockIdx.x) * E + tid] = total[tid];
    return;
  }
  const int n = tid < E ? total[tid] : 0;
  const int before = scan_workgroup(n, tid, part);
  if (tid < E) {
    total[tid] = before;
    a.offsets[tid] = before;
    if (tid == E - 1) {
      a.offsets[E] = before + n;
      part[0] = before + n;
    }
  }
  __syncthreads();
  scatter(a, 0, mask, total, tid);
  for (int i = part[0] + tid; i < a.T * a.k; i += kThreads) a.rows[i] = -1;
}

template <int N>
__global__ void __launch_bounds__(kThreads) route_scatter_kernel(RouteArgs a) {
  __shared__ uint64_t mask[64 * N];
  __shared__ int base[64 * N];
  __shared__ int part[16];
  __shared__ int used;
  const int tid = threadIdx.x;
  const int E = a.E;
  // counts of every workgroup: those before this one, and all
  int mine = 0, all = 0;
  for (int e = tid; e < 64 * N; e += kThreads) base[e] = 0, mask[e] = 0;
  __syncthreads();
  {
    // thread (q, e): every (kThreads / E)-th workgroup's count of expert e
    const int lanes = kThreads / E;
    const int q = tid / E, e = tid % E;
    if (q < lanes) {
#pragma unroll 8
      for (int g = q; g < a.groups; g += lanes) {
        const int c = a.counts[static_cast<int64_t>(g) * E + e];
        all += c;
        mine += g < static_cast<int>(blockIdx.x) ? c : 0;
      }
      // integer sums: the order of the additions does not matter
      atomicAdd(&base[e], mine);
      atomicAdd(reinterpret_cast<int*>(&mask[e]), all);
    }
  }
  __syncthreads();
  const int n = tid < E ? static_cast<int>(mask[tid]) : 0;
  const int before = scan_workgroup(n, tid, part);
  if (tid < E) {
    base[tid] += before;
    if (tid == E - 1) used = before + n;
    if (blockIdx.x == 0) {
      a.offsets[tid] = before;
      if (tid == E - 1) a.offsets[E] = before + n;
    }
  }
  for (int r = 0; r < a.per; ++r) {
    const int run = blockIdx.x * a.per + r;
    __syncthreads();
    if (tid < E) mask[tid] = 0;
    __syncthreads();
    for (int i = tid; i < kRun * a.k; i += kThreads) {
      const int q = i / a.k, t = run * kRun + q;
      if (t >= a.T) break;
      const int e = a.ids[static_cast<int64_t>(t) * a.k + i % a.k];
      if (e >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[e]), 1ull << q);
    }
    __syncthreads();
    scatter(a, run, mask, base, tid);
    __syncthreads();
    if (tid < E) base[tid] += __popcll(mask[tid]);
  }
  const int pairs = a.T * a.k;
  for (int64_t i = used + static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < pairs;
       i += static_cast<int64_t>(a.groups) * kThreads)
    a.rows[i] = -1;
}

int runs_of(int64_t T) { return static_cast<int>((T + kRun - 1) / kRun); }

template <int N>
hipError_t launch(RouteArgs a, hipStream_t st) {
  const int runs = runs_of(a.T);
  if (runs <= 1) {
    a.groups = a.per = 1;
    route_choose_kernel<N, true><<<1, kThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  a.per = (runs + kMaxGroups - 1) / kMaxGroups;
  a.groups = (runs + a.per - 1) / a.per;
  route_choose_kernel<N, false><<<a.groups, kThreads, 0, st>>>(a);
  route_scatter_kernel<N><<<a.groups, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  const int64_t runs = runs_of(T);
  if (runs <= 1) return 0;
  return static_cast<size_t>(runs < kMaxGroups ? runs : kMaxGroups) * E * 4;
}

hipError_t launch_route(const void* logits, lq_dtype dt, int64_t T, int E, int64_t ld,
                        const uint8_t* valid, int k, int renorm, int* ids, float* weight, int* pos,
                        int* rows, int* offsets, void* ws, hipStream_t st) {
  RouteArgs a{};
  a.logits = logits;
  a.dt = dt;
  a.ld = ld;
  a.valid = valid;
  a.T = static_cast<int>(T);
  a.E = E;
  a.k = k;
  a.renorm = renorm;
  a.ids = ids;
  a.weight = weight;
  a.pos = pos;
  a.rows = rows;
  a.offsets = offsets;
  a.counts = static_cast<int*>(ws);
  if (E <= 64) return launch<1>(a, st);
  if (E <= 128) return launch<2>(a, st);
  if (E <= 256) return launch<4>(a, st);
  if (E <= 512) return launch<8>(a, st);
  return launch<16>(a, st);
}

}  // namespace lq
