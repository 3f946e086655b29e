// Router of a mixture-of-experts layer: per token the k largest of E logits
// (ties to the lowest expert), their softmax weights, and the stable order
// of the (token, choice) pairs by expert, as offsets, rows and positions.
//
// Two launches (one when a single workgroup holds every token).  A workgroup
// of 16 waves takes runs of 64 tokens.  Up to 256 experts a token has 16
// lanes with up to 16 logits each (a wave four tokens, their minima taken by
// rotations within a row of lanes); beyond, a wave of 64 lanes each.  16-bit
// logits are held as one integer, inverted order-preserving bits above the
// expert, so that one minimum gives value and lowest expert at once; float32
// logits take a second one for the expert.  (One token per wave and two
// maxima for every type cost 22 us for 16384 x 256 bfloat16, k = 8.)
// A token chooses an expert at most once, so a run's choices are one 64-bit
// mask of tokens per expert in LDS: counts and stable ranks are popcounts of
// it, whatever order the waves set the bits in.  The first launch writes the
// choices and each workgroup's counts per expert; the second adds the counts
// before its own (about 256 workgroups) and scatters.  It reads every
// workgroup's counts, so these are 8 bits where a workgroup has few tokens
// (both launches, 16384 x 256: 17.8 us, 18.4 us with 16 bits throughout).
// Bound by launch latency (24 x 64: 5.3 us); the logits are read once.
#include "lq_internal.h"

namespace lq {
namespace {

constexpr int kRun = 64;                 // tokens per mask
constexpr int kThreads = 1024;
constexpr int kGroups = 256;             // workgroups, unless that makes kMaxPer runs each
constexpr int kMaxPer = 1023;            // counts are 16 bits: 64 kMaxPer < 2^16,
constexpr int kNarrowPer = 3;            // or 8, up to this many runs: 64 kNarrowPer < 2^8

// Keys: inverted order-preserving bits, so that the largest logit has the
// smallest key; kNone, behind every logit's, for what is never chosen (NaN,
// -inf).  -0 and +0 are equal logits: both take the key of +0.  Selects and
// bit operations only: written with branches, each of a lane's logits cost
// its own load, wait and jumps.
constexpr uint32_t kNone = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t key_of(uint32_t u) {       // a float's bits
  u = u == 0x80000000u ? 0u : u;
  const uint32_t sign = static_cast<uint32_t>(static_cast<int32_t>(u) >> 31);
  const uint32_t k = ~(u ^ (sign | 0x80000000u));
  const bool none = static_cast<int>((u & 0x7FFFFFFFu) > 0x7F800000u) | static_cast<int>(u == 0xFF800000u);
  return none ? kNone : k;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  const uint32_t b = ~key;
  return __uint_as_float(b ^ (b & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}
// The same for the 16 bits of a float16 or bfloat16, with the expert in the
// lower half: one minimum gives value and lowest expert.
__device__ __forceinline__ uint32_t key_of16(uint32_t u, uint32_t inf, uint32_t expert) {
  u = u == 0x8000u ? 0u : u;
  const uint32_t sign = (u >> 15) * 0xFFFFu;
  const uint32_t k = (~(u ^ (sign | 0x8000u)) << 16) | expert;
  const bool none = static_cast<int>((u & 0x7FFFu) > inf) | static_cast<int>(u == (inf | 0x8000u));
  return none ? kNone : k;
}
__device__ __forceinline__ float value_of16(uint32_t key, bool bf16) {
  const uint32_t b = ~key >> 16;
  const uint16_t u = static_cast<uint16_t>(b ^ (b & 0x8000u ? 0x8000u : 0xFFFFu));
  return bf16 ? bf16_bits_to_float(u) : f16_bits_to_float(u);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t moved(uint32_t keep, uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      static_cast<int>(keep), static_cast<int>(v), CTRL, ROW_MASK, 0xF, false));
}

// Smallest value over a token's L lanes, in all of them.
template <int L>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  v = min(v, moved<0x128, 0xF>(v, v));   // row_ror 8, 4, 2, 1
  v = min(v, moved<0x124, 0xF>(v, v));
  v = min(v, moved<0x122, 0xF>(v, v));
  v = min(v, moved<0x121, 0xF>(v, v));
  if (L == 64) {
    v = min(v, moved<0x142, 0xA>(v, v)); // row_bcast 15, 31
    v = min(v, moved<0x143, 0xC>(v, v));
    v = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
  }
  return v;
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {   // fixed order
#pragma unroll
  for (int d = L / 2; d; d /= 2) v += __shfl_xor(v, d);
  return v;
}

struct RouteArgs {
  const void* logits;
  int dt;
  int64_t ld;
  const uint8_t* valid;
  int T, E, k, renorm;
  int wide;                              // rows of logits allow 16-byte loads
  int* ids;
  float* weight;
  int* pos;
  int* rows;
  int* offsets;
  uint32_t* counts;                      // [groups][counts_pitch] words of 4 or 2 counts
  int counts_pitch;
  int narrow;                            // counts of 8 bits
  int groups, per;                       // workgroups, runs of 64 tokens per workgroup
};

// The choices of one token by L lanes of N logits each: lane l gets choices
// l and l + L (id -1: none).  DT is the logits' type.
template <int L, int N, int DT>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, bool live, int lane,
                                       int (&id)[2], float (&weight)[2]) {
  constexpr bool kPacked = DT != LQ_F32;
  constexpr int kVec = DT == LQ_F32 ? 4 : 8;           // logits of a 16-byte load
  const int E = a.E;
  const uint32_t inf = DT == LQ_F16 ? 0x7C00u : 0x7F80u;
  uint32_t b[N];
  // expert of logit j of this lane
  const bool wide = N >= kVec && a.wide;
  auto expert = [&](int j) {
    return wide ? (j / kVec * L + lane) * kVec + j % kVec : j * L + lane;
  };
  const int64_t at = static_cast<int64_t>(t) * a.ld;
  if (wide) {                                          // E is a multiple of kVec then
    uint4 q[(N + kVec - 1) / kVec];
#pragma unroll
    for (int v = 0; v < N / kVec; ++v) {
      const int64_t from = at + min((v * L + lane) * kVec, E - kVec);
      q[v] = kPacked ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.logits) + from)
                     : *reinterpret_cast<const uint4*>(static_cast<const float*>(a.logits) + from);
    }
#pragma unroll
    for (int v = 0; v < N / kVec; ++v) {
      const uint32_t w[4] = {q[v].x, q[v].y, q[v].z, q[v].w};
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        b[(v * kVec + c) % N] = kPacked ? w[c / 2] >> (16 * (c % 2)) & 0xFFFFu : w[c % 4];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t from = at + min(j * L + lane, E - 1);
      b[j] = kPacked ? static_cast<const uint16_t*>(a.logits)[from]
                     : static_cast<const uint32_t*>(a.logits)[from];
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = expert(j);
    const uint32_t k = kPacked ? key_of16(b[j], inf, static_cast<uint32_t>(e)) : key_of(b[j]);
    b[j] = static_cast<int>(e < E) & static_cast<int>(live) ? k : kNone;
  }
  auto value = [&](uint32_t key) {
    return kPacked ? value_of16(key, DT == LQ_BF16) : value_of(key);
  };
  float all = 0.f;                                     // renorm == 0: softmax over every expert
  if (!a.renorm) {
    uint32_t first = kNone;
#pragma unroll
    for (int j = 0; j < N; ++j) first = min(first, b[j]);
    const float top = value(lanes_min<L>(first));
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (b[j] != kNone) {
        const float y = value(b[j]);
        all += y == top ? 1.f : expf(y - top);         // +inf logits share the whole weight
      }
    all = lanes_sum<L>(all);
  }
  // k times the smallest key (the largest logit).  Packed keys differ, so
  // subtracting the smallest and one wraps that one past every other, and
  // `passed` is what was subtracted so far.
  int valid = 0;
  if (kPacked) {
#pragma unroll
    for (int j = 0; j < N; ++j) valid += b[j] != kNone;
#pragma unroll
    for (int d = L / 2; d; d /= 2) valid += __shfl_xor(valid, d);
  }
  uint32_t key[2] = {kNone, kNone}, top_key = kNone, passed = 0;
  for (int i = 0; i < a.k; ++i) {
    uint32_t best = b[0];
#pragma unroll
    for (int j = 1; j < N; ++j) best = min(best, b[j]);
    const uint32_t least = lanes_min<L>(best);
    uint32_t k0;
    int e;
    if (kPacked) {
      k0 = i < valid ? least + passed : kNone;
      e = static_cast<int>(k0 & 0xFFFFu);
#pragma unroll
      for (int j = 0; j < N; ++j) b[j] -= least + 1;
      passed += least + 1;
    } else {
      uint32_t low = kNone;                            // the lowest expert with it
#pragma unroll
      for (int j = 0; j < N; ++j)
        low = b[j] == least ? min(low, static_cast<uint32_t>(expert(j))) : low;
      e = static_cast<int>(lanes_min<L>(low));
      k0 = least;
#pragma unroll
      for (int j = 0; j < N; ++j) b[j] = expert(j) == e ? kNone : b[j];
    }
    if (i == 0) top_key = k0;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (i == lane + c * L) {
        id[c] = e;
        key[c] = k0;
      }
  }
  const float top = value(top_key);
  float p[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float v = value(key[c]);
    p[c] = key[c] == kNone ? 0.f : v == top ? 1.f : expf(v - top);
  }
  const float total = a.renorm ? lanes_sum<L>(p[0] + p[1]) : all;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    weight[c] = key[c] == kNone ? 0.f : p[c] / total;
    if (key[c] == kNone) id[c] = -1;
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

template <int L, int N, int DT, bool ONE>
__global__ void __launch_bounds__(kThreads) route_choose_kernel(RouteArgs a) {
  __shared__ uint64_t mask[L * N];
  __shared__ int total[L * N];
  __shared__ int part[16];
  const int tid = threadIdx.x, lane = tid % L;
  const int E = a.E, k = a.k;
  if (tid < E) total[tid] = 0;
  int id[2] = {-1, -1};
  float weight[2];
  for (int r = 0; r < a.per; ++r) {
    const int run = blockIdx.x * a.per + r;
    // past the last run: its tokens' numbers may lie past 2^31
    if (run > 0 && run > (a.T - 1) / kRun) break;
    if (tid < E) mask[tid] = 0;
    __syncthreads();
    for (int q = tid / L; q < kRun; q += kThreads / L) {
      const int t = run * kRun + q;
      if (t >= a.T) break;
      choose<L, N, DT>(a, t, !a.valid || a.valid[t], lane, id, weight);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int i = lane + c * L;
        if (i < k) {
          a.ids[static_cast<int64_t>(t) * k + i] = id[c];
          a.weight[static_cast<int64_t>(t) * k + i] = weight[c];
          if (id[c] >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[id[c]]), 1ull << q);
        }
      }
    }
    __syncthreads();
    if (tid < E) total[tid] += __popcll(mask[tid]);
  }
  if (!ONE) {
    __syncthreads();
    const int per_word = a.narrow ? 4 : 2;
    if (tid < a.counts_pitch) {
      uint32_t w = 0;
      for (int c = 0; c < per_word; ++c) {
        const int e = tid * per_word + c;
        if (e < E) w |= static_cast<uint32_t>(total[e]) << (32 / per_word * c);
      }
      a.counts[static_cast<int64_t>(blockIdx.x) * a.counts_pitch + tid] = w;
    }
    return;
  }
  const int n = tid < E ? total[tid] : 0;
  const int before = scan_workgroup(n, tid, part);
  __shared__ int used;
  if (tid < E) {
    total[tid] = before;
    a.offsets[tid] = before;
    if (tid == E - 1) a.offsets[E] = used = before + n;
  }
  __syncthreads();
  if (L == 16) {
    // every token's choices are still in its lanes
    const int t = tid / L;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = lane + c * L;
      if (t < a.T && i < k) {
        int p = -1;
        if (id[c] >= 0) {
          p = total[id[c]] + __popcll(mask[id[c]] & ((uint64_t{1} << t) - 1));
          a.rows[p] = t;
        }
        a.pos[t * k + i] = p;
      }
    }
  } else {
    for (int at = tid; at < a.T * k; at += kThreads) {
      const int t = at / k, e = a.ids[at];
      int p = -1;
      if (e >= 0) {
        p = total[e] + __popcll(mask[e] & ((uint64_t{1} << t) - 1));
        a.rows[p] = t;
      }
      a.pos[at] = p;
    }
  }
  for (int i = used + tid; i < a.T * k; i += kThreads) a.rows[i] = -1;
}

template <int EMAX>
__global__ void __launch_bounds__(kThreads) route_scatter_kernel(RouteArgs a) {
  __shared__ uint64_t mask[EMAX];
  __shared__ int base[EMAX], all[EMAX];
  __shared__ int part[16];
  __shared__ int used;
  const int tid = threadIdx.x;
  const int E = a.E, k = a.k;
  for (int e = tid; e < EMAX; e += kThreads) base[e] = all[e] = 0;
  // the first run's choices, on their way while the counts are added
  int first[2] = {-1, -1};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int i = tid + c * kThreads;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * a.per * kRun * k + i;
    if (i < kRun * k && at < static_cast<int64_t>(a.T) * k) first[c] = a.ids[at];
  }
  __syncthreads();
  {
    // thread (q, e): word e of every lanes-th workgroup's counts, its fields
    // added two at a time in 16 or all in 32 bits (a thread adds at most 64
    // words of 8-bit counts: 64 x 192 < 2^16); integer sums, so the order of the
    // additions does not matter
    const int words = a.counts_pitch, lanes = kThreads / words;
    const int q = tid / words, e = tid % words;
    if (q < lanes) {
      uint32_t sum[4] = {0, 0, 0, 0}, mine[4] = {0, 0, 0, 0};
      for (int g0 = q; g0 < a.groups; g0 += 16 * lanes) {
        uint32_t c[16];                                // sixteen loads on their way at once
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int g = min(g0 + x * lanes, a.groups - 1);
          c[x] = a.counts[static_cast<int64_t>(g) * words + e];
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int g = g0 + x * lanes;
          if (g >= a.groups) c[x] = 0;
          const uint32_t before = g < static_cast<int>(blockIdx.x) ? c[x] : 0u;
          if (a.narrow) {
            sum[0] += c[x] & 0x00FF00FFu;
            sum[1] += c[x] >> 8 & 0x00FF00FFu;
            mine[0] += before & 0x00FF00FFu;
            mine[1] += before >> 8 & 0x00FF00FFu;
          } else {
            sum[0] += c[x] & 0xFFFFu;
            sum[1] += c[x] >> 16;
            mine[0] += before & 0xFFFFu;
            mine[1] += before >> 16;
          }
        }
      }
      if (a.narrow) {                                  // fields 0, 2 and 1, 3 apart
#pragma unroll
        for (int c = 1; c >= 0; --c) {
          sum[c + 2] = sum[c] >> 16;
          sum[c] &= 0xFFFFu;
          mine[c + 2] = mine[c] >> 16;
          mine[c] &= 0xFFFFu;
        }
      }
      const int fields = a.narrow ? 4 : 2;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < fields && fields * e + c < E) {
          atomicAdd(&base[fields * e + c], static_cast<int>(mine[c]));
          atomicAdd(&all[fields * e + c], static_cast<int>(sum[c]));
        }
    }
  }
  __syncthreads();
  const int n = tid < E ? all[tid] : 0;
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
    const int64_t at0 = static_cast<int64_t>(run) * kRun * k;
    const int pairs = static_cast<int>(min(static_cast<int64_t>(kRun) * k,
                                           max(static_cast<int64_t>(a.T) * k - at0, int64_t{0})));
    int e[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = tid + c * kThreads;
      e[c] = r == 0 ? first[c] : i < pairs ? a.ids[at0 + i] : -1;
      if (e[c] >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[e[c]]), 1ull << (i / k));
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int i = tid + c * kThreads, q = i / k;
      if (i >= pairs) continue;
      int p = -1;
      if (e[c] >= 0) {
        p = base[e[c]] + __popcll(mask[e[c]] & ((uint64_t{1} << q) - 1));
        a.rows[p] = run * kRun + q;
      }
      a.pos[at0 + i] = p;
    }
    __syncthreads();
    if (tid < E) base[tid] += __popcll(mask[tid]);
  }
  const int64_t pairs = static_cast<int64_t>(a.T) * k;
  for (int64_t i = used + static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < pairs;
       i += static_cast<int64_t>(a.groups) * kThreads)
    a.rows[i] = -1;
}

int64_t runs_of(int64_t T) { return (T + kRun - 1) / kRun; }
int per_of(int64_t T) {
  const int64_t per = (runs_of(T) + kGroups - 1) / kGroups;
  return static_cast<int>(per < kMaxPer ? per : kMaxPer);
}
int groups_of(int64_t T) { return static_cast<int>((runs_of(T) + per_of(T) - 1) / per_of(T)); }
bool narrow_of(int64_t T) { return per_of(T) <= kNarrowPer; }
int pitch_of(int64_t T, int E) { return narrow_of(T) ? (E + 3) / 4 : (E + 1) / 2; }

template <int L, int N, int DT>
hipError_t launch(RouteArgs a, hipStream_t st) {
  if (runs_of(a.T) <= 1) {
    a.groups = a.per = 1;
    route_choose_kernel<L, N, DT, true><<<1, kThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  a.per = per_of(a.T);
  a.groups = groups_of(a.T);
  route_choose_kernel<L, N, DT, false><<<a.groups, kThreads, 0, st>>>(a);
  if (a.E <= 256) route_scatter_kernel<256><<<a.groups, kThreads, 0, st>>>(a);
  else route_scatter_kernel<1024><<<a.groups, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t by_experts(const RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) return launch<16, 4, DT>(a, st);
  if (a.E <= 128) return launch<16, 8, DT>(a, st);
  if (a.E <= 256) return launch<16, 16, DT>(a, st);
  return launch<64, 16, DT>(a, st);
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int E) {
  if (runs_of(T) <= 1) return 0;
  return static_cast<size_t>(groups_of(T)) * pitch_of(T, E) * 4;
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
  const int vec = dt == LQ_F32 ? 4 : 8;
  a.wide = E % vec == 0 && ld % vec == 0 && reinterpret_cast<uint64_t>(logits) % 16 == 0;
  a.ids = ids;
  a.weight = weight;
  a.pos = pos;
  a.rows = rows;
  a.offsets = offsets;
  a.counts = static_cast<uint32_t*>(ws);
  a.counts_pitch = pitch_of(T, E);
  a.narrow = narrow_of(T);
  if (dt == LQ_F32) return by_experts<LQ_F32>(a, st);
  return dt == LQ_F16 ? by_experts<LQ_F16>(a, st) : by_experts<LQ_BF16>(a, st);
}

}  // namespace lq
