// C ABI of the 8-bit floating point layers and of the rows sorted by expert
// (declarations in include/lq.h): host-side validation and dispatch.
#include "lq_checks.h"

namespace {

using namespace lq::api;

constexpr int64_t kMostPositions = int64_t{1} << 22, kMostColumns = int64_t{1} << 30;

bool is8(lq_dtype dt) { return dt == LQ_E4M3 || dt == LQ_E5M2; }
bool is16(lq_dtype dt) { return dt == LQ_F16 || dt == LQ_BF16; }
int64_t whole(int64_t K) { return (K + 127) / 128 * 128; }
int64_t blocks(int64_t K) { return (K + 127) / 128; }

// 8-bit rows of K positions and their exponents.
lq_status check_rows8(const char* what, const void* q, int64_t K, int64_t ldq, const void* exps, int64_t lde) {
  if (ldq < whole(K) || lde < blocks(K))
    return fail(LQ_ERR_SHAPE, "%s: pitch %lld < %lld values or %lld < %lld scales", what,
                (long long)ldq, (long long)whole(K), (long long)lde, (long long)blocks(K));
  if (ldq % 16 || lde % 4 || !aligned(q, 16) || !aligned(exps, 4))
    return fail(LQ_ERR_ALIGN, "%s: values and their pitch must be 16-byte aligned, exponents 4-byte",
                what);
  return LQ_OK;
}

lq_status check_quant(const void* x, lq_dtype dtype, int64_t K, int64_t ld) {
  if (K < 1 || K > kMostPositions || ld < K)
    return fail(LQ_ERR_SHAPE, "K=%lld (1..2^22) ld=%lld", (long long)K, (long long)ld);
  if (!aligned(x, dtype_size(dtype))) return fail(LQ_ERR_ALIGN, "misaligned input");
  return LQ_OK;
}

// Outputs over the values that other workgroups still read.
lq_status check_quant_out(const void* x, const void* q, const void* exps) {
  if (!x || !q || !exps) return fail(LQ_ERR_NULL, "null pointer");
  if (q == x || exps == x) return fail(LQ_ERR_UNSUPPORTED, "q or exps overlaps the input");
  return LQ_OK;
}

// ---- the products
struct Plan8 {
  bool few;                    // on the few-row kernel
  bool quantize;               // 16-bit activations by a launch of its own
  lq::F8FewPlan fp;
  lq::F8ManyPlan mp;
  int slices;
  int64_t ldq, lde, ldz;       // of the quantized rows, of the slices' sums
  size_t exps_at, sums_at, bytes;
};

lq_status check_sizes8(int64_t E, int64_t m, int64_t K, lq_dtype a_dtype, int64_t a_rows, int64_t R) {
  if (!is8(a_dtype) && !is16(a_dtype))
    return fail(LQ_ERR_DTYPE, "activations must be LQ_E4M3, LQ_E5M2, LQ_F16 or LQ_BF16");
  if (E < 1 || E > 1024) return fail(LQ_ERR_SHAPE, "E=%lld outside 1..1024", (long long)E);
  if (m < 1 || m > INT32_MAX || K < 1 || K > kMostPositions || a_rows < 0 || a_rows > INT32_MAX ||
      R < 0 || R > INT32_MAX)
    return fail(LQ_ERR_SHAPE, "m=%lld K=%lld (1..2^22) rows=%lld, %lld", (long long)m, (long long)K,
                (long long)a_rows, (long long)R);
  if (a_rows * whole(K) > INT64_C(0xFFFFFFFF))
    return fail(LQ_ERR_SHAPE, "%lld rows of %lld positions exceed the 4 GiB of 8-bit activations of "
                "one call", (long long)a_rows, (long long)K);
  return LQ_OK;
}

// The rows of one matrix, or of a run on average, up to which the few-row kernel is the
// faster one, us there and on tiles.  To float32: 16 (16 x 8192 -> 8192: 25 and 27; 64
// experts, 2048 -> 2816, 16 each: 100 and 112, 24: 135 and 112).  To 16 bits: 11 of a run (8
// each 77 and 85, 12 each 91 and 85; 8 experts, 4096 -> 28672: 181 and 192, 199 and 191), 16 of one
// matrix (16 x 4096 -> 4096: 10.7 and 14, -> 57344: 55 and 54; 24 -> 4096: 15.4 and 13.9), 8 from 8192 positions
// on, where the activations that each block of rows reads again weigh most (16 x 14336 ->
// 4096: 21.3 and 17.6, 16 x 16384 -> 8192: 37 and 28; 6: 31 and 29).
int64_t few_rows(int64_t K, bool grouped, bool precise) {
  return precise ? 16 : grouped ? 11 : blocks(K) >= 64 ? 8 : 16;
}

Plan8 plan8(int64_t E, int64_t m, int64_t K, lq_dtype a_dtype, int64_t a_rows, int64_t R, bool gated,
            bool grouped, bool float_scales, bool precise) {
  Plan8 p{};
  const int64_t runs = grouped ? (E < R ? E : R < 1 ? 1 : R) : 1;
  p.few = R <= few_rows(K, grouped, precise) * runs;
  p.fp = lq::few_f8_plan(E, m, K, R < 1 ? 1 : R, gated, grouped);
  p.mp = lq::many_f8_plan(E, m, K, R < 1 ? 1 : R, gated, grouped, float_scales, precise);
  p.slices = p.few ? p.fp.slices : p.mp.slices;
  p.ldq = whole(K);
  p.lde = (blocks(K) + 3) / 4 * 4;
  p.quantize = is16(a_dtype) && !(p.few && p.fp.held);
  if (p.quantize) {
    p.exps_at = round256(static_cast<size_t>(a_rows * p.ldq));
    p.bytes = p.exps_at + round256(static_cast<size_t>(a_rows * p.lde));
  }
  p.sums_at = p.bytes;
  p.ldz = (m + 3) / 4 * 4;
  if (p.slices > 1) p.bytes += static_cast<size_t>(p.slices) * R * p.ldz * 4;
  return p;
}

// What any call of these sizes needs: gated or not (an odd m has no gated form), scales
// and outputs of either kind.
size_t bytes8(int64_t E, int64_t m, int64_t K, lq_dtype a_dtype, int64_t a_rows, int64_t R, bool grouped) {
  size_t most = 0;
  for (int kind = 0; kind < 8; ++kind) {
    if ((kind & 1) && m % 2) continue;
    const size_t n = plan8(E, m, K, a_dtype, a_rows, R, kind & 1, grouped, kind & 2, kind & 4).bytes;
    if (n > most) most = n;
  }
  return most;
}

lq_status check_product8(const void* w, int64_t m, int64_t K, int64_t ldw, const void* scales,
                         lq_dtype scale_type, int64_t lds, const void* a, lq_dtype a_dtype,
                         int64_t lda, const uint8_t* exps, int64_t lde, int64_t a_rows,
                         const float* bias, lq_act act, int32_t gated, lq_dtype out_dtype) {
  if (scale_type != LQ_E8M0 && scale_type != LQ_F32)
    return fail(LQ_ERR_DTYPE, "scales must be LQ_E8M0 or LQ_F32");
  if (!valid_dtype(out_dtype)) return fail(LQ_ERR_DTYPE, "unknown output dtype");
  if (act < LQ_ACT_NONE || act > LQ_ACT_GELU_TANH)
    return fail(LQ_ERR_UNSUPPORTED, "activation %d", (int)act);
  if (gated && m % 2) return fail(LQ_ERR_SHAPE, "gated rows m=%lld must be even", (long long)m);
  if (ldw < whole(K)) return fail(LQ_ERR_SHAPE, "ldw=%lld < %lld", (long long)ldw, (long long)whole(K));
  if (ldw > INT32_MAX || m * ldw > INT32_MAX)
    return fail(LQ_ERR_SHAPE, "weights of one matrix exceed the 2 GiB per-call limit");
  if (lds < blocks(K)) return fail(LQ_ERR_SHAPE, "lds=%lld < %lld", (long long)lds, (long long)blocks(K));
  if (lds > INT32_MAX || blocks(m) * lds > (int64_t{1} << 29))
    return fail(LQ_ERR_SHAPE, "scales of one matrix exceed the 2^29 per-call limit");
  if (ldw % 16 || !aligned(w, 16)) return fail(LQ_ERR_ALIGN, "w and ldw must be 16-byte aligned");
  if (!aligned(scales, 4) || (scale_type == LQ_E8M0 && lds % 4))
    return fail(LQ_ERR_ALIGN, "scales must be 4-byte aligned, LQ_E8M0 rows whole words");
  if (!aligned(bias, 4)) return fail(LQ_ERR_ALIGN, "misaligned bias");
  if (is8(a_dtype)) {
    if (!exps) return fail(LQ_ERR_NULL, "exps is null");
    const lq_status st = check_rows8("activations", a, K, lda, exps, lde);
    if (st != LQ_OK) return st;
    if (lda > INT64_C(0xFFFFFFFF) || a_rows * lda > INT64_C(0xFFFFFFFF) || lde > lda)
      return fail(LQ_ERR_SHAPE, "8-bit activations exceed the 4 GiB per-call limit (or lde > lda)");
  } else {
    if (lda < K) return fail(LQ_ERR_SHAPE, "lda=%lld < K=%lld", (long long)lda, (long long)K);
    if (!aligned(a, 2)) return fail(LQ_ERR_ALIGN, "misaligned activations");
  }
  return LQ_OK;
}

// The product of a checked call; p lacks only what the plan decides.
hipError_t run8(lq::F8Product& p, const Plan8& plan, const void* a, lq_dtype a_dtype, int64_t lda,
                const uint8_t* exps, int64_t lde, int64_t a_rows, void* workspace, hipStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int type = a_dtype;
  p.a = a;
  p.lda = lda;
  p.exps = exps;
  p.lde = lde;
  p.a_rows = static_cast<int>(a_rows);
  const bool precise = p.out_dt == LQ_F32;
  p.pieces = p.K % 8 == 0 && lda % 8 == 0 && aligned(a, 16);
  if (plan.quantize) {
    const hipError_t e = lq::launch_quant8(a, a_dtype, a_rows, p.K, lda, ws, LQ_E4M3, plan.ldq,
                                           ws + plan.exps_at, plan.lde, st);
    if (e != hipSuccess) return e;
    p.a = ws;
    p.lda = plan.ldq;
    p.exps = ws + plan.exps_at;
    p.lde = plan.lde;
    type = LQ_E4M3;
  }
  p.slices = plan.slices;
  p.slice_steps = plan.few ? plan.fp.slice_steps : plan.mp.slice_steps;
  p.ldz = plan.ldz;
  p.sums = plan.slices > 1 ? reinterpret_cast<float*>(ws + plan.sums_at) : nullptr;
  hipError_t e;
  if (plan.few) {
    e = lq::launch_gemv8(p, type, plan.fp, precise, st);
  } else {
    lq::F8Product q = p;
    if (p.sums) {                          // plain rows, in their own order
      q.act = LQ_ACT_NONE;
      q.gated = 0;
      q.residual = nullptr;
      q.out = p.sums;
      q.ldo = p.ldz;
      q.out_dt = LQ_F32;
    }
    e = lq::launch_gemm8(q, type, plan.mp, precise, st);
  }
  if (e == hipSuccess && p.sums) {
    lq::F6Product q{};                     // what the reduction reads of it
    q.m = p.m;
    q.act = p.act;
    q.gated = p.gated;
    q.residual = p.residual;
    q.ldr = p.ldr;
    q.out = p.out;
    q.ldo = p.ldo;
    q.out_dt = p.out_dt;
    q.R = p.R;
    q.offsets = p.offsets;
    q.E = p.E;
    q.slices = p.slices;
    q.sums = p.sums;
    q.ldz = p.ldz;
    e = lq::launch_f6_reduce(q, st);
  }
  return e;
}

lq::F8Product product8(const void* w, int64_t m, int64_t K, int64_t ldw, const void* scales,
                       lq_dtype scale_type, int64_t lds, const float* bias, int act, int gated,
                       void* out, int out_dt, int64_t ldo, int64_t R) {
  lq::F8Product p{};
  p.w = static_cast<const uint8_t*>(w);
  p.ldw = ldw;
  p.w_matrix = m * ldw;
  p.m = static_cast<int>(m);
  p.K = static_cast<int>(K);
  p.steps = static_cast<int>(blocks(K));
  p.scales = scales;
  p.lds = lds;
  p.scales_matrix = blocks(m) * lds;
  p.float_scales = scale_type == LQ_F32;
  p.bias = bias;
  p.act = act;
  p.gated = gated != 0;
  p.out = out;
  p.out_dt = out_dt;
  p.ldo = ldo;
  p.R = static_cast<int>(R);
  p.E = 1;
  return p;
}

}  // namespace

extern "C" {

lq_status lq_quant8(const void* x, lq_dtype dtype, int64_t rows, int64_t K, int64_t ld, void* q,
                    lq_dtype q_dtype, int64_t ldq, uint8_t* exps, int64_t lde, void* stream) {
  if (!valid_dtype(dtype) || !is8(q_dtype)) return fail(LQ_ERR_DTYPE, "unknown dtype");
  if (rows < 0 || rows > INT32_MAX) return fail(LQ_ERR_SHAPE, "rows=%lld", (long long)rows);
  lq_status st = check_quant(x, dtype, K, ld);
  if (st == LQ_OK) st = check_rows8("outputs", q, K, ldq, exps, lde);
  if (st != LQ_OK) return st;
  if (rows == 0) return ok();
  st = check_quant_out(x, q, exps);
  if (st != LQ_OK) return st;
  return hip_status(lq::launch_quant8(x, dtype, rows, K, ld, static_cast<uint8_t*>(q), q_dtype, ldq,
                                      exps, lde, as_stream(stream)),
                    "lq_quant8 launch");
}

lq_status lq_quant8_blocks(const void* w, lq_dtype dtype, int64_t E, int64_t m, int64_t K,
                           int64_t ld, void* q, int64_t ldq, uint8_t* exps, int64_t lde,
                           void* stream) {
  if (!valid_dtype(dtype)) return fail(LQ_ERR_DTYPE, "unknown dtype");
  if (E < 1 || E > 1024 || m < 1 || m > kMostPositions)
    return fail(LQ_ERR_SHAPE, "E=%lld (1..1024) m=%lld (1..2^22)", (long long)E, (long long)m);
  lq_status st = check_quant(w, dtype, K, ld);
  if (st == LQ_OK) st = check_rows8("outputs", q, K, ldq, exps, lde);
  if (st == LQ_OK) st = check_quant_out(w, q, exps);
  if (st != LQ_OK) return st;
  return hip_status(lq::launch_quant8_blocks(w, dtype, E, m, K, ld, static_cast<uint8_t*>(q), ldq,
                                             exps, lde, as_stream(stream)),
                    "lq_quant8_blocks launch");
}

lq_status lq_gemm8_workspace_size(int64_t m, int64_t K, lq_dtype a_dtype, int64_t B,
                                  size_t* bytes) {
  if (!bytes) return fail(LQ_ERR_NULL, "bytes is null");
  const lq_status st = check_sizes8(1, m, K, a_dtype, B, B);
  if (st != LQ_OK) return st;
  *bytes = bytes8(1, m, K, a_dtype, B, B, false);
  return ok();
}

lq_status lq_gemm8(const void* w, int64_t m, int64_t K, int64_t ldw, const void* scales,
                   lq_dtype scale_type, int64_t lds, const void* a, lq_dtype a_dtype, int64_t lda,
                   const uint8_t* exps, int64_t lde, int64_t B, const float* bias, lq_act act,
                   int32_t gated, const void* residual, int64_t ldr, void* out,
                   lq_dtype out_dtype, int64_t ldo, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!w || !scales || !a || !out) return fail(LQ_ERR_NULL, "null pointer");
  lq_status st = check_sizes8(1, m, K, a_dtype, B, B);
  if (st != LQ_OK) return st;
  if (B < 1) return fail(LQ_ERR_SHAPE, "B=%lld", (long long)B);
  st = check_product8(w, m, K, ldw, scales, scale_type, lds, a, a_dtype, lda, exps, lde, B, bias, act,
                      gated, out_dtype);
  if (st == LQ_OK) st = check_rows_out(residual, ldr, out, out_dtype, ldo, gated ? m / 2 : m, B);
  if (st != LQ_OK) return st;
  const Plan8 plan = plan8(1, m, K, a_dtype, B, B, gated != 0, false, scale_type == LQ_F32,
                           out_dtype == LQ_F32);
  st = check_workspace(workspace, workspace_bytes, plan.bytes);
  if (st == LQ_OK) st = check_overlap(a, residual, ldr, out, ldo, B);
  if (st != LQ_OK) return st;
  lq::F8Product p = product8(w, m, K, ldw, scales, scale_type, lds, bias, act, gated, out, out_dtype, ldo, B);
  p.residual = residual;
  p.ldr = ldr;
  return hip_status(run8(p, plan, a, a_dtype, lda, exps, lde, B, workspace, as_stream(stream)),
                    "lq_gemm8 launch");
}

lq_status lq_gemm8_grouped_workspace_size(int64_t E, int64_t m, int64_t K, lq_dtype a_dtype,
                                          int64_t a_rows, int64_t R, size_t* bytes) {
  if (!bytes) return fail(LQ_ERR_NULL, "bytes is null");
  const lq_status st = check_sizes8(E, m, K, a_dtype, a_rows, R);
  if (st != LQ_OK) return st;
  *bytes = bytes8(E, m, K, a_dtype, a_rows, R, true);
  return ok();
}

lq_status lq_gemm8_grouped(const void* w, int64_t E, int64_t m, int64_t K, int64_t ldw,
                           const void* scales, lq_dtype scale_type, int64_t lds, const void* a,
                           lq_dtype a_dtype, int64_t lda, const uint8_t* exps, int64_t lde,
                           int64_t a_rows, const int32_t* rows, const int32_t* offsets, int64_t R,
                           const float* bias, lq_act act, int32_t gated, void* out,
                           lq_dtype out_dtype, int64_t ldo, void* workspace,
                           size_t workspace_bytes, void* stream) {
  lq_status st = check_sizes8(E, m, K, a_dtype, a_rows, R);
  if (st != LQ_OK) return st;
  if (!rows && a_rows < R)
    return fail(LQ_ERR_SHAPE, "a_rows=%lld < R=%lld without row indices", (long long)a_rows,
                (long long)R);
  if (R == 0) return ok();
  if (a_rows < 1) return fail(LQ_ERR_SHAPE, "a_rows=%lld", (long long)a_rows);
  if (!w || !scales || !a || !out || !offsets) return fail(LQ_ERR_NULL, "null pointer");
  if (!aligned(offsets, 4) || !aligned(rows, 4))
    return fail(LQ_ERR_ALIGN, "misaligned rows or offsets");
  st = check_product8(w, m, K, ldw, scales, scale_type, lds, a, a_dtype, lda, exps, lde, a_rows, bias,
                      act, gated, out_dtype);
  if (st == LQ_OK) st = check_rows_out(nullptr, 0, out, out_dtype, ldo, gated ? m / 2 : m, R);
  if (st != LQ_OK) return st;
  const Plan8 plan = plan8(E, m, K, a_dtype, a_rows, R, gated != 0, true, scale_type == LQ_F32,
                           out_dtype == LQ_F32);
  st = check_workspace(workspace, workspace_bytes, plan.bytes);
  if (st == LQ_OK) st = check_overlap(a, nullptr, 0, out, ldo, R);
  if (st != LQ_OK) return st;
  lq::F8Product p = product8(w, m, K, ldw, scales, scale_type, lds, bias, act, gated, out, out_dtype, ldo, R);
  p.rows = rows;
  p.offsets = offsets;
  p.E = static_cast<int>(E);
  return hip_status(run8(p, plan, a, a_dtype, lda, exps, lde, a_rows, workspace, as_stream(stream)),
                    "lq_gemm8_grouped launch");
}

lq_status lq_sort_rows(const void* x, int32_t size, int64_t T, int64_t n, int64_t ldx,
                       const int32_t* rows, int64_t R, void* out, int64_t ldo, void* stream) {
  if (size != 1 && size != 2 && size != 4) return fail(LQ_ERR_DTYPE, "values of %d bytes", (int)size);
  if (T < 0 || T > INT32_MAX || R < 0 || R > INT32_MAX || n < 1 || n > kMostColumns)
    return fail(LQ_ERR_SHAPE, "T=%lld R=%lld n=%lld (1..2^30)", (long long)T, (long long)R, (long long)n);
  if ((ldx < n && T > 1) || (ldo < n && R > 1))
    return fail(LQ_ERR_SHAPE, "ldx=%lld ldo=%lld < n=%lld", (long long)ldx, (long long)ldo, (long long)n);
  if (R == 0) return ok();
  if (!rows || !out || (T > 0 && !x)) return fail(LQ_ERR_NULL, "null pointer");
  if (!aligned(x, size) || !aligned(out, size) || !aligned(rows, 4))
    return fail(LQ_ERR_ALIGN, "misaligned pointer");
  if (out == x) return fail(LQ_ERR_UNSUPPORTED, "out overlaps x");
  return hip_status(lq::launch_sort_rows(x, size, T, n, ldx, rows, R, out, ldo, as_stream(stream)),
                    "lq_sort_rows launch");
}

lq_status lq_join_rows(const void* z, lq_dtype dtype, int64_t R, int64_t n, int64_t ldz,
                       const int32_t* pos, const float* weight, int64_t T, int32_t k,
                       const void* residual, int64_t ldr, void* out, lq_dtype out_dtype,
                       int64_t ldo, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype)) return fail(LQ_ERR_DTYPE, "unknown dtype");
  lq_status st = join_sizes(T, k);
  if (st != LQ_OK) return st;
  if (R < 0 || R > INT32_MAX || n < 1 || n > kMostColumns || (ldz < n && R > 1))
    return fail(LQ_ERR_SHAPE, "R=%lld n=%lld (1..2^30) ldz=%lld", (long long)R, (long long)n, (long long)ldz);
  if (T == 0) return ok();
  if (!pos || !out || (R > 0 && !z)) return fail(LQ_ERR_NULL, "null pointer");
  if (!aligned(pos, 4) || !aligned(weight, 4) || !aligned(z, dtype_size(dtype)))
    return fail(LQ_ERR_ALIGN, "misaligned pointer");
  st = check_rows_out(residual, ldr, out, out_dtype, ldo, n, T);
  if (st == LQ_OK) st = check_overlap(z, residual, ldr, out, ldo, T);
  if (st != LQ_OK) return st;
  return hip_status(lq::launch_join_rows(z, dtype, R, n, ldz, pos, weight, T, k, residual, ldr, out,
                                         out_dtype, ldo, as_stream(stream)),
                    "lq_join_rows launch");
}

lq_status lq_join_rows_grad(const void* dy, lq_dtype dtype, int64_t ldy, const void* z, int64_t ldz,
                            int64_t R, int64_t n, const int32_t* pos, const float* weight,
                            int64_t T, int32_t k, const int32_t* rows, void* dz, int64_t lddz,
                            float* dweight, void* stream) {
  if (!valid_dtype(dtype)) return fail(LQ_ERR_DTYPE, "unknown dtype");
  const lq_status st = join_sizes(T, k);
  if (st != LQ_OK) return st;
  if (R < 0 || R > INT32_MAX || n < 1 || n > kMostColumns)
    return fail(LQ_ERR_SHAPE, "R=%lld n=%lld (1..2^30)", (long long)R, (long long)n);
  if ((ldy < n && T > 1) || ((ldz < n || lddz < n) && R > 1))
    return fail(LQ_ERR_SHAPE, "ldy=%lld ldz=%lld lddz=%lld < n=%lld", (long long)ldy, (long long)ldz,
                (long long)lddz, (long long)n);
  if (T == 0 && (!rows || R == 0)) return ok();
  if ((T > 0 && (!dy || !pos || !weight || !dweight)) || (R > 0 && (!dz || (T > 0 && !z))))
    return fail(LQ_ERR_NULL, "null pointer");
  const size_t size = dtype_size(dtype);
  if (!aligned(dy, size) || !aligned(z, size) || !aligned(dz, size) || !aligned(pos, 4) ||
      !aligned(weight, 4) || !aligned(rows, 4) || !aligned(dweight, 4))
    return fail(LQ_ERR_ALIGN, "misaligned pointer");
  if (dz && (dz == z || dz == dy)) return fail(LQ_ERR_UNSUPPORTED, "dz overlaps dy or z");
  return hip_status(lq::launch_join_rows_grad(dy, dtype, ldy, z, ldz, R, n, pos, weight, T, k, rows,
                                              dz, lddz, dweight, as_stream(stream)),
                    "lq_join_rows_grad launch");
}

}  // extern "C"
