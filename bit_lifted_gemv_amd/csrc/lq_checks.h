// Status codes, messages and the argument checks that the C entry points
// (lq_api.hip, lq_api8.hip) share.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "lq_internal.h"

namespace lq {
namespace api {

inline thread_local char g_err[512] = "";

inline lq_status fail(lq_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

inline lq_status ok() {
  g_err[0] = '\0';
  return LQ_OK;
}

inline lq_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(LQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool valid_dtype(lq_dtype dt) { return dt == LQ_F32 || dt == LQ_F16 || dt == LQ_BF16; }

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

inline size_t dtype_size(lq_dtype dt) { return dt == LQ_F32 ? 4 : 2; }

inline lq_status check_rows_out(const void* residual, int64_t ldr, const void* out, lq_dtype out_dtype,
                                int64_t ldo, int64_t width, int64_t rows) {
  if (ldo < width && rows > 1)
    return fail(LQ_ERR_SHAPE, "ldo=%lld < %lld outputs", (long long)ldo, (long long)width);
  if (residual && ldr < width && rows > 1)
    return fail(LQ_ERR_SHAPE, "ldr=%lld < %lld outputs", (long long)ldr, (long long)width);
  if (!aligned(out, dtype_size(out_dtype)) || !aligned(residual, dtype_size(out_dtype)))
    return fail(LQ_ERR_ALIGN, "misaligned out or residual");
  return LQ_OK;
}

// Outputs over what other workgroups still read.  (Rows that interleave with the
// inputs' in one buffer are fine, so only the same start is looked at.)
inline lq_status check_overlap(const void* in, const void* residual, int64_t ldr, const void* out,
                     int64_t ldo, int64_t rows) {
  if (out == in) return fail(LQ_ERR_UNSUPPORTED, "out overlaps the inputs");
  if (out == residual && ldr != ldo && rows > 1)
    return fail(LQ_ERR_UNSUPPORTED, "residual is out with another pitch");
  return LQ_OK;
}

inline lq_status check_workspace(const void* workspace, size_t have, size_t need) {
  if (need == 0) return LQ_OK;
  if (!workspace) return fail(LQ_ERR_WORKSPACE, "workspace of %zu bytes required", need);
  if (have < need) return fail(LQ_ERR_WORKSPACE, "workspace %zu bytes < %zu required", have, need);
  if (!aligned(workspace, 256)) return fail(LQ_ERR_ALIGN, "workspace must be 256-byte aligned");
  return LQ_OK;
}

inline lq_status join_sizes(int64_t T, int32_t k) {
  if (T < 0 || T > INT32_MAX || k < 1 || k > 32 || T * k > INT32_MAX)
    return fail(LQ_ERR_SHAPE, "T=%lld k=%d (k in 1..32)", (long long)T, (int)k);
  return LQ_OK;
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace api
}  // namespace lq
