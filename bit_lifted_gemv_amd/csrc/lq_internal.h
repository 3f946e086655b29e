// Internal declarations shared by the HIP translation units of liblq.
// Kernel launchers return hipError_t from the launch; argument validation
// happens in lq_api.hip before any of them is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lq.h"

namespace lq {

// ---------------------------------------------------------------- dtype helpers
__device__ __forceinline__ float bf16_bits_to_float(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

__device__ __forceinline__ uint16_t float_to_bf16_bits_rne(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return static_cast<uint16_t>(u >> 16);
}

__device__ __forceinline__ float f16_bits_to_float(uint16_t b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return static_cast<float>(h);
}

__device__ __forceinline__ uint16_t float_to_f16_bits_rne(float f) {
  _Float16 h = static_cast<_Float16>(f);   // v_cvt_f16_f32: round to nearest even
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}

// Load element i of a typed 16/32-bit array as float.
template <int DT>
__device__ __forceinline__ float load_as_float(const void* p, int64_t i);

template <>
__device__ __forceinline__ float load_as_float<LQ_F32>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}
template <>
__device__ __forceinline__ float load_as_float<LQ_F16>(const void* p, int64_t i) {
  return f16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}
template <>
__device__ __forceinline__ float load_as_float<LQ_BF16>(const void* p, int64_t i) {
  return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store_from_float(void* p, int64_t i, float v);

template <>
__device__ __forceinline__ void store_from_float<LQ_F32>(void* p, int64_t i, float v) {
  static_cast<float*>(p)[i] = v;
}
template <>
__device__ __forceinline__ void store_from_float<LQ_F16>(void* p, int64_t i, float v) {
  static_cast<uint16_t*>(p)[i] = float_to_f16_bits_rne(v);
}
template <>
__device__ __forceinline__ void store_from_float<LQ_BF16>(void* p, int64_t i, float v) {
  static_cast<uint16_t*>(p)[i] = float_to_bf16_bits_rne(v);
}

// ---------------------------------------------------------------- launchers
hipError_t launch_pack_signs(const int8_t* signs, int64_t rows, int64_t K, int64_t lds,
                             uint32_t* packed, int64_t ldw, hipStream_t st);
hipError_t launch_unpack_signs(const uint32_t* packed, int64_t rows, int64_t K, int64_t ldw,
                               int8_t* signs, int64_t lds, hipStream_t st);
hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t st);

hipError_t launch_lift(const void* a, lq_dtype a_dt, int64_t B, int64_t n, const void* t_inv,
                       lq_dtype t_dt, const float* M, int d, int D, void* out, lq_dtype out_dt,
                       hipStream_t st);

// The matrix-core lift (k_lift_mfma.hip) takes over from 8 tokens (from 4
// when n >= 12288, where T^-1 is large enough for its wider reads to pay)
// when a and T^-1 share a 16-bit type and d divides 128 (d = 4, 8, 16, 32).
bool lift_mfma_applies(lq_dtype a_dt, lq_dtype t_dt, int64_t B, int64_t n, int d, int D);
hipError_t launch_lift_mfma(const void* a, lq_dtype dt, int64_t B, int64_t n, const void* t_inv,
                            const float* M, int d, int D, void* out, lq_dtype out_dt,
                            hipStream_t st);

// Lift with the Kronecker-factored whitening (k_lift_kron.hip).
bool lift_kron_shape_ok(int64_t n, int n1, int d, int D);
// Decode-weights product, one kernel (k_gemm_dec.hip); no workspace.
bool gemm_decoded_shape_ok(int d, int D);
size_t gemm_decoded_workspace_bytes(int64_t m, int64_t n);
hipError_t launch_gemm_decoded(const uint32_t* w, int64_t m, int64_t n, int64_t ldw,
                               const float* M, int d, int D, const float* s, const void* u,
                               int64_t B, float* out, void* ws, hipStream_t st,
                               const char** why);

size_t softmin_workspace_bytes(int64_t N, int d, int D);
hipError_t launch_softmin_grad(const float* W, int64_t N, const float* M, int d, int D, float T,
                               float* loss, float* grad, void* ws, hipStream_t st);
hipError_t launch_adam(float* M, const float* g, float* m1, float* m2, int64_t count, int step,
                       float lr, float b1, float b2, float eps, hipStream_t st);

size_t encode_workspace_bytes(int D);
hipError_t launch_encode(const float* w, int64_t groups, const float* M, const float* A, int d,
                         int D, int8_t* codes, float* err, void* ws, hipStream_t st);

size_t lift_kron_workspace_bytes(int64_t B, int64_t n);
hipError_t launch_lift_kron(const void* a, lq_dtype a_dt, int64_t B, int64_t n, int n1,
                            const float* s1, const float* p1_inv, const float* p2_inv,
                            const float* s2, const float* M, int d, int D, void* out,
                            lq_dtype out_dt, void* ws, hipStream_t st);

// Plain streaming read (k_stream.hip): `groups` workgroups of 1024 threads.
hipError_t launch_stream_read(const void* p, size_t bytes, uint32_t* sink, int groups,
                              hipStream_t st);

// Compute units of the current device (cached per device).
int num_cus();

// One-token GEMV on float16 activation-sum tables (k_gemv1.hip).
size_t gemv1_workspace_bytes(int64_t m, int64_t K);
// One-token layer with the lift in the GEMV's table prologue (k_gemv1.hip).
hipError_t launch_layer_b1(const void* a, lq_dtype dt, const void* t_inv, const float* M, int d,
                           int D, const uint32_t* w, int64_t m, int64_t K, int64_t ldw,
                           const float* s, float* out, void* ws, hipStream_t st);

// GEMV for 6 <= B <= 16 on float4 sign / float8 activation-part matrix
// cores, the three parts as column blocks (k_gemv_f4m.hip).
size_t gemv_f4m_workspace_bytes(int64_t m, int64_t K, int64_t B);
hipError_t launch_gemv_f4m(const uint32_t* w, int64_t m, int64_t K, int64_t ldw, const float* s,
                           const float* a_lift, int64_t B, float* out, void* ws, hipStream_t st);

// The same product on an operand image written by the parts lift (no
// preparation launch; the workspace holds only the split partial sums).
size_t gemv_f4m_parts_workspace_bytes(int64_t m, int64_t K, int64_t B);
hipError_t launch_gemv_f4m_parts(const uint32_t* w, int64_t m, int64_t K, int64_t ldw,
                                 const float* s, const void* parts, int64_t B, float* out,
                                 void* ws, hipStream_t st);

// The lift into that image (k_lift_parts.hip): bytes for K lifted
// positions, and whether the kernel takes the shape.
size_t lift_parts_bytes(int64_t K);
bool lift_parts_applies(lq_dtype a_dt, lq_dtype t_dt, int64_t B, int64_t n, int d, int D);
hipError_t launch_lift_parts(const void* a, lq_dtype dt, int64_t B, int64_t n, const void* t_inv,
                             const float* M, int d, int D, void* image, hipStream_t st);

// Few-token GEMV on float4 sign / float8 activation-part matrix cores
// (k_gemv_f4.hip), 1 <= B <= 5.
size_t gemv_f4_workspace_bytes(int64_t m, int64_t K, int64_t B);
hipError_t launch_gemv_f4(const uint32_t* w, int64_t m, int64_t K, int64_t ldw, const float* s,
                          const float* a_lift, int64_t B, float* out, void* ws, hipStream_t st);

// One-launch GEMV for 1 <= B <= 5 (k_gemv_f4r.hip): each workgroup owns
// whole rows; no workspace.  Applies when its LDS holds the sums.
bool gemv_f4r_applies(int64_t m, int64_t K, int64_t B);
hipError_t launch_gemv_f4r(const uint32_t* w, int64_t m, int64_t K, int64_t ldw, const float* s,
                           const float* a_lift, int64_t B, float* out, hipStream_t st);

hipError_t launch_gemm(const uint32_t* w, int64_t m, int64_t K, int64_t ldw, const float* s,
                       const void* a_lift, lq_dtype dt, int64_t B, float* out, hipStream_t st);

// ---------------------------------------------------------------- float4 x float6 products
// Arguments of the products on float6 parts (f6_parts.h): lq_gemm_ep (one
// matrix, R tokens) and lq_gemm_grouped (E matrices, ragged runs of R rows).
struct F6Product {
  const uint8_t* img;          // parts of the activations
  uint32_t img_row_bytes;
  uint32_t img_bytes;
  int groups;                  // groups per image row (an even number for H = 2)
  const uint32_t* w;           // [E][m][ldw]
  int m, ldw;
  const float* s;              // [E][m]
  const float* bias;           // [E][m] or null
  int act, gated;
  const void* residual;        // [R][ldr] or null
  int64_t ldr;
  void* out;                   // [R][ldo]
  int64_t ldo;
  int out_dt;
  int R;
  const int* offsets;          // [E + 1], or null: one matrix
  int E;
  const int* rows;             // image row of each row, or null: its own
  int src_rows;                // rows of the image (with `rows`, one more of zeros follows)
  int row_tiles, token_tiles;  // set by the launcher
  int block0;                  // its launch's first workgroup
  int slices, slice_units;     // of the positions, in units of 256
  float* sums;                 // [slices][R][ldz] scaled sums of the slices, or null
  int64_t ldz;
};

// The same for at most 16 rows per matrix (k_gemv_f6.hip), which splits its
// activations itself.
struct F6FewPlan {
  int T, kv;                   // 16-row tiles per unit, waves that share a unit
  int groups;                  // groups of 512 positions
  int slices, slice_groups;
  int row_blocks, blocks_per;  // blocks of units, and how many a workgroup takes
  int tok, tiles;              // tokens per tile, tiles (grouped: at most)
  int exchange_at;             // LDS bytes before the exchange
  int64_t ldz;
  size_t sums_bytes;           // of the slices' sums, 0 for one slice
};
F6FewPlan few_f6_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                      bool grouped, bool join);
struct F6Few {
  F6Product p;                 // groups: of 512 positions; no image; sums null: outputs at once
  const void* a;
  int a_dt;
  int64_t lda;
  int K;
  int tok, kv, slice_groups, row_blocks, blocks_per, exchange_at;
  int tile0;                   // the launch's first tile
};
hipError_t launch_gemv_f6(const F6Few& f, const F6FewPlan& plan, int NP, hipStream_t st);

// 16-bit activations -> parts image (k_f6_image.hip); NP = 3, 4 or 5.
hipError_t launch_f6_image(const void* a, lq_dtype dt, int64_t rows, bool zero_row, int64_t K,
                           int64_t lda, int NP, void* img, hipStream_t st);
// Tile shape (its four template digits) and slices of the product for many rows.
struct F6ManyPlan {
  int shape, slices, slice_units;
  int64_t ldz;
  size_t sums_bytes;
};
F6ManyPlan many_f6_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, int NP,
                        bool grouped);
hipError_t launch_gemm_f6(const F6Product& p, int shape, int NP, hipStream_t st);

// The slices' sums added in order, then activation, gate, residual and store
// (k_f6_reduce.hip).
hipError_t launch_f6_reduce(const F6Product& p, hipStream_t st);

// out = residual + sum_j weight z[pos] (k_join.hip), z the sum of `slices`
// arrays [R][ldz]; ldz a multiple of 4.
hipError_t launch_join(const float* z, int slices, int64_t R, int64_t m, int64_t ldz,
                       const int* pos, const float* weight, int64_t T, int k, const void* residual, int64_t ldr,
                       void* out, int64_t ldo, int dt, hipStream_t st);

// Router (k_route.hip), E <= 1024, k <= 32.
size_t route_workspace_bytes(int64_t T, int E);
hipError_t launch_route(const void* logits, lq_dtype dt, int64_t T, int E, int64_t ld,
                        const uint8_t* valid, int k, int renorm, int* ids, float* weight, int* pos,
                        int* rows, int* offsets, void* ws, hipStream_t st);

// ---------------------------------------------------------------- 8-bit floating point
// Quantization (k_quant8.hip); rows of exps are whole words.
hipError_t launch_quant8(const void* x, lq_dtype dt, int64_t n, int64_t K, int64_t ld, uint8_t* q,
                         lq_dtype type, int64_t ldq, uint8_t* exps, int64_t lde, hipStream_t st);
hipError_t launch_quant8_blocks(const void* w, lq_dtype dt, int64_t E, int64_t m, int64_t K,
                                int64_t ld, uint8_t* q, int64_t ldq, uint8_t* exps, int64_t lde,
                                hipStream_t st);

// Arguments of the 8-bit products: lq_gemm8 (one matrix, R tokens) and
// lq_gemm8_grouped (E matrices, ragged runs of R rows).
struct F8Product {
  const uint8_t* w;            // [E][m][ldw], K up to whole 128
  int64_t ldw, w_matrix;       // bytes of a row and of a matrix
  int m, K, steps;             // steps: blocks of 128 positions
  const void* scales;          // [E][strips of 128 rows][lds], exponents or float32
  int64_t lds, scales_matrix;
  int float_scales;
  const void* a;               // [a_rows][lda], 8-bit (K up to whole 128) or 16-bit
  int64_t lda;
  int pieces;                  // 16-bit rows are whole 16-byte pieces
  const uint8_t* exps;         // [a_rows][lde], of 8-bit activations
  int64_t lde;
  int a_rows;
  const int* rows;             // row of `a` of each row, or null: its own
  const int* offsets;          // [E + 1], or null: one matrix
  int E, R;
  const float* bias;           // [E][m] or null
  int act, gated;
  const void* residual;        // [R][ldr] or null
  int64_t ldr;
  void* out;                   // [R][ldo]
  int64_t ldo;
  int out_dt;
  float* sums;                 // [slices][R][ldz] sums of the slices, or null: outputs
  int64_t ldz;
  int slices, slice_steps;     // of the positions
  int row_blocks, token_tiles, block0;      // set by the launcher
};
// Few rows per matrix (k_gemv8.hip).
struct F8FewPlan {
  int wf, waves;               // 16 wf rows and 16 tokens per workgroup of `waves`
  int slices, slice_steps;
  int held;                    // activations in LDS, 16-bit ones quantized on the way
  int64_t held_bytes;
};
F8FewPlan few_f8_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, bool grouped);
hipError_t launch_gemv8(const F8Product& p, int a_type, const F8FewPlan& plan, bool precise,
                        hipStream_t st);
// Many (k_gemm8.hip), 8-bit activations.  precise: float32 results.
enum F8Shape { kSquare, kTall, kPair, kOne };   // tiles, see many_f8_plan
struct F8ManyPlan {
  int shape;
  int slices, slice_steps;
};
F8ManyPlan many_f8_plan(int64_t E, int64_t m, int64_t K, int64_t R, bool gated, bool grouped,
                        bool float_scales, bool precise);
hipError_t launch_gemm8(const F8Product& p, int a_type, const F8ManyPlan& plan, bool precise,
                        hipStream_t st);

// Rows sorted by expert and back (k_rows.hip).
hipError_t launch_sort_rows(const void* x, int size, int64_t T, int64_t n, int64_t ldx,
                            const int* rows, int64_t R, void* out, int64_t ldo, hipStream_t st);
hipError_t launch_join_rows(const void* z, lq_dtype dt, int64_t R, int64_t n, int64_t ldz,
                            const int* pos, const float* weight, int64_t T, int k,
                            const void* residual, int64_t ldr, void* out, lq_dtype out_dt,
                            int64_t ldo, hipStream_t st);
hipError_t launch_join_rows_grad(const void* dy, lq_dtype dt, int64_t ldy, const void* z, int64_t ldz,
                                 int64_t R, int64_t n, const int* pos, const float* weight, int64_t T,
                                 int k, const int* rows, void* dz, int64_t lddz, float* dweight,
                                 hipStream_t st);

}  // namespace lq
