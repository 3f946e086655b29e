/*
 * lq.h -- C ABI of the LiftQuant lift-then-project linear layer on MI355X.
 *
 * The layer (LiftQuant notes, "LiftQuant: Continuous Bit-Width LLM via
 * Dimensional Lifting and Projection", section 关键设计 4 and the 推理 node of
 * the 整体框架 flowchart) is
 *
 *     o = diag(s) . W_q . lift(T^-1 a)
 *
 *   * W_q in {+-1}^(m x K) holds one sign per bit (关键设计 1: a d-wide weight
 *     group is w = M y with y in {+-1}^D, so K = n*D/d and the bit-width is D/d);
 *   * T^-1 is a per-layer transform, here block-diagonal with square blocks;
 *   * lift applies M^T (M is d x D) to every d-wide group of u = T^-1 a:
 *     a_hat[g*D + j] = sum_r M[r][j] u[g*d + r].  Since y.(M^T u_g) = (M y).u_g
 *     this equals the product with the reconstructed weights;
 *   * s is a per-output-row scale (the notes write diag(s) and nothing more).
 * The notes split the run-time work into one small transform of the
 * activations and then the product of the 1-bit weights with the result
 * (关键设计 4); the calls below are those two steps.
 *
 * Conventions (all calls):
 *   - Every pointer except host-side size outputs is a DEVICE pointer owned by
 *     the caller.  The library keeps no buffers of its own.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  A
 *     call validates its arguments on the host, enqueues its kernels on
 *     `stream` and returns without synchronising.
 *   - On any validation failure the call returns a nonzero lq_status, sets a
 *     thread-local message (lq_last_error) and launches nothing.  A failed
 *     launch returns LQ_ERR_HIP.
 *   - Outputs must not alias inputs.  All arrays are row-major and dense in
 *     their last dimension; leading dimensions are given where they may differ.
 *   - Calls are thread-safe; calls that share a workspace must not overlap.
 */
#ifndef LQ_H_
#define LQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t lq_status;
#define LQ_OK              0
#define LQ_ERR_NULL        1  /* a required pointer is NULL                        */
#define LQ_ERR_SHAPE       2  /* sizes inconsistent or out of range                */
#define LQ_ERR_DTYPE       3  /* unsupported element type for this argument        */
#define LQ_ERR_ALIGN       4  /* a pointer or leading dimension is misaligned      */
#define LQ_ERR_UNSUPPORTED 5  /* valid request this build does not implement        */
#define LQ_ERR_HIP         6  /* the HIP runtime reported an error                  */
#define LQ_ERR_WORKSPACE   7  /* workspace missing or too small                     */

typedef int32_t lq_dtype;
#define LQ_F32  0
#define LQ_F16  1
#define LQ_BF16 2
/* Types of lq_quant8 and the 8-bit products alone (OCP 8-bit floating point). */
#define LQ_E4M3 3  /* 4 exponent bits, 3 of fraction, largest 448, no infinity  */
#define LQ_E5M2 4  /* 5 exponent bits, 2 of fraction, largest 57344             */
#define LQ_E8M0 5  /* of scales: a byte b, the scale 2^(b - 127); 255 is a NaN  */

/* Activations of the products with an epilogue (lq_gemm_ep, lq_gemm_grouped). */
typedef int32_t lq_act;
#define LQ_ACT_NONE      0  /* z                                                   */
#define LQ_ACT_RELU      1  /* max(z, 0)                                           */
#define LQ_ACT_SILU      2  /* z / (1 + exp(-z))                                   */
#define LQ_ACT_GELU      3  /* z (1 + erf(z / sqrt 2)) / 2                         */
#define LQ_ACT_GELU_TANH 4  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2   */

/* Human-readable name of a status code (static string). */
const char* lq_status_string(lq_status st);
/* Message of the last failed call on this thread ("" if none). */
const char* lq_last_error(void);
/* Library version string. */
const char* lq_version(void);

/*
 * lq_pack_signs -- pack signs into W_q words.
 * Storage of W_q (关键设计 1: one bit per lifted sign, D signs per d weights):
 *   packed: uint32 [rows][ldw]; lifted position k of a row is bit (k & 31) of
 *   word (k >> 5); the bit is 1 iff signs[row][k] > 0 (0 and negatives pack as
 *   0, i.e. -1).  Bits at positions >= K and words >= ceil(K/32) are written 0.
 * signs:  int8 [rows][lds], lds >= K.
 * Requires rows >= 0, K >= 0, ldw >= ceil(K/32), lds >= K; rows == 0 or
 * K == 0 with ldw == 0 is a no-op.
 */
lq_status lq_pack_signs(const int8_t* signs, int64_t rows, int64_t K, int64_t lds,
                        uint32_t* packed, int64_t ldw, void* stream);

/*
 * lq_unpack_signs -- inverse of lq_pack_signs: signs[row][k] = +1 if the bit
 * is 1 else -1, for k < K (columns K..lds-1 are not written).
 */
lq_status lq_unpack_signs(const uint32_t* packed, int64_t rows, int64_t K, int64_t ldw,
                          int8_t* signs, int64_t lds, void* stream);

/*
 * lq_lift_activations -- the small transform of the activations
 * (关键设计 4, T* a, with T* read as T^-1 followed by M^T per group).
 *   u[b][tb*q + r] = sum_c T_q[r][c] * a[b][tb*q + c]      (block q of T^-1)
 *   a_lift[b][g*D + j] = sum_{r<d} M[r][j] * u[b][g*d + r]
 * a:      [B][n] of a_dtype (LQ_F16 | LQ_BF16 | LQ_F32)
 * t_inv:  [n/t_block][t_block][t_block] of t_dtype (LQ_F16 | LQ_BF16 | LQ_F32)
 * M:      float [d][D]
 * a_lift: [B][K] of lift_dtype, K = n*D/d.  LQ_F32 feeds lq_gemv; LQ_F16 or
 *         LQ_BF16 (round to nearest even) feed lq_gemm.
 * Accumulation is float32.  Requires t_block == 128, n % 128 == 0,
 * n % d == 0, 1 <= d <= 64, 1 <= D <= 256, d*D <= 8192, B >= 1; a and t_inv
 * 16-byte aligned (16-byte loads), M and a_lift aligned to their element.
 */
lq_status lq_lift_activations(const void* a, lq_dtype a_dtype, int64_t B, int64_t n,
                              const void* t_inv, lq_dtype t_dtype, int32_t t_block,
                              const float* M, int32_t d, int32_t D,
                              void* a_lift, lq_dtype lift_dtype, void* stream);

/*
 * lq_lift_kron -- the lift with the Kronecker-factored whitening of
 * 关键设计 3, T = diag(s1) (P1 (x) P2) diag(s2) with P1 n1 x n1, P2 n2 x n2,
 * n = n1 n2 and s2 constant over each d-wide lift group (so that it folds
 * into M):
 *   u      = diag(1/s2) (P1^-1 (x) P2^-1) diag(1/s1) a
 *   a_lift = (I (x) M^T) u,  a_lift[b][g*D + j] = sum_{r<d} M[r][j] u[b][g*d + r]
 * Channel c = i*n2 + j of a token is entry (i, j) of its n1 x n2 reshape.
 * a:        [B][n] of a_dtype (LQ_F16 | LQ_BF16 | LQ_F32).
 * s1:       float [n];  s2: float [n/d] (one scale per group).
 * p1_inv:   float [n1][n1] (P1^-1);  p2_inv: float [n2][n2] (P2^-1).
 * M:        float [d][D].
 * a_lift:   [B][K] of lift_dtype, K = n*D/d.
 * workspace: device buffer of >= lq_lift_kron_workspace_size bytes (the
 *           intermediate n1 x n2 products, float32), 256-byte aligned,
 *           caller-owned, no initialisation needed.
 * Requires 1 <= B <= 65535, n % n1 == 0, n2 = n/n1 <= 128, n1 <= 256,
 * n2 % d == 0, 1 <= d <= 64, 1 <= D <= 256, d*D <= 8192 (else LQ_ERR_SHAPE or
 * LQ_ERR_UNSUPPORTED, nothing launched).  float32 arithmetic throughout.
 */
lq_status lq_lift_kron_workspace_size(int64_t B, int64_t n, size_t* bytes);
lq_status lq_lift_kron(const void* a, lq_dtype a_dtype, int64_t B, int64_t n, int32_t n1,
                       const float* s1, const float* p1_inv, const float* p2_inv,
                       const float* s2, const float* M, int32_t d, int32_t D, void* a_lift,
                       lq_dtype lift_dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * lq_encode -- quantise weight groups to lattice codes: for each d-wide group
 * w, the code y in {+-1}^D whose projection M y is nearest to w (w ~ M y with
 * M of shape d x D, 关键设计 1; the nearest-point search of 关键设计 2).
 *   A == NULL: exhaustive, every y (2^D candidates; candidate t has y_j = +1
 *              iff bit j of t is set).
 *   A != NULL: the pseudo-inverse start plus auxiliary vector of 关键设计 2,
 *              read as y(v) = sign([M; A]^-1 [w; v]) for every auxiliary sign
 *              vector v in {+-1}^(D-d) (v_k = +1 iff bit k of t is set),
 *              2^(D-d) candidates.  A ((D-d) x D) completes M to an
 *              invertible matrix; with [M; A] orthogonal the candidate is
 *              sign(M^+ w + A^T v).
 * The candidate with the smallest ||w - M y||^2 is chosen, ties to the
 * smallest t, sign(0) = +1.  Arithmetic is float32 (the inverse is formed in
 * float64 and rounded), so groups whose best candidates are within float32
 * rounding of each other may resolve to either.
 * w:     float [groups][d] (group g is weights g*d .. g*d + d - 1; a weight
 *        matrix [m][n] in row-major order is groups = m*n/d).
 * M:     float [d][D];  A: float [D-d][D] or NULL (with D == d, A has no
 *        rows: pass any non-null pointer to select the search).
 * codes: int8 [groups][D], +1 / -1 (the lq_pack_signs input for a matrix of
 *        m rows and K = n*D/d).
 * err:   float [groups], the squared error of the chosen code, or NULL.
 * workspace: with A, >= lq_encode_workspace_size bytes, 256-byte aligned,
 *        caller-owned, no initialisation needed (it receives [M; A]^-1); may
 *        be NULL without A.
 * Requires 1 <= d <= D <= 32 and at most 2^24 candidates (D - d <= 24 with
 * A, D <= 24 without); else LQ_ERR_SHAPE or LQ_ERR_UNSUPPORTED, nothing
 * launched.  groups == 0 is a no-op.  A singular [M; A] gives unspecified
 * codes.  Work grows as groups * 2^(D-d) (or 2^D) * d * D.
 */
lq_status lq_encode_workspace_size(int32_t d, int32_t D, size_t* bytes);
lq_status lq_encode(const float* w, int64_t groups, const float* M, const float* A, int32_t d,
                    int32_t D, int8_t* codes, float* err, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * lq_gemm_decoded -- the layer's product for large batches with the weights
 * decoded instead of the activations lifted: W_hat[i][g*d + r] =
 * sum_j M[r][j] sigma_{i, g*D + j} (w = M y, 关键设计 1), then
 *   out[b][i] = s[i] * sum_{k<n} W_hat[i][k] * u[b][k],
 * the same linear map as lq_gemm on the lifted activations (y . (M^T x) =
 * (M y) . x), at 2 m n B flops for the product plus the reconstruction,
 * instead of 2 m K B (fewer once B > D d / (D - d)).
 * w_packed: uint32 [m][ldw] (layout of lq_pack_signs), ldw >= ceil(K/32),
 *           K = n*D/d.
 * M:        float [d][D];  s: float [m].
 * u:        float16 [B][n], the whitened activations T^-1 a (for example
 *           lq_lift_activations with M = I_4, d = D = 4).
 * out:      float [B][m].
 * workspace: none is needed (lq_gemm_decoded_workspace_size gives 0); the
 *           pointer may be null.
 * Arithmetic: one kernel reconstructs the weights on the matrix cores from
 * M rounded to float16 (exact +-1 signs, float32 sums), rounds them to
 * float16 (relative 2^-11) and contracts them with u on the matrix cores in
 * float32; s[i] scales the float32 result.  The weights never leave the
 * chip.
 * Requires n % d == 0, 1 <= d <= 64, 1 <= D <= 256, n <= 2^22, ldw <= 2^22,
 * m, B <= 2^31 - 1; u must be LQ_F16 (else LQ_ERR_DTYPE).
 */
lq_status lq_gemm_decoded_workspace_size(int64_t m, int64_t n, size_t* bytes);
lq_status lq_gemm_decoded(const uint32_t* w_packed, int64_t m, int64_t n, int64_t ldw,
                          const float* M, int32_t d, int32_t D, const float* s, const void* u,
                          lq_dtype u_dtype, int64_t B, float* out, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * lq_softmin_grad -- the objective that learns M (关键设计 2: M* minimises
 * E_w[min_y ||w - M y||] over Gaussian w, M initialised orthogonal, the inner
 * argmin replaced by a soft-argmin at temperature T, 10 in the notes) on one
 * batch, and its gradient.  Over all 2^D codes y_t (y_tj = +1 iff bit j of t):
 *   p_nt  = softmax_t(-T ||w_n - M y_t||^2),  y_hat_n = sum_t p_nt y_t,
 *   *loss = (1/N) sum_n ||w_n - M y_hat_n||^2,   grad = d loss / d M.
 * w:     float [N][d] samples (drawn by the caller).
 * M:     float [d][D].
 * loss:  device float (one value);  grad: float [d][D].
 * workspace: >= lq_softmin_workspace_size bytes, 256-byte aligned,
 *        caller-owned, no initialisation needed.
 * Requires 1 <= N <= 2^31 - 1, 1 <= d <= D <= 24 (D <= 32 is a valid shape the
 * build does not implement: LQ_ERR_UNSUPPORTED), T finite and >= 0.  float32
 * arithmetic; the result does not depend on timing (fixed partition and
 * summation order).  Work grows as N * 2^D * (d + D).
 */
lq_status lq_softmin_workspace_size(int64_t N, int32_t d, int32_t D, size_t* bytes);
lq_status lq_softmin_grad(const float* w, int64_t N, const float* M, int32_t d, int32_t D,
                          float T, float* loss, float* grad, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * lq_adam_update -- one Adam step on `count` floats in place (the optimiser
 * that learns M; the notes name none, this is the textbook bias-corrected
 * form): m1 = beta1 m1 + (1 - beta1) g, m2 = beta2 m2 + (1 - beta2) g^2,
 * M -= lr (m1 / (1 - beta1^step)) / (sqrt(m2 / (1 - beta2^step)) + eps).
 * m1, m2: caller-owned moment buffers, zero before step 1.  step >= 1,
 * 0 <= beta1, beta2 < 1, eps >= 0; count == 0 is a no-op.
 */
lq_status lq_adam_update(float* M, const float* grad, float* m1, float* m2, int64_t count,
                         int32_t step, float lr, float beta1, float beta2, float eps,
                         void* stream);

/*
 * lq_gemv_workspace_size -- bytes of workspace lq_gemv needs for this shape
 * (0 when none).  Written to *bytes.
 */
lq_status lq_gemv_workspace_size(int64_t m, int64_t K, int64_t B, size_t* bytes);

/*
 * lq_workspace_clear -- zero `bytes` bytes of a workspace on `stream` with a
 * fill kernel.  lq_gemv needs no cleared workspace (every call writes what it
 * reads back); this is a convenience for callers that want a known state.
 */
lq_status lq_workspace_clear(void* workspace, size_t bytes, void* stream);

/*
 * lq_gemv -- the product of the 1-bit weights with the float lifted
 * activations for small batches (关键设计 4 calls this the main body: an
 * ordinary GEMM between 1-bit weights and floats, with no weight codebook to
 * look up):
 *   out[b][i] = s[i] * sum_{k<K} sigma_ik * a_lift[b][k],
 *   sigma_ik = +1 if bit k of row i is 1, else -1.
 * w_packed: uint32 [m][ldw] (layout of lq_pack_signs), ldw >= ceil(K/32),
 *           ldw a multiple of 4 and w_packed 16-byte aligned (16-byte loads).
 * s:        float [m].
 * a_lift:   float [B][K] (lq_lift_activations with LQ_F32), 16-byte aligned,
 *           K % 4 == 0.
 * out:      float [B][m].
 * workspace: device buffer of >= lq_gemv_workspace_size bytes, 256-byte
 *           aligned, owned by the caller; may be NULL when that size is 0.
 *           Its contents need no initialisation.  Calls that share a
 *           workspace must not overlap.
 * Requires 1 <= B <= 16, m >= 1, K >= 1, m*ldw*4 <= 2^30 bytes (split
 * larger matrices by rows over several calls) and K <= 2^24.  Accumulation
 * is float32 and the result does not depend on timing (partial sums over the
 * lifted dimension are added in a fixed order, no float atomics).
 * Arithmetic: the product runs on the matrix cores with the signs as
 * float4 values (exact) and each activation carried by three float8 (E4M3)
 * parts of 4 significant bits each, kept in range by a power-of-two scale
 * per block of positions (1024 positions for B <= 5, 128 for B >= 6): 12
 * significant bits per value (relative error at most 2^-12 of the value,
 * less than 2^-17 of the block's largest one for small values), exact
 * products, float32 sums; about 2e-5 relative output error on the workload
 * shapes.  For B <= 5 the signs enter as 0 / c nibbles and each block adds
 * 2 R - sum(a) (R: the sum over set bits, the block's sum taken in float32).
 */
lq_status lq_gemv(const uint32_t* w_packed, int64_t m, int64_t K, int64_t ldw,
                  const float* s, const float* a_lift, int64_t B, float* out,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * lq_lift_parts_size -- bytes of the operand image lq_lift_parts writes for
 * K lifted positions (written to *bytes).
 */
lq_status lq_lift_parts_size(int64_t K, size_t* bytes);

/*
 * lq_lift_parts -- the lift of lq_lift_activations (关键设计 4: the small
 * transform of the activations, done once per input; 关键设计 1 for M),
 * written not as a_lift but as the operand image that lq_gemv_parts reads,
 * so that the product needs no conversion launch of its own.
 * a, t_inv: [B][n] and [n/t_block][t_block][t_block] of one 16-bit type
 *           (LQ_F16 or LQ_BF16: their products are exact), 16-byte aligned.
 * M:        float [d][D], 4-byte aligned.
 * parts:    device buffer of >= lq_lift_parts_size(n*D/d) bytes, 16-byte
 *           aligned, owned by the caller.  Layout (opaque to callers, fixed
 *           by this library): per 512-position span of the lifted dimension
 *           (whole groups of eight spans, padding spans zero), each token's
 *           lifted values as three float8 (E4M3) parts in the order the
 *           product's matrix operands hold them, then an int power-of-two
 *           exponent per 128 positions and token; a value is p0 + p1/16 +
 *           p2/256 times 2^-e, 12 significant bits.
 * Requires 1 <= B <= 16, t_block == 128, n % 128 == 0, d in {4, 8, 16, 32},
 * n % d == 0, d <= D <= 256.  Accumulation float32.  Errors as
 * lq_lift_activations; LQ_ERR_WORKSPACE if parts_bytes is too small.
 */
lq_status lq_lift_parts(const void* a, lq_dtype a_dtype, int64_t B, int64_t n,
                        const void* t_inv, lq_dtype t_dtype, int32_t t_block,
                        const float* M, int32_t d, int32_t D, void* parts,
                        size_t parts_bytes, void* stream);

/*
 * lq_gemv_parts_workspace_size -- bytes of workspace lq_gemv_parts needs
 * (the partial sums over splits of K), written to *bytes.
 */
lq_status lq_gemv_parts_workspace_size(int64_t m, int64_t K, int64_t B, size_t* bytes);

/*
 * lq_gemv_parts -- lq_gemv on the image of lq_lift_parts instead of float
 * lifted activations (关键设计 4, the 1-bit x float product), for 1 <= B <=
 * 16 tokens on the matrix-core kernel of lq_gemv's 6 - 16 token range:
 *   out[b][i] = s[i] * sum_{k<K} sigma_ik * a_hat[b][k].
 * w_packed, ldw, s, out, K: as lq_gemv.  parts: the image of lq_lift_parts
 * for the same K and B (parts_bytes >= lq_lift_parts_size(K)).  workspace:
 * >= lq_gemv_parts_workspace_size bytes, 256-byte aligned, caller-owned, no
 * initialisation needed; calls sharing it must not overlap.  Deterministic
 * (fixed-order sums).  Errors as lq_gemv.
 */
lq_status lq_gemv_parts(const uint32_t* w_packed, int64_t m, int64_t K, int64_t ldw,
                        const float* s, const void* parts, size_t parts_bytes, int64_t B,
                        float* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lq_stream_read -- a plain read of `bytes` bytes of device memory at
 * `buffer` (16-byte aligned, bytes % 16 == 0), each byte once: the HBM read
 * rate the one-token lq_gemv (which reads each weight byte once) is
 * measured against.  sink: device uint32 [4 * compute units], caller-owned;
 * written only in the unlikely case that the buffer's words fold to one
 * fixed value (which keeps the loads from being removed).  Errors as the
 * other calls; bytes == 0 is a no-op.
 */
lq_status lq_stream_read(const void* buffer, size_t bytes, uint32_t* sink, void* stream);

/*
 * lq_gemv_noalloc -- lq_gemv for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same arguments, kernels and result, without a workspace
 * argument.  The partial sums go to a scratch array the library holds in its
 * code object, one per GPU, LQ_GEMV_NOALLOC_MAX_BYTES bytes, kept until the
 * process ends; its device address is looked up once per device on the
 * first call there.  The call allocates nothing.
 * Every lq_gemv_noalloc call on one GPU uses that GPU's one array: calls
 * that may overlap on one GPU (other streams, other host threads) race and
 * must be ordered by the caller.  Each call writes all of the scratch it
 * reads, so no clearing is needed.
 * Errors as lq_gemv; a shape whose lq_gemv_workspace_size exceeds
 * LQ_GEMV_NOALLOC_MAX_BYTES returns LQ_ERR_WORKSPACE and launches nothing
 * (every workload shape of 1 to 16 tokens up to 28672 x 68096 fits).
 */
#define LQ_GEMV_NOALLOC_MAX_BYTES (16u << 20)
lq_status lq_gemv_noalloc(const uint32_t* w_packed, int64_t m, int64_t K, int64_t ldw,
                          const float* s, const float* a_lift, int64_t B, float* out,
                          void* stream);

/*
 * lq_layer_b1 -- the whole layer for one token, o = diag(s) W_q lift(T^-1 a)
 * (关键设计 4), with the lift computed inside the one-token product: each
 * workgroup of the weight stream computes the lifted activations of the
 * 1024-position slices its tables serve (u = T^-1 a for the slices'
 * channels, then a_hat_g = M^T u_g, float32) before building the tables,
 * while its first weights stream in.  No a_hat buffer, no lift launch; the
 * result is lq_lift_activations followed by lq_gemv with B == 1 (same table
 * arithmetic, a_hat summed in another order).
 * a:      [n] of a_dtype;  t_inv: [n/128][128][128] of t_dtype == a_dtype
 *         (LQ_F16, LQ_BF16 or LQ_F32), both 16-byte aligned;  t_block: 128.
 * M:      float [d][D];  w_packed: uint32 [m][ldw] (lq_pack_signs layout),
 *         ldw >= ceil(K/32), a multiple of 4, 16-byte aligned, K = n*D/d.
 * s:      float [m];  out: float [m].
 * workspace: >= lq_layer_b1_workspace_size bytes (0 when K <= 1024),
 *         256-byte aligned, caller-owned, no initialisation needed.
 * Requires n % 128 == 0, n % d == 0, 1 <= d <= D <= 256, d <= 64,
 * d*D <= 8192, K % 4 == 0, K <= 2^24, m*ldw*4 <= 2^30 (else LQ_ERR_SHAPE,
 * LQ_ERR_UNSUPPORTED or LQ_ERR_ALIGN; nothing launched).  Arithmetic as
 * lq_gemv with B == 1 (float16 activation-sum tables, exact power-of-two
 * scaling, float32 sums).
 */
lq_status lq_layer_b1_workspace_size(int64_t m, int64_t n, int32_t d, int32_t D,
                                     size_t* bytes);
lq_status lq_layer_b1(const void* a, lq_dtype a_dtype, int64_t n, const void* t_inv,
                      lq_dtype t_dtype, int32_t t_block, const float* M, int32_t d, int32_t D,
                      const uint32_t* w_packed, int64_t m, int64_t ldw, const float* s,
                      float* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lq_gemm -- the same product for large batches, contracted on the matrix
 * cores: out[b][i] = s[i] * sum_k sigma_ik * a_lift[b][k] with a_lift in
 * 16-bit (LQ_F16 or LQ_BF16) [B][K]; signs are expanded to exact +-1 16-bit
 * tiles and multiplied with float32 accumulation.
 * w_packed: uint32 [m][ldw] (layout of lq_pack_signs), ldw >= ceil(K/32),
 *           4-byte aligned.
 * a_lift:   16-byte aligned, K % 8 == 0.
 * out:      float [B][m].
 * Requires 1 <= B < 2^31, 1 <= m < 2^31, 1 <= K <= 2^22 and ldw <= 2^22;
 * otherwise LQ_ERR_SHAPE, LQ_ERR_ALIGN or LQ_ERR_DTYPE and nothing is
 * launched.  Each output is one float32 sum in a fixed order (deterministic).
 */
lq_status lq_gemm(const uint32_t* w_packed, int64_t m, int64_t K, int64_t ldw,
                  const float* s, const void* a_lift, lq_dtype lift_dtype, int64_t B,
                  float* out, void* stream);

/*
 * lq_gemm_ep -- the product of the 1-bit weights with 16-bit lifted
 * activations (关键设计 4), followed in the same pass by what a transformer
 * layer does with it: bias, activation or gate, residual, and the store in
 * the layer's own type.  For any number of tokens, from one:
 *   z[b][i]   = s[i] * sum_{k<K} sigma_ik * a_lift[b][k] + bias[i]
 *   out[b][i] = act(z[b][i]) + residual[b][i]                        (gated == 0)
 *   out[b][i] = act(z[b][i]) * z[b][m/2 + i] + residual[b][i], i < m/2  (gated != 0:
 *               the first m/2 rows of W_q are the gate's, the others the up rows)
 * w_packed: uint32 [m][ldw] (layout of lq_pack_signs), 16-byte aligned,
 *           ldw >= ceil(K/32), a multiple of 4, m*ldw*4 <= 2^30; bits at
 *           positions >= K may hold anything.
 * s:        float [m];  bias: float [m] or NULL.
 * a_lift:   [B] rows of K values of lift_dtype (LQ_F16 or LQ_BF16;
 *           lq_lift_activations writes them), lda apart; K and lda multiples
 *           of 8, 16-byte aligned, K <= 2^22.
 * residual: [B] rows, ldr apart, of out_dtype, or NULL; it may be `out`
 *           itself (with ldr == ldo), otherwise it must not overlap it.
 * out:      [B] rows of m (gated: m/2) values of out_dtype (LQ_F32, LQ_F16 or
 *           LQ_BF16, rounded once to nearest even), ldo apart; it must not
 *           overlap a_lift.
 * workspace: >= lq_gemm_ep_workspace_size bytes, 256-byte aligned,
 *           caller-owned, no initialisation needed.
 * Requires B >= 1; B rows of operand image (2.4 bytes per position, 3.1 for
 * float16 outputs, 3.9 for float32 ones) below 4 GiB: split more tokens over several calls.
 * Arithmetic: every value is carried by float6 (E2M3) parts of 4 significant
 * bits with one power of two per 32 positions of a token, three parts for
 * bfloat16 outputs (within 2^-14 of the 32 positions' largest value), four for
 * float16 ones (2^-19), five for float32 (2^-24): less than the outputs' own
 * rounding; exact products with the signs, float32 sums in a fixed
 * order (deterministic); epilogue in float32.  A token that holds an
 * infinity or a NaN gives NaN in all of its outputs.
 */
lq_status lq_gemm_ep_workspace_size(int64_t m, int64_t K, int64_t B, lq_dtype out_dtype,
                                    size_t* bytes);
lq_status lq_gemm_ep(const uint32_t* w_packed, int64_t m, int64_t K, int64_t ldw, const float* s,
                     const void* a_lift, lq_dtype lift_dtype, int64_t lda, int64_t B,
                     const float* bias, lq_act act, int32_t gated, const void* residual,
                     int64_t ldr, void* out, lq_dtype out_dtype, int64_t ldo, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * lq_route -- the router of a mixture-of-experts layer: each token's k
 * experts of E, their weights, and the (token, choice) pairs sorted by expert
 * (within an expert by token), which is what lq_gemm_grouped and
 * lq_gemm_join run over.
 *   ids[t][j]: the experts of the k largest logits, largest first, equal ones
 *     lowest expert first (-0 equals +0).  A NaN or -inf is never chosen; a
 *     token with fewer than k others, or with valid[t] == 0, fills up with -1.
 *   weight[t][j] = exp(l_j) / sum exp(l) over the token's chosen experts
 *     (renorm != 0) or over all of its logits (renorm == 0); 0 where ids is -1.
 *     +inf logits share the whole weight.
 *   offsets[e] .. offsets[e + 1]: the sorted positions of expert e's pairs;
 *   rows[p]: the token of sorted position p, -1 from offsets[E] on;
 *   pos[t][j]: the sorted position of the pair, -1 where ids is -1.
 * logits: [T] rows of E values of dtype, ld apart.  valid: uint8 [T] or NULL.
 * ids, pos: int32 [T][k];  weight: float [T][k];  rows: int32 [T*k];
 * offsets: int32 [E + 1].
 * workspace: >= lq_route_workspace_size bytes (0 up to 64 tokens, then it may
 *     be NULL), 256-byte aligned, caller-owned, no initialisation needed.
 * Requires 1 <= E <= 1024, 1 <= k <= min(E, 32), T >= 0, T*k < 2^31.  T == 0
 * writes zero offsets.  Float32 arithmetic; deterministic.  Weights are within
 * 2^-20 + |l_j - l_max| 2^-24 of their value (the difference is rounded).
 */
lq_status lq_route_workspace_size(int64_t T, int64_t E, int32_t k, size_t* bytes);
lq_status lq_route(const void* logits, lq_dtype dtype, int64_t T, int64_t E, int64_t ld,
                   const uint8_t* valid, int32_t k, int32_t renorm, int32_t* ids, float* weight,
                   int32_t* pos, int32_t* rows, int32_t* offsets, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * lq_gemm_grouped -- one 1-bit matrix per expert and a ragged run of rows
 * each, the way into a mixture-of-experts layer: row r of the sorted order,
 * offsets[e] <= r < offsets[e + 1], is
 *   z[r][i] = s[e][i] * sum_k sigma^e_ik * a_lift[rows[r]][k] + bias[e][i]
 *   out[r] = act(z[r]) or the gated form, as lq_gemm_ep.
 * w_packed: uint32 [E][m][ldw];  s: float [E][m];  bias: float [E][m] or NULL.
 * a_lift:   [a_rows] rows as in lq_gemm_ep.  rows: int32 [R] on the device
 *           (lq_route's), or NULL for row r itself (then a_rows >= R).  An
 *           index outside [0, a_rows) reads a row of zeros.
 * offsets:  int32 [E + 1] on the device, ascending; runs are cut to [0, R].
 * out:      [R] rows of out_dtype, ldo apart.  Rows outside every run are
 *           left as they were.
 * Everything else (limits with a_rows for B, arithmetic, workspace of
 * lq_gemm_grouped_workspace_size bytes) as lq_gemm_ep; 1 <= E <= 1024,
 * 0 <= R < 2^31 (R == 0 is a no-op).  No host synchronisation: the runs are
 * read on the device.
 */
lq_status lq_gemm_grouped_workspace_size(int64_t E, int64_t m, int64_t K, int64_t a_rows,
                                         int64_t R, lq_dtype out_dtype, size_t* bytes);
lq_status lq_gemm_grouped(const uint32_t* w_packed, int64_t E, int64_t m, int64_t K, int64_t ldw,
                          const float* s, const void* a_lift, lq_dtype lift_dtype, int64_t lda,
                          int64_t a_rows, const int32_t* rows, const int32_t* offsets, int64_t R,
                          const float* bias, lq_act act, int32_t gated, void* out,
                          lq_dtype out_dtype, int64_t ldo, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * lq_gemm_join -- the way out: the experts' products on the sorted rows and
 * their weighted sum per token,
 *   z[r][i]   = s[e][i] * sum_k sigma^e_ik * a_lift[r][k] + bias[e][i]
 *   out[t][i] = residual[t][i] + sum_j weight[t][j] * z[pos[t][j]][i].
 * a_lift:   [R] rows in the sorted order (the lifted rows of lq_gemm_grouped).
 * pos, weight: int32 and float [T][k] (lq_route's).  A position outside
 *           [0, R) adds nothing (one inside, but outside every run, adds an
 *           unspecified value: lq_route gives none).
 * residual: [T] rows of out_dtype, ldr apart, or NULL; it may be `out`
 *           (with ldr == ldo).
 * out:      [T] rows of m values of out_dtype, ldo apart; it may overlap a_lift.
 * Sums over j in float32, in order.  1 <= k <= 32, T*k < 2^31, T == 0 is a
 * no-op; everything else as lq_gemm_grouped.
 */
lq_status lq_gemm_join_workspace_size(int64_t E, int64_t m, int64_t K, int64_t R, int64_t T,
                                      int32_t k, lq_dtype out_dtype, size_t* bytes);
lq_status lq_gemm_join(const uint32_t* w_packed, int64_t E, int64_t m, int64_t K, int64_t ldw,
                       const float* s, const void* a_lift, lq_dtype lift_dtype, int64_t lda,
                       const int32_t* offsets, int64_t R, const float* bias, const int32_t* pos,
                       const float* weight, int64_t T, int32_t k, const void* residual,
                       int64_t ldr, void* out, lq_dtype out_dtype, int64_t ldo, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * lq_quant8 -- rows to 8-bit floating point with a power of two for each 128
 * positions, as the activations of lq_gemm8 are held.  With block q of a row
 * the positions 128 q .. 128 q + 127 (those from K on are zeros) and top = 448
 * (LQ_E4M3) or 57344 (LQ_E5M2):
 *   exps[r][q] = 127 + the smallest e >= -127 with max |x| <= top 2^e, the
 *                maximum over the block's finite values (127 if all are zero);
 *   q[r][k]    = x[r][k] 2^(127 - exps[r][q]), rounded once to nearest even.
 * A NaN stays a NaN; an infinity becomes one in LQ_E4M3 and stays in LQ_E5M2.
 * x:    [rows] rows of K values of dtype, ld apart (any alignment of whole
 *       values; 16-byte aligned rows are read fastest).
 * q:    uint8 [rows][ldq], ldq >= K in whole 128, a multiple of 16, 16-byte aligned;
 *       positions from K to the whole 128 are written as zeros.
 * exps: uint8 [rows][lde], lde >= ceil(K / 128), a multiple of 4, 4-byte aligned;
 *       the bytes behind the last block up to a whole word are written too.
 * Requires 1 <= K <= 2^22, 0 <= rows < 2^31 (0 is a no-op); q and exps must not
 * overlap x.
 */
lq_status lq_quant8(const void* x, lq_dtype dtype, int64_t rows, int64_t K, int64_t ld, void* q,
                    lq_dtype q_dtype, int64_t ldq, uint8_t* exps, int64_t lde, void* stream);

/*
 * lq_quant8_blocks -- E matrices of m rows to LQ_E4M3 with a power of two for
 * each block of 128 rows x 128 positions, as the weights of lq_gemm8 are
 * held: as lq_quant8 with the maximum over the block.
 * w:    [E * m] rows of K values of dtype (LQ_F32, LQ_F16, LQ_BF16), ld apart.
 * q:    uint8 [E * m][ldq].   exps: uint8 [E][ceil(m / 128)][lde].
 * Conditions as lq_quant8; 1 <= E <= 1024, 1 <= m <= 2^22.
 */
lq_status lq_quant8_blocks(const void* w, lq_dtype dtype, int64_t E, int64_t m, int64_t K,
                           int64_t ld, void* q, int64_t ldq, uint8_t* exps, int64_t lde,
                           void* stream);

/*
 * lq_gemm8 -- the product of 8-bit weights with a scale for each block of 128
 * rows x 128 positions and 8-bit activations with a power of two for each 128
 * positions, with the epilogue of lq_gemm_ep, for any number of tokens from one:
 *   z[b][i]   = sum_q S[i / 128][q] 2^(exps[b][q] - 127) sum_{k in block q} w[i][k] a[b][k] + bias[i]
 *   out[b][i] = act(z[b][i]) + residual[b][i], or the gated form (lq_gemm_ep).
 * w:       LQ_E4M3 [m][ldw], ldw >= K in whole 128, a multiple of 16, 16-byte aligned,
 *          m * ldw < 2^31; positions from K to the whole 128 hold zeros
 *          (lq_quant8_blocks writes them).
 * scales:  scale_type LQ_E8M0: uint8 [ceil(m / 128)][lds], lds a multiple of 4, 4-byte
 *          aligned; LQ_F32: float of any value, [ceil(m / 128)][lds]; lds >= ceil(K / 128).
 * a:       [B] rows, lda apart, of a_dtype:
 *          LQ_E4M3 or LQ_E5M2 (gradients): as lq_quant8 writes them, with exps
 *          [B][lde]; lda a multiple of 16, 16-byte aligned, lde a multiple of 4;
 *          LQ_F16 or LQ_BF16: K values, any lda >= K; the call quantizes them as
 *          lq_quant8 to LQ_E4M3 (the same result bit for bit); exps is ignored.
 * bias, act, gated, residual, out, out_dtype: as lq_gemm_ep.
 * workspace: >= lq_gemm8_workspace_size bytes (it may be 0), 256-byte aligned,
 *          caller-owned, no initialisation needed.
 * Requires 1 <= K <= 2^22, B >= 1, B rows of 8-bit activations below 4 GiB (also as
 * quantized from 16 bits), lde <= lda, at most 2^29 scales; out must not be a.
 * Exact products, float32 sums in a fixed order (deterministic); epilogue in
 * float32.  For out_dtype LQ_F16 and LQ_BF16 the 8-bit matrix instructions add
 * the products of eight consecutive positions and cut each off, toward zero, 13 binary
 * places below the largest sum of two factors' exponents: 2^-16 of a typical z (root of the
 * mean square) where the factors are normally distributed, 2^-14.5 where one position
 * in a hundred is 20 times the others.  A sum that nearly cancels keeps that error;
 * for LQ_F32 16-bit instructions keep 24 bits, at half the rate or less.
 * A value times its block's power of two lies within float32's normal range, of either
 * operand, and so does a block's sum before its LQ_F32 scale: smaller ones may count
 * as zeros, larger ones as infinities.  A NaN in a token or a byte 255 of its exponents
 * gives NaN in its outputs, a byte 255 of the weights' scales in the outputs of its rows.
 * The gradient of the activations is the same product with the transposed
 * weights and scales (128 x 128 blocks transpose onto blocks).
 */
lq_status lq_gemm8_workspace_size(int64_t m, int64_t K, lq_dtype a_dtype, int64_t B,
                                  size_t* bytes);
lq_status lq_gemm8(const void* w, int64_t m, int64_t K, int64_t ldw, const void* scales,
                   lq_dtype scale_type, int64_t lds, const void* a, lq_dtype a_dtype, int64_t lda,
                   const uint8_t* exps, int64_t lde, int64_t B, const float* bias, lq_act act,
                   int32_t gated, const void* residual, int64_t ldr, void* out,
                   lq_dtype out_dtype, int64_t ldo, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * lq_gemm8_grouped -- the same product with one matrix per expert on ragged runs
 * of rows: row r of the sorted order, offsets[e] <= r < offsets[e + 1], is row
 * rows[r] of a (r itself without rows) through matrix e; an index outside
 * [0, a_rows) counts as a row of zeros.  Rows outside every run are left as
 * they were; runs are cut to [0, R] and read on the device.
 * w: [E][m][ldw];  scales: [E][ceil(m / 128)][lds];  bias: float [E][m] or NULL.
 * a: [a_rows] rows (a_rows >= R without rows).  rows: int32 [R];  offsets:
 * int32 [E + 1], ascending;  out: [R] rows.
 * 1 <= E <= 1024, 0 <= R < 2^31 (0 is a no-op); everything else as lq_gemm8.
 */
lq_status lq_gemm8_grouped_workspace_size(int64_t E, int64_t m, int64_t K, lq_dtype a_dtype,
                                          int64_t a_rows, int64_t R, size_t* bytes);
lq_status lq_gemm8_grouped(const void* w, int64_t E, int64_t m, int64_t K, int64_t ldw,
                           const void* scales, lq_dtype scale_type, int64_t lds, const void* a,
                           lq_dtype a_dtype, int64_t lda, const uint8_t* exps, int64_t lde,
                           int64_t a_rows, const int32_t* rows, const int32_t* offsets, int64_t R,
                           const float* bias, lq_act act, int32_t gated, void* out,
                           lq_dtype out_dtype, int64_t ldo, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * lq_sort_rows -- tokens' rows in the experts' order: out[r] = x[rows[r]], zeros
 * for an index outside [0, T) (lq_route's -1 behind the last run).  Values are
 * moved as they are, `size` bytes each (1, 2 or 4), n to a row; x: [T] rows,
 * ldx apart; out: [R] rows, ldo apart; rows: int32 [R].
 * Requires 1 <= n <= 2^30, T and R < 2^31 (R == 0 is a no-op); out must not
 * overlap x.  Its gradient is lq_join_rows without weights.
 */
lq_status lq_sort_rows(const void* x, int32_t size, int64_t T, int64_t n, int64_t ldx,
                       const int32_t* rows, int64_t R, void* out, int64_t ldo, void* stream);

/*
 * lq_join_rows -- the experts' rows back in the tokens' order, weighted and added:
 *   out[t] = residual[t] + sum_j weight[t][j] z[pos[t][j]],
 * without weights (NULL) their plain sum.  A position outside [0, R) adds nothing.
 * z: [R] rows of n values of dtype, ldz apart.  pos: int32 [T][k];  weight:
 * float [T][k] or NULL.  residual: [T] rows of out_dtype, ldr apart, or NULL;
 * it may be `out` (with ldr == ldo).  out: [T] rows of out_dtype, ldo
 * apart; it must not overlap z.  Float32 sums over j in order, residual last.
 * Requires 1 <= n <= 2^30, 1 <= k <= 32, 0 <= R < 2^31, T*k < 2^31 (T == 0 is a no-op).
 */
lq_status lq_join_rows(const void* z, lq_dtype dtype, int64_t R, int64_t n, int64_t ldz,
                       const int32_t* pos, const float* weight, int64_t T, int32_t k,
                       const void* residual, int64_t ldr, void* out, lq_dtype out_dtype,
                       int64_t ldo, void* stream);

/*
 * lq_join_rows_grad -- the gradients of lq_join_rows with weights, from that of its
 * output dy [T] rows of n:
 *   dz[pos[t][j]] = weight[t][j] dy[t]  (rounded once),
 *   dweight[t][j] = sum_i dy[t][i] z[pos[t][j]][i]  (0 for a position outside [0, R)).
 * With `rows` (lq_route's, int32 [R]) the rows of dz whose rows[r] is outside
 * [0, T) are cleared; without, rows that no pair names are left as they were.
 * Positions of two pairs must differ, as lq_route's do.
 * dy, z, dz: of dtype, ldy, ldz and lddz apart; dz must not overlap dy or z.
 * dweight: float [T][k].  Float32 sums in a fixed order.  Limits as lq_join_rows
 * (T == 0 with rows clears what they say).
 */
lq_status lq_join_rows_grad(const void* dy, lq_dtype dtype, int64_t ldy, const void* z, int64_t ldz,
                            int64_t R, int64_t n, const int32_t* pos, const float* weight,
                            int64_t T, int32_t k, const int32_t* rows, void* dz, int64_t lddz,
                            float* dweight, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LQ_H_ */
