/*
 * forge_ops.h - C ABI of the operators around the fused weight-gradient step
 * (forge.h) for AMD Instinct MI355X (gfx950): the embedding's lookup and
 * gradient, the global gradient norm with the clipped optimizer steps, and
 * microscaled 4-bit products.
 *
 * The conventions of forge.h hold here too: device pointers owned by the
 * caller, dense row-major arrays, 16-byte aligned pointers, nothing allocated,
 * no state between calls, validation before anything is launched,
 * asynchronous and ordered on `stream`, current device gfx950. Outputs must
 * not overlap each other or an input, unless said otherwise. Sums are float32
 * or wider and no call uses atomics, so every result is bitwise the same from
 * run to run.
 *
 * Workspaces. Where a call takes `workspace`, it is caller-owned device memory
 * of at least the stated size, 16-byte aligned, overlapping nothing else; its
 * contents are scratch, need no initialisation and mean nothing after the call.
 * Two calls that may run at the same time (two streams, two captured graphs
 * replayed side by side) need two workspaces.
 */
#ifndef FORGE_OPS_H
#define FORGE_OPS_H

#include "forge.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The global gradient norm over many tensors, and clipping.
 *
 * Exact global-norm clipping needs the norm of the whole gradient before any
 * weight moves, so it is refused by the fused steps
 * (FORGE_ERR_CLIP_NOT_FUSABLE). This is the path for it: gradients stored by
 * forge_wgrad, forge_wgrad_bf16, forge_wgrad_fp8, forge_matmul_mxfp4 or
 * forge_embedding_grad, one pass for their norm, one for the step. */

/*
 * One tensor of a list. n elements, 0 <= n <= 2^40 and at most 2^42 in the
 * list (else FORGE_ERR_SHAPE); a tensor of n == 0 is skipped and its pointers
 * are not looked at. Each call names the fields that it uses
 * and does not look at the others.
 */
typedef struct {
  const void* grad;       /* gradient, FORGE_F32 or FORGE_BF16          */
  void* out;              /* clipped gradient, of the gradient's type   */
  float* W;               /* weight                                     */
  float* m;               /* first moment (AdamW) or momentum buffer    */
  float* v;               /* second moment (AdamW)                      */
  int64_t n;              /* elements                                   */
  forge_dtype grad_dtype; /* FORGE_F32 or FORGE_BF16                    */
} forge_tensor;

/* Most tensors of one list. Their addresses are below 2^52, as every device
 * address is (else FORGE_ERR_ALIGN). */
#define FORGE_MAX_TENSORS 65536

/* Bytes of forge_grad_norm's workspace for `count` tensors, at least 16; 0 if
 * count is out of range. */
FORGE_API int64_t forge_grad_norm_workspace(int32_t count);

/*
 * norm_coef[0] = sqrt(sum over all tensors of g^2), norm_coef[1] =
 * min(1, max_norm / (norm + 1e-6)), both float32 on the device.
 *   tensors HOST array of count entries; uses grad, n, grad_dtype. Gradients
 *   may overlap or recur (each entry counts). Squares are formed and summed
 *   in 64 bits, so no finite gradient overflows or vanishes; a norm beyond
 *   float32 is stored as +inf, with the coefficient of its 64-bit value. A
 *   NaN or infinity among the gradients gives a NaN or +inf norm and a
 *   coefficient of NaN or 0. With no elements at all the norm is 0.
 *   max_norm >= 0; +inf asks for the norm alone (the coefficient is then 1,
 *   or NaN where the norm is not finite). NaN or negative: FORGE_ERR_HPARAM.
 *   workspace: forge_grad_norm_workspace(count) bytes.
 */
FORGE_API forge_status forge_grad_norm(const forge_tensor* tensors, int32_t count, double max_norm,
                             float* norm_coef, void* workspace, int64_t workspace_bytes,
                             void* stream);

/*
 * out = coef * grad for every tensor: the float32 product, rounded to the
 * gradient's type.
 *   coef: ONE float32 on the device (norm_coef + 1 of forge_grad_norm; any
 *   alignment that a float has). Uses grad, out, n, grad_dtype. out may equal
 *   grad (in place); partial overlap of any two arrays is FORGE_ERR_ALIAS.
 */
FORGE_API forge_status forge_clip_grads(const forge_tensor* tensors, int32_t count, const float* coef,
                              void* stream);

/*
 * The optimizer step of forge_adamw / forge_sgdm on coef * grad for every
 * tensor, the product formed in float32 in registers: no clipped gradient is
 * stored. Uses grad, W, m (and v for AdamW), n, grad_dtype; W, m, v are
 * float32 and updated in place. coef as in forge_clip_grads. With a
 * coefficient of exactly 1 the result is bitwise forge_adamw's (forge_sgdm's).
 * The clip is in coef: p->max_grad_norm must be 0, as in forge.h. Gradients
 * may overlap each other; W, m and v overlap nothing.
 */
FORGE_API forge_status forge_adamw_clipped(const forge_tensor* tensors, int32_t count,
                                 const float* coef, const forge_adamw_params* p, void* stream);
FORGE_API forge_status forge_sgdm_clipped(const forge_tensor* tensors, int32_t count,
                                const float* coef, const forge_sgdm_params* p, void* stream);

/* ------------------------------------------------------------------------
 * The embedding: lookup with scaling, and its gradient by sorted tokens.
 *
 * The embedding is the weight whose gradient is a sum over tokens without a
 * matrix product: g[r] = scale * sum over t with ids[t] == r of dY[t].
 *   ids [T] int32 or int64 (id_bytes 4 or 8, else FORGE_ERR_DTYPE), on the
 *   device, aligned as such integers are. An id outside [0, V) is nobody's row: its lookup is a row of
 *   zeros and it adds to no gradient (padding, or the tokens of another
 *   shard of the vocabulary).
 *   scale: finite (else FORGE_ERR_HPARAM), rounded to float32.
 *   0 <= T <= 2^30, 0 <= V <= 2^22, d a multiple of 8 up to 2^22. T == 0, V == 0
 *   and d == 0 are allowed.
 */

/*
 * out[t] = scale * table[ids[t]]: the float32 product, rounded to out's type.
 *   table [V, d] of table_dtype, out [T, d] of out_dtype, each FORGE_F32 or
 *   FORGE_BF16.
 */
FORGE_API forge_status forge_embedding(const void* table, forge_dtype table_dtype, const void* ids,
                             int32_t id_bytes, void* out, forge_dtype out_dtype, int64_t T,
                             int64_t V, int64_t d, double scale, void* stream);

/* Bytes of the workspace of the gradient calls below, at least 16; 0 if a size
 * is out of range. */
FORGE_API int64_t forge_embedding_workspace(int64_t T, int64_t V, int64_t d);

/*
 * grad [V, d] float32: the gradient of every row, zero for rows without a
 * token; accumulate != 0 adds it to what grad holds instead (a tied weight,
 * after the output layer's forge_wgrad), and rows without a token are then
 * neither read nor written.
 *   dY [T, d] of dY_dtype (FORGE_F32 or FORGE_BF16). A row's tokens are summed
 *   in float32 in an order that ids alone decide, and the sum is scaled once.
 */
FORGE_API forge_status forge_embedding_grad(const void* ids, int32_t id_bytes, const void* dY,
                                  forge_dtype dY_dtype, float* grad, int64_t T, int64_t V,
                                  int64_t d, double scale, int32_t accumulate, void* workspace,
                                  int64_t workspace_bytes, void* stream);

/*
 * The same gradient consumed by the optimizer as it is formed, never stored:
 * the step of forge_wgrad_adamw (forge_wgrad_sgdm) on W, m, v (W, mom)
 * [V, d] float32, in place. Rows without a token take the step with a zero
 * gradient: their moments and weights still decay. For an untied embedding
 * (see the preconditions in forge.h). The result is bitwise
 * forge_embedding_grad followed by forge_adamw (forge_sgdm).
 */
FORGE_API forge_status forge_embedding_adamw(const void* ids, int32_t id_bytes, const void* dY,
                                   forge_dtype dY_dtype, float* W, float* m, float* v, int64_t T,
                                   int64_t V, int64_t d, double scale,
                                   const forge_adamw_params* p, void* workspace,
                                   int64_t workspace_bytes, void* stream);
FORGE_API forge_status forge_embedding_sgdm(const void* ids, int32_t id_bytes, const void* dY,
                                  forge_dtype dY_dtype, float* W, float* mom, int64_t T,
                                  int64_t V, int64_t d, double scale, const forge_sgdm_params* p,
                                  void* workspace, int64_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Microscaled 4-bit operands (OCP MX, MXFP4) and their product.
 *
 * Values along the contraction K are cut into blocks of 32. A block has one
 * scale, a power of two 2^(s - 127) stored as the byte s (E8M0), and 32 codes
 * of 4 bits (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit). s is the
 * biased float32 exponent of the block's largest magnitude minus 2, at least
 * 0; values are rounded to the nearest code, ties to the even code, and
 * magnitudes beyond 6 become 6. A block with a NaN or an infinity has s = 255
 * (NaN), and every value of it is NaN.
 *
 * An operand of R rows and K columns, with Kp = FORGE_MXFP4_K(K):
 *   codes  [Kp / 128, R, 64] bytes: entry (g, r) holds row r's columns
 *          128 g .. 128 g + 127, the even one in the low half of a byte;
 *   scales [Kp / 128, R, 4] bytes: byte b of entry (g, r) is the scale of
 *          row r's columns 128 g + 32 b .. + 31.
 * Columns K .. Kp - 1 hold zero codes.
 */
#define FORGE_MXFP4_K(K) (((int64_t)(K) + 127) / 128 * 128)

/* Largest padded contraction length; an operand has at most 2^22 rows and a
 * product at most 2^40 elements (else FORGE_ERR_SHAPE). */
#define FORGE_MXFP4_MAX_K 1073741824

/*
 * Quantises x [R, C] (x_dtype FORGE_F32 or FORGE_BF16) into either or both of
 *   row_codes, row_scales: the operand of R rows with K = C (blocks along a
 *     row of x: the contraction runs over x's columns);
 *   col_codes, col_scales: the operand of C rows with K = R (blocks along a
 *     column of x, transposed: the contraction runs over x's rows, as the
 *     tokens of a weight gradient).
 * A pair is left out by two NULLs; one NULL of a pair, or both pairs left
 * out, is FORGE_ERR_NULL. C % 8 == 0, any R. Both pairs read x once.
 */
FORGE_API forge_status forge_quantize_mxfp4(const void* x, forge_dtype x_dtype, int64_t R, int64_t C,
                                  void* row_codes, void* row_scales, void* col_codes,
                                  void* col_scales, void* stream);

/*
 * out [M, N] (FORGE_F32, or FORGE_BF16 rounded to nearest even) = A B^T for
 * operands A of M rows and B of N rows, both of the padded length Kp
 * (a multiple of 128, else FORGE_ERR_ALIGN). N % 8 == 0, any M.
 * Kp == 0 writes zeros. Products are exact; they are accumulated in float32
 * in ascending steps of 64 columns, so every tile gives the same bits.
 *   Weight gradient   g = dY^T X:  A = dY by columns, B = X by columns.
 *   Input gradient    dX = dY W:   A = dY by rows,    B = W by columns.
 *   Layer output      Y = X W^T:   A = X by rows,     B = W by rows.
 * tile: the ids of forge.h over [N, M]; the default may also take smaller
 * tiles, for outputs that would leave most of the chip idle.
 */
FORGE_API forge_status forge_matmul_mxfp4(const void* a_codes, const void* a_scales,
                                const void* b_codes, const void* b_scales, void* out,
                                forge_dtype out_dtype, int64_t M, int64_t N, int64_t Kp,
                                forge_tile tile, void* stream);

/*
 * Weight gradient from microscaled operands, consumed by AdamW in the
 * product's epilogue as in forge_wgrad_adamw: x the operand of d_in rows and
 * dy the operand of d_out rows over the tokens (both quantised by columns),
 * W, m, v [d_out, d_in] float32, in place. Kp == 0 takes a pure decay step.
 * The result is bitwise forge_matmul_mxfp4 followed by forge_adamw.
 */
FORGE_API forge_status forge_wgrad_adamw_mxfp4(const void* x_codes, const void* x_scales,
                                     const void* dy_codes, const void* dy_scales, float* W,
                                     float* m, float* v, int64_t Kp, int64_t d_in, int64_t d_out,
                                     const forge_adamw_params* p, forge_tile tile, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FORGE_OPS_H */
