// Host-side argument validation of the entry points of forge_ops.h. Pure C++,
// as validate.hpp. Order of checks: DTYPE, NULL, SHAPE, ALIGN, ALIAS,
// CLIP_NOT_FUSABLE, HPARAM, TILE.
#pragma once

#include <cstdint>

#include "forge_ops.h"
#include "validate.hpp"

namespace forge {

// Elements of all tensors of a list together: keeps the norm's chunk indexes
// within 31 bits.
constexpr int64_t kMaxListElems = int64_t(1) << 42;

int64_t grad_norm_workspace(int32_t count);
forge_status validate_grad_norm(const forge_tensor* tensors, int32_t count, double max_norm,
                                const float* norm_coef, const void* workspace,
                                int64_t workspace_bytes);
forge_status validate_clip_grads(const forge_tensor* tensors, int32_t count, const float* coef);
forge_status validate_adamw_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                    const forge_adamw_params* p);
forge_status validate_sgdm_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                   const forge_sgdm_params* p);

// Byte offsets of the parts of the embedding gradient's workspace.
struct EmbeddingWorkspace {
  int64_t keys[2], pos[2], count, bound, chunk, bytes;
};
// Tokens whose sum is formed ahead of a row's, as a power of two. A row of n
// tokens adds up at most 2 (C - 1) + n / C terms one after the other: 32 serve
// frequent ids of thousands of tokens, more those of tens of thousands. Of 16384
// tokens into 32000 x 1024 with 4400 of one id: 52 us with 32, 64 with 128. Of
// 262144 with 71500 of one id: 320 us with 32, 191 with 128, 209 with 256 (spread
// evenly 162 with each). Of 1048576 into 32000 x 512 with 286000: 991 with 32, 441
// with 128, 354 with 256, and spread evenly over 300 rows 304, 315 and 338.
inline int embedding_chunk_bits(int64_t T) { return T <= 32768 ? 5 : T <= 524288 ? 7 : 8; }
bool embedding_sizes_ok(int64_t T, int64_t V, int64_t d);
EmbeddingWorkspace embedding_workspace(int64_t T, int64_t V, int64_t d);
forge_status validate_embedding(const void* table, forge_dtype table_dtype, const void* ids,
                                int32_t id_bytes, const void* out, forge_dtype out_dtype,
                                int64_t T, int64_t V, int64_t d, double scale);
// outs: the float32 arrays [V, d] that the call writes.
forge_status validate_embedding_grad(const void* ids, int32_t id_bytes, const void* dY,
                                     forge_dtype dY_dtype, const void* const* outs, int n_outs,
                                     int64_t T, int64_t V, int64_t d, double scale,
                                     const void* workspace, int64_t workspace_bytes);

forge_status validate_quantize_mxfp4(const void* x, forge_dtype x_dtype, int64_t R, int64_t C,
                                     const void* row_codes, const void* row_scales,
                                     const void* col_codes, const void* col_scales);
forge_status validate_matmul_mxfp4(const void* a_codes, const void* a_scales, const void* b_codes,
                                   const void* b_scales, const void* out, forge_dtype out_dtype,
                                   int64_t M, int64_t N, int64_t Kp, forge_tile tile);
forge_status validate_wgrad_adamw_mxfp4(const void* x_codes, const void* x_scales,
                                        const void* dy_codes, const void* dy_scales,
                                        const float* W, const float* m, const float* v, int64_t Kp,
                                        int64_t d_in, int64_t d_out, const forge_adamw_params* p,
                                        forge_tile tile);

// Most partial sums of the layer norm's weight gradients (one workgroup each).
constexpr int64_t kLayernormParts = 512;
int64_t layernorm_workspace(int64_t T, int64_t d);
forge_status validate_layernorm(const void* x, forge_dtype x_dtype, const float* gamma,
                                const float* beta, const void* y, forge_dtype y_dtype,
                                const float* mean, const float* rstd, int64_t T, int64_t d,
                                double eps);
forge_status validate_layernorm_backward(const void* dY, forge_dtype y_dtype, const void* x,
                                         forge_dtype x_dtype, const float* gamma,
                                         const float* mean, const float* rstd, const void* dX,
                                         const float* dgamma, const float* dbeta, int64_t T,
                                         int64_t d, const void* workspace,
                                         int64_t workspace_bytes);

// Columns of a chunk of a row of logits, which one workgroup goes through.
constexpr int64_t kDistillChunk = 4096;
// Most columns of a row of bf16 logits that a workgroup's registers hold; float32 half.
constexpr int64_t kDistillHeld = 131072;
// Most rows that are cut into chunks, of any type of logits, and whether a call's are.
constexpr int64_t kDistillChunkRows = 656;
bool distill_in_chunks(int64_t T, int64_t V, bool bf16, bool grad);
// Byte offsets of the parts of distillation's workspace: each chunk's maximum
// and sum of exponentials, and the student's logits of the teacher's ids. Only
// rows that are cut into chunks have them, but its size never falls with T, V or K: what was
// made for the largest batch does for a smaller one.
struct DistillWorkspace {
  int64_t stats, logit, bytes;
};
bool distill_sizes_ok(int64_t T, int64_t V, int64_t K);
DistillWorkspace distill_workspace(int64_t T, int64_t V, int64_t K);
forge_status validate_distill(const void* logits, forge_dtype z_dtype, int64_t ld,
                              const void* teacher, forge_dtype teacher_dtype, const void* ids,
                              int32_t id_bytes, const float* weight, const float* loss,
                              const void* grad, forge_dtype grad_dtype, int64_t T, int64_t V,
                              int64_t K, double temperature, double scale, const void* workspace,
                              int64_t workspace_bytes);

forge_status validate_quantize_fp8_block(const void* x, forge_dtype x_dtype, int64_t R, int64_t C,
                                         forge_dtype fmt, const void* row_codes,
                                         const void* row_scales, const void* col_codes,
                                         const void* col_scales);
forge_status validate_matmul_fp8_block(const void* a_codes, const void* a_scales, forge_dtype a_fmt,
                                       const void* b_codes, const void* b_scales, forge_dtype b_fmt,
                                       const void* out, int64_t M, int64_t N, int64_t Kp,
                                       forge_tile tile);

}  // namespace forge
