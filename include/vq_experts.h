/*
 * vq_experts.h -- C ABI of libvq, part three: the codebook-indexed layers of a
 * mixture of experts (the weights are vq.h's, one layer per expert).
 *
 * A router gives every token top_k expert ids and weights.  vq_group_rows
 * puts the picks in the order of their experts, vq_gemm_experts multiplies
 * each group of rows by its expert's weights, vq_combine_rows adds a token's
 * results up.  Group sizes stay on the device: no call waits for them, and a
 * captured CUDA graph of the calls serves any routing of the same sizes.
 *
 * The conventions of vq.h hold (pointers, streams, errors, thread safety).
 * The status word of a workspace is set to VQ_ERR_TIMEOUT when a bounded
 * device-side wait gave up and is left alone otherwise: zero it when the
 * workspace is made, and it covers every call since.  The rest of a
 * workspace's contents on entry does not matter.
 */
#ifndef VQ_EXPERTS_H_
#define VQ_EXPERTS_H_

#include "vq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VQ_EXPERTS_VERSION 1
#define VQ_MAX_EXPERTS 1024
#define VQ_MAX_TOP_K 64

/*
 * Experts of one shape.  `layer` describes expert 0 as in vq.h (vec_dim up to
 * 16, either index order); expert e's arrays lie e strides further on:
 *   idx_stride[m]       32-bit words, a multiple of 4
 *   codebook_stride[m]  fp16 values, a multiple of 8; 0: one book for all
 *   scale_stride, bias_stride, out_bias_stride   fp16 values (of the arrays
 *                       that the layer has); 0: one array for all
 * Strides are not negative.
 */
typedef struct vq_experts_desc {
    vq_layer_desc layer;
    int32_t n_experts;        /* 1..VQ_MAX_EXPERTS */
    int32_t reserved;         /* must be 0 */
    int64_t idx_stride[2];
    int64_t codebook_stride[2];
    int64_t scale_stride;
    int64_t bias_stride;
    int64_t out_bias_stride;
} vq_experts_desc;

/*
 * vq_group_rows -- a stable counting sort of the picks by expert.
 *   ids      device int32 [n_tokens][ld_ids], top_k columns used; an id outside
 *            0..n_experts-1 (a padded token, a dropped pick) gets no row
 *   offsets  device int32 [n_experts + 1]: expert e's rows are offsets[e] ..
 *            offsets[e+1]-1, offsets[0] = 0
 *   rows     device int32 [n_tokens * top_k]: the token of each grouped row; -1
 *            behind the last group.  Inside a group, tokens ascend (and picks
 *            of one token keep their order).
 *   pos      device int32 [n_tokens][top_k]: the grouped row of each pick, -1
 *            for one without
 * One launch, no workspace.  top_k 1..VQ_MAX_TOP_K, n_tokens * top_k <= 2^30.
 * Errors: VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED (too many experts, picks or
 * top_k), VQ_ERR_ALIGNMENT, VQ_ERR_CUDA.
 */
VQ_API vq_status vq_group_rows(const int32_t* ids, int32_t n_tokens, int32_t top_k, int64_t ld_ids,
                               int32_t n_experts, int32_t* offsets, int32_t* rows, int32_t* pos,
                               void* stream);

/* Bytes of device workspace vq_gemm_experts needs for these experts and m
 * grouped rows (host-only, launches nothing). */
VQ_API vq_status vq_gemm_experts_workspace_size(const vq_experts_desc* experts, int32_t m, size_t* bytes);

/*
 * vq_gemm_experts -- y[r][o] = sum_k x[src(r)][k] W_e[o][k] + out_bias_e[o] for
 * every expert e and row r of its group, W_e[o][k] = (C1[i1] + C2[i2]) s_e[o] +
 * t_e[o] as in vq.h, without writing W to global memory.  Products of fp16
 * operands with fp32 accumulation on the tcgen05 tensor cores.
 *   x, x_rows, ldx   device bf16 or fp16 [x_rows][ldx], ldx >= Kin
 *   rows       NULL: src(r) = r (x_rows >= m); else device int32 [m]: src(r) =
 *              rows[r] (a row outside 0..x_rows-1 counts as zeros)
 *   offsets    device int32 [n_experts + 1] as vq_group_rows writes it.  The
 *              kernels clamp what they read to 0..m and to ascending order
 *   m          rows that y (and rows) have room for; rows from offsets[n_experts]
 *              on are not written
 *   y          device, y_dtype (bf16, fp16 or fp32) [m][ldy], ldy >= N
 *   workspace  at least vq_gemm_experts_workspace_size() bytes, 256-byte
 *              aligned; first 32-bit word: status (see above)
 * Each row of x is scaled by a power of two into fp16 (values below 2^-29 of
 * the row's largest lose precision as fp16 subnormals); with two books c1 + c2
 * is rounded once to fp16; scale and bias are applied in fp32 to the sum: y =
 * s sum_k x (c1 + c2) + t sum_k x + out_bias.  The order of every sum depends
 * on the sizes and the group sizes only, so repeated calls agree bit for bit.
 * A row of x that holds an infinity or a NaN has non-finite products; the
 * other rows are not touched by it.
 * Errors: VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED (m > 2^24, or (n_experts +
 * m / 16) * ceil(N / 128) >= 2^31), VQ_ERR_ALIGNMENT
 * (arrays; x and y to their element sizes), VQ_ERR_WORKSPACE, VQ_ERR_CUDA.
 */
VQ_API vq_status vq_gemm_experts(const vq_experts_desc* experts, const void* x, vq_dtype x_dtype,
                                 int32_t x_rows, int64_t ldx, const int32_t* rows, const int32_t* offsets,
                                 int32_t m, void* y, vq_dtype y_dtype, int64_t ldy, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * vq_combine_rows -- y[t][c] = sum_{j < top_k} weight[t][j] * z[pos[t][j]][c],
 * the sum in fp32 with j ascending, rounded once to y's type.  A pos outside
 * 0..z_rows-1 adds nothing (its weight is not read into the sum).
 *   z, z_rows, ldz   device z_dtype (bf16, fp16 or fp32) [z_rows][ldz], n columns
 *   pos        device int32 [n_tokens][top_k]
 *   weight     device fp32 [n_tokens][ld_weight], ld_weight >= top_k
 *   y          device, y_dtype [n_tokens][ldy]; may not overlap z
 * Errors: VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED (top_k), VQ_ERR_ALIGNMENT,
 * VQ_ERR_CUDA.
 */
VQ_API vq_status vq_combine_rows(const void* z, vq_dtype z_dtype, int32_t z_rows, int32_t n, int64_t ldz,
                                 const int32_t* pos, const float* weight, int64_t ld_weight,
                                 int32_t n_tokens, int32_t top_k, void* y, vq_dtype y_dtype, int64_t ldy,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VQ_EXPERTS_H_ */
