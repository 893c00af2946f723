/*
 * vq_i8.h -- C ABI of libvq, part two: linear layers in 8-bit integers, for
 * the projections of a model that do not stand two or three bits a weight
 * (attention, shared experts, heads) beside its codebook-indexed ones (vq.h).
 *
 * The method
 * ----------
 * Activations x [m][Kin] are quantised symmetrically row by row ("per token"):
 *     s[i] = fp32(max_k |x[i][k]| / 127),   q[i][k] = rne(x[i][k] / s[i]),
 * rne rounding the exact quotient to the nearest integer, ties to even; q lies
 * in -127..127.  A row of zeros has s = 0 and q = 0.  A row that holds an
 * infinity or a NaN has s = NaN and q = 0, so its products are NaN.  Weights
 * are int8 [N][ldw] with one fp32 scale per output channel (the same
 * quantisation, applied to the rows of W, produces them).  The product is
 *     y[i][o] = (float(sum_k q[i][k] w[o][k]) * w_scale[o]) * s[i] + out_bias[o]
 * with the sum exact in 32-bit integers (Kin <= 131071, so that no sum of
 * products of -128 overflows) and the rest fp32 operations, rounded once to
 * y's type.  Weights and activations may hold any int8 value, -128 included.
 *
 * The conventions of vq.h hold (pointers, streams, errors, thread safety),
 * with one difference: the status word of a workspace here is set to
 * VQ_ERR_TIMEOUT when a bounded device-side wait gave up and is left alone
 * otherwise, so that a call needs no launch to clear it.  Zero it when the
 * workspace is made; it then covers every call since.  The rest of a
 * workspace's contents on entry does not matter.
 */
#ifndef VQ_I8_H_
#define VQ_I8_H_

#include "vq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VQ_I8_VERSION 1
#define VQ_I8_MAX_IN_FEATURES 131071

/*
 * One layer.  All pointers are device pointers.
 *   out_features   N >= 0
 *   in_features    Kin, 0..VQ_I8_MAX_IN_FEATURES
 *   w, ldw         int8 [N][ldw], 16-byte aligned, ldw >= Kin a multiple of 16;
 *                  columns past Kin are not used
 *   scale          fp32 [N]
 *   out_bias       fp16 [N], or NULL
 */
typedef struct vq_i8_desc {
    int32_t out_features;
    int32_t in_features;
    const int8_t* w;
    int64_t ldw;
    const float* scale;
    const uint16_t* out_bias;
} vq_i8_desc;

/*
 * vq_quant_i8 -- the quantisation above of `rows` rows of n values: x (bf16 or
 * fp16) [rows][ldx] to q int8 [rows][ldq] and scale fp32 [rows].  Columns of q
 * past n are not written.  Works on activations (a row per token) and on
 * weights (a row per output channel).  Any alignment of whole elements; rows
 * that start on 16 bytes (x) and 8 bytes (q) are read and written in one pass.
 * Errors: VQ_ERR_INVALID_ARG (sizes, types, short strides, NULL buffers with
 * data), VQ_ERR_ALIGNMENT, VQ_ERR_CUDA.
 */
VQ_API vq_status vq_quant_i8(const void* x, vq_dtype x_dtype, int32_t rows, int32_t n, int64_t ldx,
                             int8_t* q, int64_t ldq, float* scale, void* stream);

/* Bytes of device workspace vq_gemm_i8 needs for this layer and row count
 * (host-only, launches nothing). */
VQ_API vq_status vq_gemm_i8_workspace_size(const vq_i8_desc* layer, int32_t m, size_t* bytes);

/*
 * vq_gemm_i8 -- the product above of quantised rows, on the tcgen05 integer
 * tensor cores.  One row (a decoding token) to any number of them.
 *   q, ldq     device int8 [m][ldq], 16-byte aligned, ldq >= Kin a multiple
 *              of 16; columns past Kin are not used
 *   q_scale    device fp32 [m]
 *   y          device, y_dtype (bf16, fp16 or fp32) [m][ldy], ldy >= N
 *   workspace  at least vq_gemm_i8_workspace_size() bytes, 256-byte aligned;
 *              first 32-bit word: status (see above)
 * The sums are exact, so y does not depend on how the work is split.
 * Errors: VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED (Kin or m out of range, m >
 * 2^30), VQ_ERR_ALIGNMENT, VQ_ERR_WORKSPACE, VQ_ERR_CUDA.
 */
VQ_API vq_status vq_gemm_i8(const vq_i8_desc* layer, const int8_t* q, int64_t ldq, const float* q_scale,
                            int32_t m, void* y, vq_dtype y_dtype, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * vq_linear_i8 -- vq_quant_i8 of x into the workspace, then vq_gemm_i8: a
 * layer's whole forward from bf16 or fp16 activations (any 2-byte alignment).
 * Layers that share x are served better by one vq_quant_i8 and a vq_gemm_i8
 * each.  Same results and errors as the two calls.
 */
VQ_API vq_status vq_linear_i8_workspace_size(const vq_i8_desc* layer, int32_t m, size_t* bytes);
VQ_API vq_status vq_linear_i8(const vq_i8_desc* layer, const void* x, vq_dtype x_dtype, int32_t m,
                              int64_t ldx, void* y, vq_dtype y_dtype, int64_t ldy, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VQ_I8_H_ */
