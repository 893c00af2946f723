// experts.cu -- vq_gemm_experts: products of codebook-indexed experts over the
// ragged groups of rows that a router made (include/vq_experts.h).
#include <algorithm>

#include "codebook.cuh"
#include "vq_experts.h"

namespace vqk {
namespace {

// A validated description, passed to kernels by value.
struct Experts {
  Layer L;                 // expert 0
  int e;                   // number of experts
  int64_t si[2], sb[2];    // strides between experts: index words, book values
  int64_t ss, st, so;      //   scale, bias, output bias values
};

// Expert x's layer.
__device__ __forceinline__ Layer expert_layer(const Experts& E, int x) {
  Layer L = E.L;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    L.idx[m] += x * E.si[m];
    L.book[m] += x * E.sb[m];
  }
  if (L.scale) L.scale += x * E.ss;
  if (L.bias) L.bias += x * E.st;
  if (L.ob) L.ob += x * E.so;
  return L;
}

// One grouped row and 128 outputs per block.
__global__ void __launch_bounds__(128) gemm_experts_kernel(Experts E, const uint16_t* __restrict__ x, int x_fp16,
                                                           int x_rows, int64_t ldx, const int32_t* __restrict__ rows,
                                                           const int32_t* __restrict__ offsets, int m,
                                                           void* __restrict__ y, vq_dtype yt, int64_t ldy) {
  const int o = blockIdx.x * 128 + threadIdx.x;
  for (int r = blockIdx.y; r < m; r += gridDim.y) {
    int ex = -1, last = 0;
    for (int k = 0; k < E.e && ex < 0; ++k) {
      last = max(last, min(m, offsets[k + 1]));
      if (r < last && r >= min(m, max(0, offsets[k]))) ex = k;
    }
    if (ex < 0 || o >= E.L.n) continue;
    const Layer L = expert_layer(E, ex);
    const int src = rows ? rows[r] : r;
    const bool live = src >= 0 && src < x_rows;
    float acc = 0.0f, sum = 0.0f;
    for (int j = 0; live && j < L.nvec; ++j) {
      uint32_t i[2];
      for (int b = 0; b < L.nb; ++b)
        i[b] = L.layout == VQ_IDX_ROWS
                   ? load_field(L.idx[b] + o * L.rw[b], static_cast<int64_t>(j) * L.b[b], L.b[b])
                   : load_field(L.idx[b] + (j >> 2) * L.rw[b], (4 * static_cast<int64_t>(o) + (j & 3)) * L.b[b], L.b[b]);
      for (int k = 0; k < L.d && j * L.d + k < L.kin; ++k) {
        const uint16_t u = __ldg(x + src * ldx + j * L.d + k);
        const float v = x_fp16 ? h2f(u) : bf2f(u);
        float c = h2f(L.book[0][static_cast<int64_t>(i[0]) * L.d + k]);
        if (L.nb == 2) c += h2f(L.book[1][static_cast<int64_t>(i[1]) * L.d + k]);
        acc = fmaf(v, c, acc);
        sum += v;
      }
    }
    const float s = L.scale ? h2f(L.scale[o]) : 1.0f, t = L.bias ? h2f(L.bias[o]) : 0.0f;
    store_out(y, yt, r * ldy + o, s * acc + t * sum + out_bias_of(L.ob, o));
  }
}

constexpr int kMaxGroupedRows = 1 << 24;

vq_status check_experts(const vq_experts_desc* d, Experts* E) {
  if (!d) return VQ_ERR_INVALID_ARG;
  if (d->n_experts < 1 || d->reserved != 0) return VQ_ERR_INVALID_ARG;
  if (d->n_experts > VQ_MAX_EXPERTS) return VQ_ERR_UNSUPPORTED;
  vq_status st = check_layer(&d->layer, &E->L);
  if (st != VQ_OK) return st;
  if (d->scale_stride < 0 || d->bias_stride < 0 || d->out_bias_stride < 0) return VQ_ERR_INVALID_ARG;
  for (int m = 0; m < E->L.nb; ++m) {
    if (d->idx_stride[m] < 0 || d->codebook_stride[m] < 0) return VQ_ERR_INVALID_ARG;
    if (d->idx_stride[m] % 4 != 0 || d->codebook_stride[m] % 8 != 0) return VQ_ERR_ALIGNMENT;
    E->si[m] = d->idx_stride[m];
    E->sb[m] = d->codebook_stride[m];
  }
  if (E->L.nb == 1) {
    E->si[1] = E->si[0];
    E->sb[1] = E->sb[0];
  }
  E->e = d->n_experts;
  E->ss = d->scale_stride;
  E->st = d->bias_stride;
  E->so = d->out_bias_stride;
  return VQ_OK;
}

size_t experts_bytes(const Experts& E, int m) { return 256; }

vq_status launch_gemm_experts(const Experts& E, const void* x, bool x_fp16, int x_rows, int64_t ldx,
                              const int32_t* rows, const int32_t* offsets, int m, void* y, vq_dtype yt, int64_t ldy,
                              void* ws, cudaStream_t stream) {
  count_launch();
  gemm_experts_kernel<<<dim3((E.L.n + 127) / 128, std::min(m, 65535)), 128, 0, stream>>>(
      E, static_cast<const uint16_t*>(x), x_fp16 ? 1 : 0, x_rows, ldx, rows, offsets, m, y, yt, ldy);
  return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace vqk

using namespace vqk;

extern "C" {

vq_status vq_gemm_experts_workspace_size(const vq_experts_desc* experts, int32_t m, size_t* bytes) {
  Experts E;
  if (!bytes) return VQ_ERR_INVALID_ARG;
  vq_status st = check_experts(experts, &E);
  if (st != VQ_OK) return st;
  if (m < 0) return VQ_ERR_INVALID_ARG;
  if (m > kMaxGroupedRows) return VQ_ERR_UNSUPPORTED;
  *bytes = m == 0 || E.L.n == 0 ? 0 : experts_bytes(E, m);
  return VQ_OK;
}

vq_status vq_gemm_experts(const vq_experts_desc* experts, const void* x, vq_dtype x_dtype, int32_t x_rows,
                          int64_t ldx, const int32_t* rows, const int32_t* offsets, int32_t m, void* y,
                          vq_dtype y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  Experts E;
  vq_status st = check_experts(experts, &E);
  if (st != VQ_OK) return st;
  if (m < 0 || x_rows < 0 || !(x_dtype == VQ_BF16 || x_dtype == VQ_FP16) ||
      !(y_dtype == VQ_BF16 || y_dtype == VQ_FP16 || y_dtype == VQ_FP32) || ldx < E.L.kin || ldy < E.L.n)
    return VQ_ERR_INVALID_ARG;
  if (m > kMaxGroupedRows) return VQ_ERR_UNSUPPORTED;
  if (!rows && x_rows < m) return VQ_ERR_INVALID_ARG;
  if (m == 0 || E.L.n == 0) return VQ_OK;
  if (!y || !offsets || (!x && x_rows > 0 && E.L.kin > 0)) return VQ_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(y, y_dtype == VQ_FP32 ? 4 : 2))
    return VQ_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < experts_bytes(E, m)) return VQ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return VQ_ERR_ALIGNMENT;
  return launch_gemm_experts(E, x, x_dtype == VQ_FP16, x_rows, ldx, rows, offsets, m, y, y_dtype, ldy, workspace,
                             static_cast<cudaStream_t>(stream));
}

}  // extern "C"
