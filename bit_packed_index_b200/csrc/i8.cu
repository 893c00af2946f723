// i8.cu -- linear layers in 8-bit integers: vq_quant_i8, vq_gemm_i8,
// vq_linear_i8.
//
// Quantisation of a row (include/vq_i8.h): s = fp32(max|x| / 127) and q =
// rne(x / s) of the exact quotient.  The kernel multiplies by 1 / s instead of
// dividing: |x / s| <= 127 (1 + 2^-23), and the product's error is below 127 *
// 2^-22 < 4e-5, so the nearest integer is right unless the product lies within
// 1e-4 of a half.  There the sign of x - (n + 1/2) s decides, which one fused
// multiply-add gives exactly (its only rounding cannot change a sign).  One
// element in 5000 takes that path; the kernel stays at the memory's speed.
#include <algorithm>

#include "vq_i8.h"
#include "vq_internal.cuh"

namespace vqk {
namespace {

// ---------------------------------------------------------------------------
// Quantisation.
// ---------------------------------------------------------------------------

// Below this scale (rows whose largest value is under 127 * 2^-100) 1 / s and
// the products of the exact test could leave fp32's normal range: such rows
// divide in fp64, whose 53 bits separate any quotient of a 24-bit scale and an
// 11-bit value from a half-integer that it is not equal to.
constexpr float kTinyScale = 7.888609052210118e-31f;   // 2^-100

__device__ __forceinline__ int quant_one(float x, float s, float inv) {
  if (s < kTinyScale) {
    if (s == 0.0f) return 0;
    const double r = rint(static_cast<double>(x) / static_cast<double>(s));
    return static_cast<int>(fmin(127.0, fmax(-127.0, r)));
  }
  const float t = x * inv;
  float r = rintf(t);
  if (fabsf(t - r) > 0.4999f) {
    const float lo = floorf(t);
    const float d = fmaf(-(lo + 0.5f), s, x);     // sign of x - (lo + 1/2) s
    const float even = (static_cast<int>(lo) & 1) ? lo + 1.0f : lo;
    r = d > 0.0f ? lo + 1.0f : (d < 0.0f ? lo : even);
  }
  return static_cast<int>(fminf(127.0f, fmaxf(-127.0f, r)));
}

template <bool FP16>
__device__ __forceinline__ float val16(uint32_t bits) {
  return FP16 ? h2f(static_cast<uint16_t>(bits)) : __uint_as_float(bits << 16);
}

// The scale of a row from the largest |x| as 16-bit pattern: NaN where the
// row holds an infinity or a NaN (all-ones exponent).
template <bool FP16>
__device__ __forceinline__ float row_scale(uint32_t top) {
  if (top >= (FP16 ? 0x7C00u : 0x7F80u)) return __uint_as_float(0x7FC00000u);
  return __fdiv_rn(val16<FP16>(top), 127.0f);
}

// One row per block.  V > 0: rows of at most blockDim * V groups of eight
// values stay in registers between the maximum and the rounding.  V = 0: rows
// of any length or alignment, read twice value by value (the second time from
// the caches).
template <bool FP16, int V>
__global__ void __launch_bounds__(1024) quant_i8_kernel(const uint16_t* __restrict__ x, int n, int64_t ldx,
                                                        int8_t* __restrict__ q, int64_t ldq,
                                                        float* __restrict__ scale) {
  __shared__ uint32_t s_top[32];
  const int64_t row = blockIdx.x;
  const uint16_t* xr = x + row * ldx;
  int8_t* qr = q + row * ldq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t top = 0;                                   // two 16-bit maxima of |x|
  uint4 u[V > 0 ? V : 1];
  if constexpr (V > 0) {
    const int groups = (n + 7) / 8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = v * blockDim.x + tid;
      u[v] = make_uint4(0u, 0u, 0u, 0u);
      if (g < groups) {
        if (8 * g + 8 <= n) {
          u[v] = __ldg(reinterpret_cast<const uint4*>(xr) + g);
        } else {                                      // the last values of a row
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * g + e < n) w[e >> 1] |= static_cast<uint32_t>(__ldg(xr + 8 * g + e)) << (16 * (e & 1));
          u[v] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      top = __vmaxu2(top, __vmaxu2(u[v].x & 0x7FFF7FFFu, u[v].y & 0x7FFF7FFFu));
      top = __vmaxu2(top, __vmaxu2(u[v].z & 0x7FFF7FFFu, u[v].w & 0x7FFF7FFFu));
    }
  } else {
    for (int k = tid; k < n; k += blockDim.x) top = max(top, static_cast<uint32_t>(__ldg(xr + k)) & 0x7FFFu);
  }
  top = max(top & 0xFFFFu, top >> 16);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  top = lane < static_cast<int>(blockDim.x >> 5) ? s_top[lane] : 0u;
  top = __reduce_max_sync(0xffffffffu, top);
  float s = row_scale<FP16>(top);
  if (tid == 0) scale[row] = s;
  const bool bad = !(s == s);
  if (bad) s = 0.0f;                                  // q = 0
  const float inv = s >= kTinyScale ? __fdiv_rn(1.0f, s) : 0.0f;
  if constexpr (V > 0) {
    const int groups = (n + 7) / 8;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = v * blockDim.x + tid;
      if (g >= groups) continue;
      const uint32_t w[4] = {u[v].x, u[v].y, u[v].z, u[v].w};
      uint32_t p[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = quant_one(val16<FP16>((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu), s, inv);
        p[e >> 2] |= (static_cast<uint32_t>(i) & 0xFFu) << (8 * (e & 3));
      }
      if (8 * g + 8 <= n) {
        *reinterpret_cast<uint2*>(qr + 8 * g) = make_uint2(p[0], p[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * g + e < n) qr[8 * g + e] = static_cast<int8_t>((p[e >> 2] >> (8 * (e & 3))) & 0xFFu);
      }
    }
  } else {
    for (int k = tid; k < n; k += blockDim.x)
      qr[k] = static_cast<int8_t>(quant_one(val16<FP16>(__ldg(xr + k)), s, inv));
  }
}

template <bool FP16>
cudaError_t launch_quant(const uint16_t* x, int rows, int n, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                         cudaStream_t stream) {
  const bool vec = aligned(x, 16) && ldx % 8 == 0 && aligned(q, 8) && ldq % 8 == 0;
  const int groups = (n + 7) / 8;
  // threads: about two groups each, so that a row's loads are all in flight
  // and short rows leave room for many blocks
  int threads = 64;
  while (threads < 1024 && threads * 2 < groups) threads *= 2;
  const int v = (groups + threads - 1) / threads;
  count_launch();
#define VQ_QUANT(V) quant_i8_kernel<FP16, V><<<rows, threads, 0, stream>>>(x, n, ldx, q, ldq, scale)
  if (!vec || v > 8) VQ_QUANT(0);
  else if (v <= 1) VQ_QUANT(1);
  else if (v <= 2) VQ_QUANT(2);
  else if (v <= 4) VQ_QUANT(4);
  else VQ_QUANT(8);
#undef VQ_QUANT
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Product.
// ---------------------------------------------------------------------------
struct I8Layer {
  int n, kin;
  const int8_t* w;
  int64_t ldw;
  const float* scale;
  const uint16_t* ob;
};

constexpr int kTile = 64;     // outputs and rows of a block
constexpr int kStep = 64;     // bytes of k per step

// y tile of 64 rows x 64 outputs per block of 256 threads, four by four per
// thread, dp4a on words staged in shared memory.
__global__ void __launch_bounds__(256) gemm_i8_kernel(I8Layer L, const int8_t* __restrict__ q, int64_t ldq,
                                                      const float* __restrict__ qs, int m, void* __restrict__ y,
                                                      vq_dtype yt, int64_t ldy) {
  __shared__ int sa[kTile][kStep / 4 + 1], sb[kTile][kStep / 4 + 1];
  const int o0 = blockIdx.x * kTile, i0 = blockIdx.y * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < L.kin; k0 += kStep) {
    for (int w = threadIdx.x; w < kTile * (kStep / 4); w += 256) {
      const int r = w / (kStep / 4), c = w % (kStep / 4);
      const int k = k0 + 4 * c;
      int a = 0, b = 0;
      if (k < L.kin) {
        const int keep = min(4, L.kin - k);
        const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        if (i0 + r < m) a = *reinterpret_cast<const int*>(q + (i0 + r) * ldq + k) & mask;
        if (o0 + r < L.n) b = *reinterpret_cast<const int*>(L.w + (o0 + r) * L.ldw + k) & mask;
      }
      sa[r][c] = a;
      sb[r][c] = b;
    }
    __syncthreads();
    for (int c = 0; c < kStep / 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(sa[ty + 16 * i][c], sb[tx + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ty + 16 * i, o = o0 + tx + 16 * j;
      if (r < m && o < L.n)
        store_out(y, yt, r * ldy + o, (__int2float_rn(acc[i][j]) * L.scale[o]) * qs[r] + out_bias_of(L.ob, o));
    }
}

vq_status check_i8(const vq_i8_desc* d, I8Layer* L) {
  if (!d || d->out_features < 0 || d->in_features < 0 || d->ldw < d->in_features) return VQ_ERR_INVALID_ARG;
  if (d->in_features > VQ_I8_MAX_IN_FEATURES) return VQ_ERR_UNSUPPORTED;
  if (d->out_features > 0) {
    if (!d->scale || (!d->w && d->in_features > 0)) return VQ_ERR_INVALID_ARG;
    if (d->in_features > 0 && (!aligned(d->w, 16) || d->ldw % 16 != 0)) return VQ_ERR_ALIGNMENT;
    if (!aligned(d->scale, 4) || !aligned(d->out_bias, 2)) return VQ_ERR_ALIGNMENT;
  }
  *L = {d->out_features, d->in_features, d->w, d->ldw, d->scale, d->out_bias};
  return VQ_OK;
}

constexpr int kMaxRows = 1 << 30;
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
bool type16(vq_dtype t) { return t == VQ_BF16 || t == VQ_FP16; }

size_t gemm_i8_bytes(const I8Layer& L, int m) { return 256; }

// Where vq_linear_i8 keeps q and its scales behind vq_gemm_i8's workspace.
struct LinearLayout {
  int64_t ldq;
  size_t off_scale, off_q, total;
};
LinearLayout linear_layout(const I8Layer& L, int m) {
  LinearLayout l;
  l.ldq = (static_cast<int64_t>(L.kin) + 15) / 16 * 16;
  l.off_scale = round256(gemm_i8_bytes(L, m));
  l.off_q = l.off_scale + round256(static_cast<size_t>(m) * 4);
  l.total = l.off_q + round256(static_cast<size_t>(m) * l.ldq);
  return l;
}

vq_status launch_gemm_i8(const I8Layer& L, const int8_t* q, int64_t ldq, const float* qs, int m, void* y, vq_dtype yt,
                         int64_t ldy, void* ws, cudaStream_t stream) {
  count_launch();
  gemm_i8_kernel<<<dim3((L.n + kTile - 1) / kTile, (m + kTile - 1) / kTile), 256, 0, stream>>>(L, q, ldq, qs, m, y, yt,
                                                                                              ldy);
  return cuda_status(cudaGetLastError());
}

vq_status check_out(const I8Layer& L, int m, void* y, vq_dtype yt, int64_t ldy) {
  if (m < 0 || !(type16(yt) || yt == VQ_FP32) || ldy < L.n) return VQ_ERR_INVALID_ARG;
  if (m > kMaxRows) return VQ_ERR_UNSUPPORTED;
  if (m > 0 && L.n > 0) {
    if (!y) return VQ_ERR_INVALID_ARG;
    if (!aligned(y, yt == VQ_FP32 ? 4 : 2)) return VQ_ERR_ALIGNMENT;
  }
  return VQ_OK;
}

vq_status check_workspace(void* ws, size_t have, size_t need) {
  if (!ws || have < need) return VQ_ERR_WORKSPACE;
  return aligned(ws, 256) ? VQ_OK : VQ_ERR_ALIGNMENT;
}

}  // namespace
}  // namespace vqk

using namespace vqk;

extern "C" {

vq_status vq_quant_i8(const void* x, vq_dtype x_dtype, int32_t rows, int32_t n, int64_t ldx, int8_t* q, int64_t ldq,
                      float* scale, void* stream) {
  if (rows < 0 || n < 0 || ldx < n || ldq < n || !type16(x_dtype)) return VQ_ERR_INVALID_ARG;
  if (rows == 0) return VQ_OK;
  if (!scale || (n > 0 && (!x || !q))) return VQ_ERR_INVALID_ARG;
  if (!aligned(x, 2) || !aligned(scale, 4)) return VQ_ERR_ALIGNMENT;
  auto run = x_dtype == VQ_FP16 ? launch_quant<true> : launch_quant<false>;
  return cuda_status(run(static_cast<const uint16_t*>(x), rows, n, ldx, q, ldq, scale,
                         static_cast<cudaStream_t>(stream)));
}

vq_status vq_gemm_i8_workspace_size(const vq_i8_desc* layer, int32_t m, size_t* bytes) {
  I8Layer L;
  if (!bytes) return VQ_ERR_INVALID_ARG;
  vq_status st = check_i8(layer, &L);
  if (st != VQ_OK) return st;
  if (m < 0) return VQ_ERR_INVALID_ARG;
  if (m > kMaxRows) return VQ_ERR_UNSUPPORTED;
  *bytes = m == 0 || L.n == 0 ? 0 : gemm_i8_bytes(L, m);
  return VQ_OK;
}

vq_status vq_gemm_i8(const vq_i8_desc* layer, const int8_t* q, int64_t ldq, const float* q_scale, int32_t m, void* y,
                     vq_dtype y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  I8Layer L;
  vq_status st = check_i8(layer, &L);
  if (st == VQ_OK) st = check_out(L, m, y, y_dtype, ldy);
  if (st != VQ_OK) return st;
  if (ldq < L.kin) return VQ_ERR_INVALID_ARG;
  if (m == 0 || L.n == 0) return VQ_OK;
  if (!q_scale || (!q && L.kin > 0)) return VQ_ERR_INVALID_ARG;
  if ((L.kin > 0 && (!aligned(q, 16) || ldq % 16 != 0)) || !aligned(q_scale, 4)) return VQ_ERR_ALIGNMENT;
  st = check_workspace(workspace, workspace_bytes, gemm_i8_bytes(L, m));
  if (st != VQ_OK) return st;
  return launch_gemm_i8(L, q, ldq, q_scale, m, y, y_dtype, ldy, workspace, static_cast<cudaStream_t>(stream));
}

vq_status vq_linear_i8_workspace_size(const vq_i8_desc* layer, int32_t m, size_t* bytes) {
  I8Layer L;
  if (!bytes) return VQ_ERR_INVALID_ARG;
  vq_status st = check_i8(layer, &L);
  if (st != VQ_OK) return st;
  if (m < 0) return VQ_ERR_INVALID_ARG;
  if (m > kMaxRows) return VQ_ERR_UNSUPPORTED;
  *bytes = m == 0 || L.n == 0 ? 0 : linear_layout(L, m).total;
  return VQ_OK;
}

vq_status vq_linear_i8(const vq_i8_desc* layer, const void* x, vq_dtype x_dtype, int32_t m, int64_t ldx, void* y,
                       vq_dtype y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  I8Layer L;
  vq_status st = check_i8(layer, &L);
  if (st == VQ_OK) st = check_out(L, m, y, y_dtype, ldy);
  if (st != VQ_OK) return st;
  if (ldx < L.kin || !type16(x_dtype)) return VQ_ERR_INVALID_ARG;
  if (m == 0 || L.n == 0) return VQ_OK;
  if (!x && L.kin > 0) return VQ_ERR_INVALID_ARG;
  if (!aligned(x, 2)) return VQ_ERR_ALIGNMENT;
  const LinearLayout lay = linear_layout(L, m);
  st = check_workspace(workspace, workspace_bytes, lay.total);
  if (st != VQ_OK) return st;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  int8_t* q = reinterpret_cast<int8_t*>(w + lay.off_q);
  float* qs = reinterpret_cast<float*>(w + lay.off_scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto run = x_dtype == VQ_FP16 ? launch_quant<true> : launch_quant<false>;
  st = cuda_status(run(static_cast<const uint16_t*>(x), m, L.kin, ldx, q, lay.ldq, qs, s));
  if (st != VQ_OK) return st;
  return launch_gemm_i8(L, q, lay.ldq, qs, m, y, y_dtype, ldy, workspace, s);
}

}  // extern "C"
