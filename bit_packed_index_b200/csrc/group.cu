// group.cu -- vq_group_rows and vq_combine_rows: a router's picks put in the
// order of their experts, and the experts' results added up per token.
//
// Grouping is a stable counting sort, pos(p) = #{picks of smaller experts} +
// #{earlier picks of the same expert}, in one launch: a cluster of up to sixteen
// CTAs shares the picks, each warp owning a run of consecutive ones.
//   1. every warp counts its run into a histogram of its own (shared memory);
//   2. a scan over the warps, the CTAs (their totals through distributed
//      shared memory) and the experts turns the counts into first rows;
//   3. every warp walks its run again, 32 picks at a time: match.any gives the
//      lanes with the same expert, so a lane's rank is the count of lower ones.
// No atomic decides an order, so the result is the same on every run.  Picks
// and results are a few hundred KB at most and stay in L2: the call's time is
// its three dependent passes, which is why it is one launch.
//
// Combining reads every picked row once and writes every token once (HBM is
// the bound for a prefill chunk); a thread owns eight columns of a token and
// issues the loads of several picks before the first sum, past the caches'
// keeping (each row is read once).
#include <algorithm>
#include <mutex>
#include <vector>

#include <cooperative_groups.h>

#include "vq_experts.h"
#include "vq_internal.cuh"

namespace vqk {
namespace {

namespace cg = cooperative_groups;

constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;

size_t group_smem(int n_experts) {
  return (static_cast<size_t>(kGroupWarps + 3) * n_experts + 64) * sizeof(int);
}

// n / d for n < 2^30 (d >= 1) as a multiplication.
struct Divisor {
  uint32_t mul;
  int shift;
};
Divisor divisor(uint32_t d) {
  int s = 0;
  while ((1u << s) < d) ++s;
  return {static_cast<uint32_t>((((1ull << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ int quotient(int n, Divisor d) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), d.mul) + static_cast<uint32_t>(n)) >> d.shift);
}

constexpr int kHeld = 8;      // passes of a run whose ids stay in registers between counting and placing

__global__ void __launch_bounds__(kGroupThreads) group_rows_kernel(const int32_t* __restrict__ ids, int n_tokens,
                                                                  int top_k, Divisor by_k, int64_t ld_ids, int n_experts,
                                                                  int32_t* __restrict__ offsets,
                                                                  int32_t* __restrict__ rows,
                                                                  int32_t* __restrict__ pos) {
  extern __shared__ int s_mem[];
  int* hist = s_mem;                                   // [warp][expert]
  int* total = hist + kGroupWarps * n_experts;         // this CTA's picks per expert (read by the cluster)
  int* first = total + n_experts;                      // first row of this CTA's picks of an expert
  int* scan = first + n_experts;                       // [32] warp sums of the scan, [1] the number of rows
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = static_cast<int>(cluster.num_blocks()), c = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int picks = n_tokens * top_k;
  const int nw = nc * kGroupWarps;
  const int run = (picks + nw * 32 - 1) / (nw * 32) * 32;   // picks of a warp, a multiple of 32
  const int p0 = static_cast<int>(min(static_cast<int64_t>(picks), static_cast<int64_t>(c * kGroupWarps + warp) * run));
  const int p1 = static_cast<int>(min(static_cast<int64_t>(picks), static_cast<int64_t>(p0) + run));
  int* mine = hist + warp * n_experts;

  // the id of pick p, or -1 where it names no expert (or there is no pick p)
  auto load = [&](int p) {
    if (p >= p1) return -1;
    int64_t at = p;
    if (ld_ids != top_k) {
      const int t = quotient(p, by_k);
      at = t * ld_ids + (p - t * top_k);
    }
    const int id = __ldg(ids + at);
    return id >= 0 && id < n_experts ? id : -1;
  };
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = load(p0 + 32 * i + lane);
  for (int i = tid; i < kGroupWarps * n_experts; i += kGroupThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (held[i] >= 0) atomicAdd(&mine[held[i]], 1);
  for (int p = p0 + 32 * kHeld + lane; p < p1; p += 32) {
    const int id = load(p);
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  if (tid < n_experts) {                               // exclusive over the warps
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kGroupWarps; ++w) {
      const int v = hist[w * n_experts + tid];
      hist[w * n_experts + tid] = sum;
      sum += v;
    }
    total[tid] = sum;
  }
  cluster.sync();
  int all = 0, below = 0;
  if (tid < n_experts) {
#pragma unroll 8
    for (int k = 0; k < nc; ++k) {
      const int v = *cluster.map_shared_rank(total + tid, k);
      below += k < c ? v : 0;
      all += v;
    }
  }
  // exclusive scan of `all` over the experts (one per thread)
  int incl = all;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int v = scan[lane];
    int s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += u;
    }
    scan[lane] = s - v;
    if (lane == 31) scan[32] = s;
  }
  __syncthreads();
  const int excl = scan[warp] + incl - all;
  if (tid < n_experts) {
    first[tid] = excl + below;
    if (c == 0) offsets[tid] = excl;
  }
  const int n_rows = scan[32];
  if (c == 0 && tid == 0) offsets[n_experts] = n_rows;
  cluster.sync();                                      // `first` is set, and no CTA leaves while others read `total`
  // 32 picks in order: every pick's row is the expert's next one plus the lower
  // lanes with the same expert; the highest of them moves the expert on
  auto place = [&](int p, int id) {
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int r = -1;
    if (id >= 0) r = first[id] + mine[id] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && (same >> lane) == 1u) mine[id] += __popc(same);
    __syncwarp();
    if (p < p1) {
      pos[p] = r;
      if (id >= 0) rows[r] = quotient(p, by_k);
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (p0 + 32 * i < p1) place(p0 + 32 * i + lane, held[i]);
  for (int q = p0 + 32 * kHeld; q < p1; q += 32) place(q + lane, load(q + lane));
  for (int64_t i = n_rows + static_cast<int64_t>(c) * kGroupThreads + tid; i < picks; i += static_cast<int64_t>(nc) * kGroupThreads)
    rows[i] = -1;
}

template <typename T>
struct Load8;   // eight consecutive values as fp32
template <>
struct Load8<__half> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = h2f(static_cast<uint16_t>(w[i] & 0xFFFFu));
      v[2 * i + 1] = h2f(static_cast<uint16_t>(w[i] >> 16));
    }
  }
};
template <>
struct Load8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Load8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

template <typename T>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(p)[i];
  else if constexpr (std::is_same<T, __half>::value) return h2f(reinterpret_cast<const uint16_t*>(p)[i]);
  else return bf2f(reinterpret_cast<const uint16_t*>(p)[i]);
}

constexpr int kCombineThreads = 256;
// Picks whose loads are in flight together, and blocks per SM.  8192 tokens x 8
// picks x 4096 columns (cold): 8 and 2 took 124 us, 8 and 4 108, 4 and 6 142, 4
// and 4 103, 4 and 5 102 us (5.9 TB/s); 2048 x 2 x 8192: 52, 40, 44, 31, 29 us.
constexpr int kCombineAhead = 4;
constexpr int kCombineBlocks = 5;

// One group of eight columns of a token per thread; VEC: rows of z (and y)
// start on 16 bytes, so whole groups move as 16-byte words.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kCombineThreads, kCombineBlocks) combine_rows_kernel(
    const T* __restrict__ z, int z_rows, int n, int64_t ldz, const int32_t* __restrict__ pos,
    const float* __restrict__ weight, int64_t ld_weight, int n_tokens, int top_k, void* __restrict__ y, vq_dtype yt,
    int64_t ldy) {
  const int groups = n / 8 + (n % 8 != 0);
  const int64_t total = static_cast<int64_t>(n_tokens) * groups;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kCombineThreads) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kCombineThreads) {
    const int t = static_cast<int>(i / groups);
    const int c = static_cast<int>(i - static_cast<int64_t>(t) * groups) * 8;
    const int32_t* pt = pos + static_cast<int64_t>(t) * top_k;
    const float* wt = weight + t * ld_weight;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    if (VEC && n - c >= 8) {
      for (int j0 = 0; j0 < top_k; j0 += kCombineAhead) {
        Load8<T> q[kCombineAhead];
        float w[kCombineAhead];
        bool ok[kCombineAhead];
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j) {
          const int r = j0 + j < top_k ? __ldg(pt + j0 + j) : -1;
          ok[j] = r >= 0 && r < z_rows;
          if (ok[j]) {
            w[j] = __ldg(wt + j0 + j);
            q[j].load(z + r * ldz + c);
          }
        }
#pragma unroll
        for (int j = 0; j < kCombineAhead; ++j) {
          if (!ok[j]) continue;
          float v[8];
          q[j].get(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[j], v[e], acc[e]);
        }
      }
      if (yt == VQ_FP32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(y) + t * ldy + c);
        d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      } else {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          p[e] = yt == VQ_FP16 ? f2h(acc[2 * e]) | (static_cast<uint32_t>(f2h(acc[2 * e + 1])) << 16)
                               : f2bf(acc[2 * e]) | (static_cast<uint32_t>(f2bf(acc[2 * e + 1])) << 16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + t * ldy + c) = make_uint4(p[0], p[1], p[2], p[3]);
      }
    } else {
      const int live = min(8, n - c);
      for (int j = 0; j < top_k; ++j) {
        const int r = __ldg(pt + j);
        if (r < 0 || r >= z_rows) continue;
        const float w = __ldg(wt + j);
        for (int e = 0; e < live; ++e) acc[e] = fmaf(w, load1<T>(z, r * ldz + c + e), acc[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < live) store_out(y, yt, t * ldy + c + e, acc[e]);
    }
  }
}

template <typename T>
cudaError_t launch_combine(bool vec, const void* z, int z_rows, int n, int64_t ldz, const int32_t* pos,
                           const float* weight, int64_t ld_weight, int n_tokens, int top_k, void* y, vq_dtype yt,
                           int64_t ldy, cudaStream_t stream) {
  auto k = vec ? combine_rows_kernel<T, true> : combine_rows_kernel<T, false>;
  const int64_t total = static_cast<int64_t>(n_tokens) * ((static_cast<int64_t>(n) + 7) / 8);
  const int64_t most = static_cast<int64_t>(device_sm_count()) *
                       resident_blocks_per_sm(reinterpret_cast<const void*>(k), kCombineThreads, 0) * 8;
  const int grid = static_cast<int>(std::min<int64_t>((total + kCombineThreads - 1) / kCombineThreads, most));
  count_launch();
  k<<<grid, kCombineThreads, 0, stream>>>(static_cast<const T*>(z), z_rows, n, ldz, pos, weight, ld_weight, n_tokens,
                                          top_k, y, yt, ldy);
  return cudaGetLastError();
}

// Whether a cluster of sixteen CTAs with this much shared memory fits the
// current device (remembered per device and size).
bool wide_clusters(size_t smem) {
  struct Entry {
    int dev;
    size_t smem;
    bool ok;
  };
  static std::mutex mu;
  static std::vector<Entry> known;
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : known)
      if (e.dev == dev && e.smem == smem) return e.ok;
  }
  const void* k = reinterpret_cast<const void*>(group_rows_kernel);
  bool ok = set_func_attr(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  if (ok) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kGroupThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    ok = cudaOccupancyMaxActiveClusters(&n, group_rows_kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();   // leave no error for the launch to report
  }
  std::lock_guard<std::mutex> lock(mu);
  known.push_back({dev, smem, ok});
  return ok;
}

// One pick per thread and pass is the least a CTA can do; more CTAs pay once
// a warp's run is longer than a few passes (the two cluster barriers cost
// about as much as two passes).
// Sixteen CTAs (more than a portable cluster) halve the time of long runs,
// which scattered stores bound, where the device can place them.
int group_ctas(int64_t picks, size_t smem) {
  int c = 1;
  while (c < 16 && picks > static_cast<int64_t>(c) * kGroupThreads * 2) c *= 2;
  return c == 16 && !wide_clusters(smem) ? 8 : c;
}

bool float_type(vq_dtype t) { return t == VQ_BF16 || t == VQ_FP16 || t == VQ_FP32; }
size_t type_size(vq_dtype t) { return t == VQ_FP32 ? 4 : 2; }

}  // namespace
}  // namespace vqk

using namespace vqk;

extern "C" {

vq_status vq_group_rows(const int32_t* ids, int32_t n_tokens, int32_t top_k, int64_t ld_ids, int32_t n_experts,
                        int32_t* offsets, int32_t* rows, int32_t* pos, void* stream) {
  if (n_tokens < 0 || top_k < 1 || ld_ids < top_k || n_experts < 1) return VQ_ERR_INVALID_ARG;
  if (n_experts > VQ_MAX_EXPERTS || top_k > VQ_MAX_TOP_K) return VQ_ERR_UNSUPPORTED;
  const int64_t picks = static_cast<int64_t>(n_tokens) * top_k;
  if (picks > (1 << 30)) return VQ_ERR_UNSUPPORTED;
  if (!offsets || (picks > 0 && (!ids || !rows || !pos))) return VQ_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4)) return VQ_ERR_ALIGNMENT;
  const size_t smem = group_smem(n_experts);
  cudaError_t e = set_func_attr(reinterpret_cast<const void*>(group_rows_kernel),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_status(e);
  const int nc = group_ctas(picks, smem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cuda_status(cudaLaunchKernelEx(&cfg, group_rows_kernel, ids, static_cast<int>(n_tokens),
                                        static_cast<int>(top_k), divisor(static_cast<uint32_t>(top_k)), ld_ids,
                                        static_cast<int>(n_experts), offsets, rows, pos));
}

vq_status vq_combine_rows(const void* z, vq_dtype z_dtype, int32_t z_rows, int32_t n, int64_t ldz, const int32_t* pos,
                          const float* weight, int64_t ld_weight, int32_t n_tokens, int32_t top_k, void* y,
                          vq_dtype y_dtype, int64_t ldy, void* stream) {
  if (z_rows < 0 || n < 0 || n_tokens < 0 || top_k < 1 || ldz < n || ldy < n || ld_weight < top_k ||
      !float_type(z_dtype) || !float_type(y_dtype))
    return VQ_ERR_INVALID_ARG;
  if (top_k > VQ_MAX_TOP_K) return VQ_ERR_UNSUPPORTED;
  if (n_tokens == 0 || n == 0) return VQ_OK;
  if (!y || !pos || !weight || (!z && z_rows > 0)) return VQ_ERR_INVALID_ARG;
  if (!aligned(z, type_size(z_dtype)) || !aligned(y, type_size(y_dtype)) || !aligned(pos, 4) || !aligned(weight, 4))
    return VQ_ERR_ALIGNMENT;
  const bool vec = aligned(z, 16) && aligned(y, 16) && ldz * type_size(z_dtype) % 16 == 0 &&
                   ldy * type_size(y_dtype) % 16 == 0;
  auto run = z_dtype == VQ_FP32 ? launch_combine<float>
                                : (z_dtype == VQ_FP16 ? launch_combine<__half> : launch_combine<__nv_bfloat16>);
  return cuda_status(run(vec, z, z_rows, n, ldz, pos, weight, ld_weight, n_tokens, top_k, y, y_dtype, ldy,
                         static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
