// i8.cu -- linear layers in 8-bit integers: vq_quant_i8, vq_gemm_i8,
// vq_linear_i8.
//
// Quantisation of a row (include/vq_i8.h): s = fp32(max|x| / 127) and q =
// rne(x / s) of the exact quotient.  The kernel multiplies by 1 / s instead of
// dividing: |x / s| <= 127 (1 + 2^-23), and the product's error is below 127 *
// 2^-22 < 4e-5, so the nearest integer is right unless the product lies within
// 1e-4 of a half.  There the sign of x - (n + 1/2) s decides, which one fused
// multiply-add gives exactly (its only rounding cannot change a sign).  One
// element in 5000 takes that path.  Measured (B200, cold): 4096 x 8192 from bf16
// 33 us (3.0 TB/s, less than half of what memory gives: a row's two passes and
// two barriers leave little in flight); rows that do not start on 16 bytes are
// read value by value, 4096 x 8190 90 us (1.1 TB/s).
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "sm100.cuh"
#include "vq_i8.h"

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
  // the product after this kernel may start loading its weights
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.x;
  const uint16_t* xr = x + row * ldx;
  int8_t* qr = q + row * ldq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t top = 0;                                   // two 16-bit maxima of |x|
  uint4 u[V > 0 ? V : 1];
  if constexpr (V > 0) {
    const int groups = n / 8 + (n % 8 != 0);
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
    // (unsigned: k passes 2^31 behind the longest rows)
    for (uint32_t k = tid; k < static_cast<uint32_t>(n); k += blockDim.x)
      top = max(top, static_cast<uint32_t>(__ldg(xr + k)) & 0x7FFFu);
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
    const int groups = n / 8 + (n % 8 != 0);
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
    for (uint32_t k = tid; k < static_cast<uint32_t>(n); k += blockDim.x)
      qr[k] = static_cast<int8_t>(quant_one(val16<FP16>(__ldg(xr + k)), s, inv));
  }
}

template <bool FP16>
cudaError_t launch_quant(const uint16_t* x, int rows, int n, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                         cudaStream_t stream) {
  const bool vec = aligned(x, 16) && ldx % 8 == 0 && aligned(q, 8) && ldq % 8 == 0;
  const int groups = n / 8 + (n % 8 != 0);
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
// Product: y^T = W q^T on the integer tensor cores (tcgen05 kind::i8, exact
// 32-bit sums).  W's rows are the MMA's M and the activations' rows its N, so
// that one token and four thousand take the same path: a decode step is W
// streamed once past a narrow N.  Both operands come by TMA as 128-byte
// swizzled rows (128 values of k a step); rows and columns past the matrices
// read as zeros.  A thread of the epilogue owns one output channel, so its
// scale and bias are registers and a warp stores 32 neighbouring outputs of a
// token at a time.  Measured (B200, the product alone): 24 x 8192 x 8192 16.6 us
// (4.0 TB/s of weights, cold), 16 x 16384 x 16384 46 us (5.8 TB/s), 4096 x 8192 x
// 8192 159 to 167 us for a few calls (3.3 to 3.5 POP/s; tensor pipe 86 % busy at
// 2048 rows), 194 us (2.8 POP/s) once the power cap holds the clocks down.
// ---------------------------------------------------------------------------
using namespace sm100;

struct I8Layer {
  int n, kin;
  const int8_t* w;
  int64_t ldw;
  const float* scale;
  const uint16_t* ob;
};

struct I8Args {
  int n, m;               // outputs, activation rows
  int num_kt;             // steps of 128 values
  int tn;                 // activation rows per tile (MMA N)
  const float* ws;        // weight scales
  const uint16_t* ob;
  const float* qs;        // activation scales
  void* y;
  vq_dtype yt;
  int64_t ldy;
  int* status;
  long long budget;
  int split_log2;         // narrow kernel: log2 of the CTAs of a cluster
  int tiles_n, tiles_m;   // wide kernel: tiles of 256 outputs, of tn rows
  int stages;
};

constexpr int kRows = 128;                 // output channels per CTA
constexpr int kStepBytes = 128;            // values of k per step
constexpr int kWTile = kRows * kStepBytes;
constexpr int kMaxStages = 8;
constexpr int kCtrlBytes = 3 * 1024;       // control block in front of the stages (a multiple of 1024)
constexpr long long kDrain = 1LL << 26;    // SM clocks: far above any load's latency

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One output from its exact sum.
__device__ __forceinline__ float i8_out(int acc, float w, float s, float b) {
  return __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(acc), w), s), b);
}

// Outputs of one channel (its column in y: yo) for `n` of sixteen rows.  The
// output type is a template argument: the epilogue is one warp per scheduler,
// which a branch per value would keep longer than the products take.
template <int YT>
__device__ __forceinline__ void store_rows(uint8_t* yo, int64_t ldb, const uint32_t* acc, int n, const float4* scales,
                                           float w, float b) {
  using T = typename std::conditional<YT == VQ_FP32, float, uint16_t>::type;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 e = scales[i / 4];
    const float s[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = i8_out(static_cast<int>(acc[i + j]), w, s[j], b);
      T x;
      if constexpr (YT == VQ_FP32) x = v;
      else x = YT == VQ_FP16 ? f2h(v) : f2bf(v);
      if (i + j < n) *reinterpret_cast<T*>(yo + (i + j) * ldb) = x;
    }
  }
}
__device__ __forceinline__ void store_rows(vq_dtype yt, uint8_t* yo, int64_t ldb, const uint32_t* acc, int n,
                                           const float4* scales, float w, float b) {
  if (yt == VQ_BF16) store_rows<VQ_BF16>(yo, ldb, acc, n, scales, w, b);
  else if (yt == VQ_FP16) store_rows<VQ_FP16>(yo, ldb, acc, n, scales, w, b);
  else store_rows<VQ_FP32>(yo, ldb, acc, n, scales, w, b);
}

// ---- few rows: W's bytes are the bound ------------------------------------
// A cluster of S CTAs shares a tile of 128 outputs, each CTA a run of k, so
// that a layer of few outputs keeps up to eight times as many SMs loading (64 of
// 148 for 1024 outputs).  The partial sums meet in distributed shared memory: integers, so the split changes nothing
// in y, and no workspace, counter or second launch is needed.
struct NarrowCtrl {
  uint64_t full[kMaxStages], empty[kMaxStages], acc;
  uint32_t tmem;
  int abort;
  alignas(16) float scales[64];            // activation scales (kNarrowRows of them)
};
static_assert(sizeof(NarrowCtrl) <= kCtrlBytes, "control block");
// Rows up to which this kernel runs: 8192 x 8192 from bf16 takes 18.3 us here and
// 19.7 in the wide kernel for 24 rows, 19.6 and 20.6 for 48, 20.8 in both for 64
// (the product alone 19.3 and 17.8).
constexpr int kNarrowRows = 48;
constexpr int kNarrowThreads = 192;        // warp 0: loads, warp 1: products, warps 2-5: epilogue

__global__ void __launch_bounds__(kNarrowThreads) gemm_i8_narrow_kernel(const __grid_constant__ CUtensorMap wmap,
                                                                        const __grid_constant__ CUtensorMap xmap,
                                                                        I8Args g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1024(smem_raw);
  NarrowCtrl* ctrl = reinterpret_cast<NarrowCtrl*>(base);
  uint8_t* stages = base + kCtrlBytes;
  const int stage = kWTile + g.tn * kStepBytes;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int splits = gridDim.y, split = blockIdx.y;          // the cluster spans the grid's y
  const int row0 = blockIdx.x * kRows;
  const int kt0 = split * g.num_kt >> g.split_log2;          // even runs: they differ by a step at most
  const int nkt = ((split + 1) * g.num_kt >> g.split_log2) - kt0;
  int issued = 0;                                            // warp 0: steps loaded
  volatile int* abort_flag = &ctrl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    mbar_init(&ctrl->acc, 1);
    ctrl->abort = 0;
    fence_barrier_init();
    // the first weight tiles do not wait for the kernel before this one (the
    // quantisation of the activations)
    for (int i = 0; i < min(nkt, g.stages); ++i) {
      mbar_arrive_expect_tx(&ctrl->full[i], stage);
      tma_load_2d(stages + i * stage, &wmap, &ctrl->full[i], (kt0 + i) * kStepBytes, row0);
    }
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(ctrl->tmem);
  pdl_wait();

  if (warp == 0) {
    issued = min(nkt, g.stages);
    if (elect_one())
      for (int i = 0; i < issued; ++i)
        tma_load_2d(stages + i * stage + kWTile, &xmap, &ctrl->full[i], (kt0 + i) * kStepBytes, 0);
    __syncwarp();
    int s = 0, sp = 0;
    for (int i = issued; i < nkt; ++i) {
      if (!warp_wait(&ctrl->empty[s], sp, abort_flag, g.status, g.budget)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(&ctrl->full[s], stage);
        tma_load_2d(stages + s * stage, &wmap, &ctrl->full[s], (kt0 + i) * kStepBytes, row0);
        tma_load_2d(stages + s * stage + kWTile, &xmap, &ctrl->full[s], (kt0 + i) * kStepBytes, 0);
      }
      __syncwarp();
      issued = i + 1;
      if (++s == g.stages) {
        s = 0;
        sp ^= 1;
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = i8_idesc(kRows, g.tn);
    const uint64_t desc0 = sw128_kmajor_desc(smem_addr(stages));
    int s = 0, sp = 0;
    bool ready = false;
    for (int i = 0; i < nkt; ++i) {
      if (!ready && !warp_wait(&ctrl->full[s], sp, abort_flag, g.status, g.budget)) break;
      tc_fence_after();
      const uint64_t ad = desc0 + static_cast<uint32_t>(s * stage >> 4), bd = ad + (kWTile >> 4);
      uint64_t* free_bar = &ctrl->empty[s];
      if (++s == g.stages) {
        s = 0;
        sp ^= 1;
      }
      const bool next = mbar_test_wait(&ctrl->full[s], sp);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kStepBytes / 32; ++kk) umma_i8(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (i | kk) != 0);
        umma_commit(free_bar);
      }
      ready = __all_sync(0xffffffffu, next) && i + 1 < nkt;
    }
    if (elect_one()) {
      umma_commit(&ctrl->acc);
      drain_phase(&ctrl->acc, 0, kDrain);                    // nothing runs in tensor memory after this
    }
  } else {
    const int lq = warp & 3, r = 32 * lq + lane, o = row0 + r;
    if (r < kNarrowRows) ctrl->scales[r] = r < g.m ? g.qs[r] : 0.0f;
    const bool ok = warp_wait(&ctrl->acc, 0, abort_flag, g.status, g.budget);
    asm volatile("bar.sync 1, 128;" ::: "memory");           // the scales of all rows are there
    tc_fence_after();
    const uint32_t t = tmem + (static_cast<uint32_t>(32 * lq) << 16);
    if (splits == 1) {
      const bool live = ok && o < g.n;
      const float w = live ? g.ws[o] : 0.0f, b = live ? out_bias_of(g.ob, o) : 0.0f;
      const int64_t ldb = g.ldy * (g.yt == VQ_FP32 ? 4 : 2);
      uint8_t* yo = static_cast<uint8_t*>(g.y) + static_cast<int64_t>(o) * (g.yt == VQ_FP32 ? 4 : 2);
      for (int c = 0; c < g.m; c += 16) {
        uint32_t acc[16];
        tmem_ld16(t + c, acc);
        tmem_wait_ld();
        if (live) store_rows(g.yt, yo + c * ldb, ldb, acc, g.m - c, reinterpret_cast<const float4*>(ctrl->scales + c), w, b);
      }
    } else if (ok) {
      // partial sums to the (spent) stage memory, [row of x][128]
      int* red = reinterpret_cast<int*>(stages);
      for (int c = 0; c < g.m; c += 16) {
        uint32_t acc[16];
        tmem_ld16(t + c, acc);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) red[(c + i) * kRows + r] = static_cast<int>(acc[i]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (splits > 1) {
    cluster_arrive();
    cluster_wait();
    // This CTA's share of the tile's outputs.  The activation scales come from
    // its table: the kernel may have started before the one that wrote them
    // ended, so they are not constant over its life and no load of constant
    // data (__ldg) may fetch them.
    const int total = g.m * kRows, share = (total + splits - 1) / splits;
    const int last = min(total, (split + 1) * share);
    if (!*abort_flag) {
      for (int i = split * share + threadIdx.x; i < last; i += kNarrowThreads) {
        const int* mine = reinterpret_cast<const int*>(stages) + i;
        int sum = 0;
        for (int s = 0; s < splits; ++s) {
          int v;
          asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(mine, s)) : "memory");
          sum += v;
        }
        const int c = i / kRows, o = row0 + (i & (kRows - 1));
        if (o < g.n) store_out(g.y, g.yt, c * g.ldy + o, i8_out(sum, g.ws[o], ctrl->scales[c], out_bias_of(g.ob, o)));
      }
    }
    cluster_arrive();                                        // no CTA leaves while others read its sums
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  // Loads in flight land before the block ends if some warp gave up: no warp
  // raises the flag behind the barrier above.  (The same wait where the loads
  // end, whether or not the flag is up, took 0.1 to 0.3 us of a call.)
  if (warp == 0 && *abort_flag && lane == 0)
    for (int i = max(0, issued - g.stages); i < issued; ++i)
      drain_phase(&ctrl->full[i % g.stages], (i / g.stages) & 1, kDrain);
}

// ---- more rows: the tensor cores are the bound ----------------------------------
// Persistent pairs of CTAs (cta_group::2): a tile is 256 outputs by up to 256
// rows, each CTA loading 128 rows of W and half the rows of q per step, so
// that shared memory feeds the products at half the bytes a lone CTA would
// need.  Two accumulators alternate in tensor memory: the epilogue of a tile
// runs under the products of the next.
struct WideCtrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t accf[2], acce[2];
  uint32_t tmem;
  int abort;
  alignas(16) float scales[2][256];        // activation scales of a tile's rows, two tiles in turn
};
static_assert(sizeof(WideCtrl) <= kCtrlBytes, "control block");
constexpr int kWideThreads = 256;          // warp 0: loads, warp 1: products, warps 4-7: epilogue
constexpr int kWideTn = 256;
constexpr uint32_t kWideCols = 512;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    gemm_i8_wide_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, I8Args g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = align1024(smem_raw);
  WideCtrl* ctrl = reinterpret_cast<WideCtrl*>(base);
  uint8_t* stages = base + kCtrlBytes;
  const int half = g.tn / 2;                                 // rows of q per CTA
  const int stage = kWTile + half * kStepBytes;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = g.tiles_n * g.tiles_m;
  volatile int* abort_flag = &ctrl->abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->accf[b], 1);
      mbar_init(&ctrl->acce[b], 8);                          // the epilogue warps of both CTAs
    }
    ctrl->abort = 0;
    fence_barrier_init();
    tma_prefetch(&wmap);
    tma_prefetch(&xmap);
  }
  if (warp == 2) {
    tmem_alloc_pair(&ctrl->tmem, kWideCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_arrive();                                          // both CTAs' barriers exist
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = uniform(ctrl->tmem);
  pdl_wait();

  if (warp == 0) {
    int s = 0, sp = 0, gs = 0;
    bool stop = false;
    for (int tile = pair; tile < tiles && !stop; tile += pairs) {
      const int row0 = (tile / g.tiles_m) * 2 * kRows + rank * kRows;
      const int t0 = (tile % g.tiles_m) * g.tn + rank * half;
      for (int i = 0; i < g.num_kt; ++i, ++gs) {
        if (!warp_wait(&ctrl->empty[s], sp ^ 1, abort_flag, g.status, g.budget)) {
          stop = true;
          break;
        }
        if (elect_one()) {
          const uint32_t bar = cluster_addr(&ctrl->full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&ctrl->full[s], 2 * stage);
          tma_load_2d_pair(stages + s * stage, &wmap, bar, i * kStepBytes, row0);
          tma_load_2d_pair(stages + s * stage + kWTile, &xmap, bar, i * kStepBytes, t0);
        }
        __syncwarp();
        if (++s == g.stages) {
          s = 0;
          sp ^= 1;
        }
      }
    }
    // the last products' arrivals on this CTA's barriers are in
    for (int i = max(0, gs - g.stages); i < gs && !stop; ++i)
      stop = !warp_wait(&ctrl->empty[i % g.stages], (i / g.stages) & 1, abort_flag, g.status, g.budget);
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = i8_idesc(2 * kRows, g.tn);
      const uint64_t desc0 = sw128_kmajor_desc(smem_addr(stages));
      int s = 0, sp = 0, it = 0;
      bool stop = false, ready = false;
      for (int tile = pair; tile < tiles && !stop; tile += pairs, ++it) {
        const int buf = it & 1;
        if (it >= 2 && !warp_wait(&ctrl->acce[buf], ((it >> 1) & 1) ^ 1, abort_flag, g.status, g.budget)) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * kWideTn;
        for (int i = 0; i < g.num_kt; ++i) {
          if (!ready && !warp_wait(&ctrl->full[s], sp, abort_flag, g.status, g.budget)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + static_cast<uint32_t>(s * stage >> 4), bd = ad + (kWTile >> 4);
          uint64_t* free_bar = &ctrl->empty[s];
          if (++s == g.stages) {
            s = 0;
            sp ^= 1;
          }
          const bool next = mbar_test_wait(&ctrl->full[s], sp);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kStepBytes / 32; ++kk) umma_i8_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, (i | kk) != 0);
            umma_commit_pair(free_bar);
          }
          ready = __all_sync(0xffffffffu, next);
        }
        if (!stop && elect_one()) umma_commit_pair(&ctrl->accf[buf]);
        __syncwarp();
      }
    }
  } else if (warp >= 4) {
    const int lq = warp & 3, r = 32 * lq + lane;
    const int64_t ldb = g.ldy * (g.yt == VQ_FP32 ? 4 : 2);
    int it = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++it) {
      const int buf = it & 1;
      const int o = (tile / g.tiles_m) * 2 * kRows + rank * kRows + r;
      const int t0 = (tile % g.tiles_m) * g.tn;
      const bool live = o < g.n;
      const float w = live ? __ldg(g.ws + o) : 0.0f, b = live ? out_bias_of(g.ob, o) : 0.0f;
      for (int i = r; i < g.tn; i += 128) ctrl->scales[buf][i] = t0 + i < g.m ? g.qs[t0 + i] : 0.0f;
      const bool ok = warp_wait(&ctrl->accf[buf], (it >> 1) & 1, abort_flag, g.status, g.budget);
      // the table is written; no warp goes on alone (it would wait here for the others)
      if (barrier_all(1, 128, ok)) {
        tc_fence_after();
      } else {
        break;
      }
      const int cols = min(g.tn, g.m - t0);
      uint8_t* yo = static_cast<uint8_t*>(g.y) + t0 * ldb + static_cast<int64_t>(o) * (g.yt == VQ_FP32 ? 4 : 2);
      for (int c = 0; c < g.tn; c += 32) {
        if (c >= cols) break;
        uint32_t acc[32];
        tmem_ld32(tmem + buf * kWideTn + c + (static_cast<uint32_t>(32 * lq) << 16), acc);
        tmem_wait_ld();
        if (!live) continue;
        const float4* e = reinterpret_cast<const float4*>(ctrl->scales[buf] + c);
        store_rows(g.yt, yo + c * ldb, ldb, acc, cols - c, e, w, b);
        store_rows(g.yt, yo + (c + 16) * ldb, ldb, acc + 16, cols - c - 16, e + 4, w, b);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&ctrl->acce[buf], 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  cluster_wait();
  if (*abort_flag) {
    // Loads and products in flight end before tensor memory is freed and the
    // block ends.  Their barriers may never complete once a CTA of the pair has
    // given up, so time does.  No warp raises the flag behind the barrier above;
    // a CTA whose flag is down has seen all of its loads and products end.
    const long long t0 = clock64();
    while (clock64() - t0 < kDrain / 16) __nanosleep(1000);
    __syncwarp();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kWideCols);
  }
}

// y = bias for a layer without inputs.
__global__ void i8_bias_kernel(int n, int m, const uint16_t* __restrict__ ob, const float* __restrict__ ws,
                               const float* __restrict__ qs, void* __restrict__ y, vq_dtype yt, int64_t ldy) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < static_cast<int64_t>(m) * n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / n;
    const int o = static_cast<int>(i - r * n);
    store_out(y, yt, r * ldy + o, i8_out(0, ws[o], qs[r], out_bias_of(ob, o)));
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

long long wait_budget() {
  if (const char* env = std::getenv("VQ_WAIT_BUDGET")) return std::atoll(env);
  return 4000000000LL;
}

// Splits of the narrow kernel (a power of two): double the cluster while the
// grid stays within two CTAs per SM and each CTA keeps at least four steps (512
// bytes of k).  Cold weights, 1, 2, 4, 8 CTAs a cluster, the choice marked: 1 x
// 1024 x 16384 25.7, 15.6, 10.4, 8.3* us; 4 x 4096 x 4096 9.2, 8.2, 7.0, 6.9*; 24 x
// 8192 x 8192 18.1, 17.4, 16.3*, 19.0; 16 x 14336 x 4096 13.2, 15.1*, -, 23.2, where
// 112 tiles fill the SMs already and the rule doubles once too often.
int narrow_splits(int tiles, int num_kt, int sms) {
  int s = 1;
  while (s < 8 && tiles * s * 2 <= 2 * sms && num_kt >= 8 * s) s *= 2;
  return s;
}

// Rows per tile of the wide kernel: the multiple of 32 that takes the fewest
// clocks over the last wave of pairs, a step costing 2 tn clocks of the tensor
// cores or the time its 16 KB of weights and tn / 2 rows take to arrive.  With
// 64, 128, 256 rows and the rule's choice: 333 x 4100 x 2000 13.2, 11.0, 15.4 and
// 10.1 us (96 rows), 1000 x 2048 x 4096 14.5, 12.1, 18.8 and 12.2, 512 x 8192 x
// 8192 44.4, 30.5, 29.5 and 29.7.
int wide_rows(int m, int tiles_n, int pairs) {
  int best = kWideTn;
  int64_t least = -1;
  for (int tn = kWideTn; tn >= 32; tn -= 32) {
    const int64_t tiles = static_cast<int64_t>(tiles_n) * ((m + tn - 1) / tn);
    const int64_t cost = (tiles + pairs - 1) / pairs * std::max(2 * tn, 320 + tn);
    if (least < 0 || cost < least) {
      least = cost;
      best = tn;
    }
  }
  return best;
}

// pdl: the kernel before this one on the stream is the quantisation that wrote q.
vq_status launch_gemm_i8(const I8Layer& L, const int8_t* q, int64_t ldq, const float* qs, int m, void* y, vq_dtype yt,
                         int64_t ldy, void* ws, cudaStream_t stream, bool pdl) {
  const int sms = device_sm_count();
  if (L.kin == 0) {
    count_launch();
    const int64_t total = static_cast<int64_t>(m) * L.n;
    i8_bias_kernel<<<static_cast<int>(std::min<int64_t>((total + 255) / 256, 8 * sms)), 256, 0, stream>>>(
        L.n, m, L.ob, L.scale, qs, y, yt, ldy);
    return cuda_status(cudaGetLastError());
  }
  I8Args g{};
  g.n = L.n;
  g.m = m;
  g.num_kt = (L.kin + kStepBytes - 1) / kStepBytes;
  g.ws = L.scale;
  g.ob = L.ob;
  g.qs = qs;
  g.y = y;
  g.yt = yt;
  g.ldy = ldy;
  g.status = static_cast<int*>(ws);
  g.budget = wait_budget();
  const bool narrow = m <= kNarrowRows;
  int box = 0;
  if (narrow) {
    g.tn = (m + 15) / 16 * 16;
    box = g.tn;
  } else {
    g.tiles_n = (L.n - 1) / (2 * kRows) + 1;
    g.tn = wide_rows(m, g.tiles_n, sms / 2);
    g.tiles_m = (m + g.tn - 1) / g.tn;
    box = g.tn / 2;
  }
  CUtensorMap wmap, xmap;
  if (!make_map_u8_sw128(&wmap, L.w, L.kin, L.n, L.ldw, kRows) || !make_map_u8_sw128(&xmap, q, L.kin, m, ldq, box))
    return VQ_ERR_CUDA;
  const int stage = kWTile + box * kStepBytes;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  const void* k;
  if (narrow) {
    const int tiles = (L.n - 1) / kRows + 1;
    const int splits = narrow_splits(tiles, g.num_kt, sms);
    for (g.split_log2 = 0; 1 << g.split_log2 < splits; ++g.split_log2) {}
    g.stages = std::min(kMaxStages, (device_smem_optin() / 2 - 1024 - kCtrlBytes - 1024) / stage);   // two CTAs per SM
    cfg.gridDim = dim3(tiles, splits);
    cfg.blockDim = dim3(kNarrowThreads);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = splits;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    k = reinterpret_cast<const void*>(gemm_i8_narrow_kernel);
  } else {
    g.stages = std::min(kMaxStages, (device_smem_optin() - 1024 - kCtrlBytes) / stage);
    cfg.gridDim = dim3(2 * std::min(g.tiles_n * g.tiles_m, sms / 2));
    cfg.blockDim = dim3(kWideThreads);
    k = reinterpret_cast<const void*>(gemm_i8_wide_kernel);
  }
  cfg.dynamicSmemBytes = 1024 + kCtrlBytes + static_cast<size_t>(g.stages) * stage;
  cudaError_t e = set_func_attr(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(cfg.dynamicSmemBytes));
  if (e != cudaSuccess) return cuda_status(e);
  count_launch();
  return cuda_status(narrow ? cudaLaunchKernelEx(&cfg, gemm_i8_narrow_kernel, wmap, xmap, g)
                            : cudaLaunchKernelEx(&cfg, gemm_i8_wide_kernel, wmap, xmap, g));
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
  return launch_gemm_i8(L, q, ldq, q_scale, m, y, y_dtype, ldy, workspace, static_cast<cudaStream_t>(stream),
                        false);
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
  return launch_gemm_i8(L, q, lay.ldq, qs, m, y, y_dtype, ldy, workspace, s, true);
}

}  // extern "C"
