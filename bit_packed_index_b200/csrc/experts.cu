// experts.cu -- vq_gemm_experts: products of codebook-indexed experts over the
// ragged groups of rows that a router made (include/vq_experts.h).
#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "codebook.cuh"
#include "sm100.cuh"
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

// ---------------------------------------------------------------------------
// x' = x * 2^-e in fp16, one row per grouped row, with 2^e and kSumUnit sum_k x.
// e puts the row's largest magnitude in [2^15, 2^16) (bf16 and fp16 values there
// are exact in fp16), so 2^e is at most 2^112 and times any fp16 scale stays in
// fp32's range; so does the sum of 2^24 of the largest values in its unit.
// Vector j of the layer (d values) takes columns H j .. H j + d - 1, H = 8 (d <=
// 8) or 16, zeros in the rest, so that the weight tiles hold centroids in whole
// 16-byte chunks.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr float kSumUnit = 1.0f / (1 << 24);

__device__ __forceinline__ float value16(uint16_t u, int x_fp16) { return x_fp16 ? h2f(u) : bf2f(u); }

__global__ void __launch_bounds__(kPrepThreads) experts_prep_kernel(
    const uint16_t* __restrict__ x, int x_fp16, int x_rows, int64_t ldx, const int32_t* __restrict__ rows,
    const int32_t* __restrict__ offsets, int n_experts, int kin, int d, int64_t kp, int vec, uint16_t* __restrict__ xh,
    float* __restrict__ xe, float* __restrict__ xsum, int* __restrict__ joined, int n_joined) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float s_max[kPrepThreads / 32], s_sum[kPrepThreads / 32];
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (r == 0)
    for (int i = tid; i < n_joined; i += kPrepThreads) joined[i] = 0;
  bool used = false;                       // is the row in front of some group's end?
  for (int k = tid; k <= n_experts; k += kPrepThreads) used |= __ldg(offsets + k) > r;
  if (!__syncthreads_or(used)) return;
  const int src = rows ? __ldg(rows + r) : r;
  const bool live = src >= 0 && src < x_rows;
  const uint16_t* xr = x + (live ? src : 0) * ldx;
  float mx = 0.0f, sm = 0.0f;
  if (live) {
    const int whole = vec ? kin / 8 : 0;
    for (int g = tid; g < whole; g += kPrepThreads) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(xr) + g);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = value16(static_cast<uint16_t>(w[i] & 0xFFFFu), x_fp16);
        const float hi = value16(static_cast<uint16_t>(w[i] >> 16), x_fp16);
        mx = fmaxf(mx, fmaxf(fabsf(lo), fabsf(hi)));
        sm = fmaf(lo, kSumUnit, sm);
        sm = fmaf(hi, kSumUnit, sm);
      }
    }
    for (uint32_t k = 8 * whole + tid; k < static_cast<uint32_t>(kin); k += kPrepThreads) {
      const float v = value16(__ldg(xr + k), x_fp16);
      mx = fmaxf(mx, fabsf(v));
      sm = fmaf(v, kSumUnit, sm);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    sm += __shfl_xor_sync(0xffffffffu, sm, off);
  }
  if (lane == 0) {
    s_max[warp] = mx;
    s_sum[warp] = sm;
  }
  __syncthreads();
  mx = sm = 0.0f;
#pragma unroll
  for (int w = 0; w < kPrepThreads / 32; ++w) {
    mx = fmaxf(mx, s_max[w]);
    sm += s_sum[w];
  }
  int e = 0;
  if (mx > 0.0f && mx < INFINITY) e = max(-126, min(127, static_cast<int>(__float_as_uint(mx) >> 23) - 127 - 15));
  const float f1 = __uint_as_float(static_cast<uint32_t>(127 - e / 2) << 23);   // 2^-e as two normal factors
  const float f2 = __uint_as_float(static_cast<uint32_t>(127 - (e - e / 2)) << 23);
  const uint32_t chunks = static_cast<uint32_t>(kp / 8), per = d > 8 ? 2 : 1;   // up to 2^31
  for (uint32_t g = tid; g < chunks; g += kPrepThreads) {
    const int at = 8 * static_cast<int>(g % per);
    const int64_t first = static_cast<int64_t>(g / per) * d + at;      // element in column 8 g
    const int n = live ? static_cast<int>(min(static_cast<int64_t>(min(8, d - at)), kin - first)) : 0;
    float v[8];
    if (vec && d % 8 == 0 && n == 8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(xr + first));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = value16(static_cast<uint16_t>(w[i] & 0xFFFFu), x_fp16);
        v[2 * i + 1] = value16(static_cast<uint16_t>(w[i] >> 16), x_fp16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? value16(__ldg(xr + first + i), x_fp16) : 0.0f;
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = f2h(v[2 * i] * f1 * f2) | (static_cast<uint32_t>(f2h(v[2 * i + 1] * f1 * f2)) << 16);
    *reinterpret_cast<uint4*>(xh + r * kp + 8 * static_cast<int64_t>(g)) = make_uint4(h[0], h[1], h[2], h[3]);
  }
  if (tid == 0) {
    xe[r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    xsum[r] = sm;
  }
}

// ---------------------------------------------------------------------------
// The product.  y^T = W_e x'^T per expert: 128 rows of W are the MMA's M, up to
// 384 rows of the group (512 where W's tiles lie in shared memory) its N, in two
// halves, so that a decoding step's one row and a prompt's hundreds take the
// same path and W is decoded once per 384 or 512 rows.
//
// What bounds it, per step of 128 x 64 weights (1024 vectors of eight), in
// clocks of the SM: the lookups of two staged books, 333 + 128 shared-memory
// wavefronts (16-byte rows of a 2^12 book at random, 2.6 lanes of a phase on a
// bank; the residual's eight copies meet none); for n rows n more to write x'
// and n to read it, and 2 n of tensor time.  So few rows cost what the lookups
// cost, 384 rows 1230 clocks of shared memory against 768 of products.  A 2^16
// book costs 1024 gathers at the 0.84 a clock that L2 hands out, 1220 clocks.
// Measured (B200, 148 SMs, weights cold): two 14336 x 4096 experts of 12 + 8 bits
// for one row 53 us (0.35 us a step, 20 us before the first and after the last);
// eight of them for 8192 rows, 1024 each, 1.02 ms a call, 942 TFLOP/s, and 1.17 ms
// (821) in a loop of calls under the power cap; sixteen 4096 x 2048 experts with
// 2^16 books for 62 rows each 99 us.
//
// W's two centroids are added in fp16, since the tensor cores take 16-bit
// operands and a product of its own for each book would double their work: half
// a step of 2^-11 per weight, 2.1e-4 of y in the root mean square (one book: no
// rounding, 6e-7).
//
//  * Sixteen producer warps decode W.  They work in four groups of 128 threads,
//    group i taking every fourth step (64 columns) from the i-th on; a thread
//    owns one row of the tile: it reads the row's index fields of the step
//    (loaded one turn ahead), gathers the centroids (small books staged in
//    shared memory, large ones through L2), adds the two books' and writes the
//    row of the tile.  Whole steps per group keep the per-step cost (a
//    barrier, the addresses) at a quarter of what it is when all warps share
//    each step, and the other groups' steps hide a group's gather latency.
//  * x' arrives by TMA in a ring of its own; one warp issues tcgen05.mma; four
//    warps read the accumulators back and store y.
//  * The work of all groups is one line of (expert, row tile, token tile,
//    step), cut into shares of equal cost, one per CTA, whatever the group sizes.  A
//    tile that two or more CTAs share is joined through the workspace: each
//    writes its partial sums, and the one that arrives last adds them in the
//    order of the shares (no wait, and the same order every time).
//  * Every wait is bounded (VQ_ERR_TIMEOUT in the status word).
// ---------------------------------------------------------------------------
using namespace sm100;

constexpr int kRowTile = 128;
constexpr int kATile = kRowTile * 128;            // one step of W: 64 halves a row
constexpr int kThreads = 768;                     // warp 0: x', 1: products, 4-7: epilogue, 8-23: producers
constexpr int kProducer0 = 256;
constexpr int kProducers = 512;
constexpr int kGroups = 4;                        // of 128 producer threads, each with its own steps
constexpr int kMaxA = 4, kMaxX = 8;
constexpr int kTmemCols = 512;
constexpr int kMinSteps = 8;                      // least steps worth a CTA
constexpr int kSnap = 4;                          // a share's border this near a tile's is moved there
constexpr long long kDrain = 1LL << 26;

struct Ctrl {
  uint64_t fulla[kMaxA];      // of a slot: its rows are written
  uint64_t donea[kGroups];    // of step % kGroups: its products are done
  uint64_t fullx[kMaxX], emptyx[kMaxX];
  uint64_t accf[2], acce[2];
  uint64_t idle;              // every product issued is done
  uint32_t tmem;
  int abort;
  int last;                                       // the epilogue's CTA is the last at a joined tile
};

struct Args {
  Experts E;
  const int32_t* offsets;
  int m;
  int nkt;                  // steps of the input dimension
  int row_tiles;
  int tokens;               // largest token tile (multiple of 16)
  int na, nx;               // slots of the two rings
  int xk;                   // steps of an x slot
  int xslot;                // bytes of an x slot
  int staged;               // bit m: book m in shared memory
  int copies;               // bit m: eight copies of it
  int off_book[2];          // its first byte behind the rings
  int off_table;            // the same of the borders' tables
  int off_scales;           // the same of the rows' scales
  const float* xe;
  const float* xsum;
  void* y;
  vq_dtype yt;
  int64_t ldy;
  float* part;              // [CTA][2][tokens][128] partial sums
  int* joined;              // [CTA] arrivals at the tile that CTA starts and does not finish
  int* status;
  long long budget;
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t hadd2_u32(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 hadd8(const uint4& a, const uint4& b) {
  return make_uint4(hadd2_u32(a.x, b.x), hadd2_u32(a.y, b.y), hadd2_u32(a.z, b.z), hadd2_u32(a.w, b.w));
}

// A place on the line of work: step kt of a tile (kt < steps of a tile).
struct Place {
  int tile, kt;
  __device__ __forceinline__ bool operator==(const Place& o) const { return tile == o.tile && kt == o.kt; }
  __device__ __forceinline__ bool operator<(const Place& o) const {
    return tile < o.tile || (tile == o.tile && kt < o.kt);
  }
};

// The line of work, its tables in shared memory: off, the group borders
// (clamped); first, the token tiles before each expert; border[c], where CTA
// c's share starts (border[CTAs]: the end).
struct Line {
  const int* off;
  const int* first;
  const Place* border;
  int experts, row_tiles, nkt;
  int acc;                  // rows of an accumulator: a tile of more takes two
};

// Cost of a step of a tile of n rows: a part that does not depend on n (W is
// decoded) and one that does.  Measured (ns): 500 + 1.5 n with books in shared
// memory, 700 + 2.1 n with a 2^16 book, about the same proportion; 1670 + 2.0 n in
// the general kernel (10 + 6 bits, tiled), for which this counts rows too high.
__host__ __device__ constexpr int step_cost(int n) { return 330 + n; }

// Rows of a token tile of an expert with `count` rows in `tt` tiles.
__device__ __forceinline__ int tile_rows(int count, int tt) { return ((count + tt - 1) / tt + 15) / 16 * 16; }

// First place of CTA c's share: the line cut into `ctas` parts of equal cost.
// cost[e]: what the token tiles before expert e cost, per row tile and step.
__device__ __forceinline__ Place share_border(const Line& l, const int64_t* cost, int ctas, int c) {
  const int tiles = l.first[l.experts] * l.row_tiles;
  if (c >= ctas) return {tiles, 0};
  const int64_t per_step = cost[l.experts] * l.row_tiles;          // all tiles' cost for one step each
  const int64_t at = static_cast<int64_t>(static_cast<double>(per_step) * l.nkt / ctas * c);
  const int64_t unit = static_cast<int64_t>(l.row_tiles) * l.nkt;  // cost[e] counts this often
  int lo = 0, hi = l.experts - 1;                                  // the expert the place falls into
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cost[mid] * unit <= at) lo = mid;
    else hi = mid - 1;
  }
  const int tt = l.first[lo + 1] - l.first[lo];
  if (tt == 0) return {l.first[lo] * l.row_tiles, 0};
  const int64_t step = (at - cost[lo] * unit) / step_cost(tile_rows(l.off[lo + 1] - l.off[lo], tt));
  int tile = static_cast<int>(step / l.nkt), kt = static_cast<int>(step - static_cast<int64_t>(tile) * l.nkt);
  if (kt < kSnap) kt = 0;
  else if (l.nkt - kt < kSnap) ++tile, kt = 0;
  if (tile >= tt * l.row_tiles) tile = tt * l.row_tiles, kt = 0;
  return {l.first[lo] * l.row_tiles + tile, kt};
}

// One CTA's part of one tile: from `at` to the tile's end or `end`, where it
// moves `at`.
struct Part {
  int tile, expert, row0, r0, live, n;     // first W row; first grouped row, its rows, those padded to 16
  int kt0, kt1;
  int acc;

  __device__ __forceinline__ Part(const Line& l, Place& at, const Place& end) {
    acc = l.acc;
    tile = at.tile;
    kt0 = at.kt;
    kt1 = at.tile == end.tile ? end.kt : l.nkt;
    at = at.tile == end.tile ? end : Place{at.tile + 1, 0};
    // the expert: the last one whose tiles start at or before this one
    int lo = 0, hi = l.experts - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (l.first[mid] * l.row_tiles <= tile) lo = mid;
      else hi = mid - 1;
    }
    expert = lo;
    const int tt = l.first[lo + 1] - l.first[lo];
    const int in = tile - l.first[lo] * l.row_tiles;           // row tile major
    const int rt = in / tt, j = in - rt * tt;
    const int count = l.off[lo + 1] - l.off[lo];
    const int per = tile_rows(count, tt);
    row0 = rt * kRowTile;
    r0 = l.off[lo] + j * per;
    live = min(per, count - j * per);
    n = (live + 15) / 16 * 16;
  }
  __device__ __forceinline__ int halves() const { return n > acc ? 2 : 1; }
  // rows of half h (multiples of 16, at most acc)
  __device__ __forceinline__ int half_rows(int h) const {
    if (n <= acc) return n;
    const int a = (n / 2 + 15) / 16 * 16;
    return h == 0 ? a : n - a;
  }
};

// The eight B-bit fields (B in 4, 8, 12, 16) of row o in a step, as the words
// that hold them.  Row order: B consecutive bytes of the row's stream.  Tiled:
// the row's 4B-bit records of two tiles.  Words past the stream's row, and
// tiles past the last, read as zero: their fields belong to vectors past the
// last, which meet zeros of x'.
template <int LAYOUT, int B>
struct Words {
  static constexpr int per = LAYOUT == VQ_IDX_TILE4 ? (B == 4 ? 1 : B / 8 + (B == 12)) : B / 4;   // words of a record, of a step
  static constexpr int count = LAYOUT == VQ_IDX_TILE4 ? 2 * per : per;
  const uint32_t* base;
  int64_t stride;           // tiled: words of a tile; row order: words that the row's own fields take, which may be
                            // fewer than lie between two rows (the last row need not own the rest)
  int tiles, shift;

  __device__ __forceinline__ void set(const Layer& L, int m, int64_t o) {
    if constexpr (LAYOUT == VQ_IDX_TILE4) {
      stride = L.rw[m];
      base = L.idx[m] + ((o * (4 * B)) >> 5);
      shift = static_cast<int>((o * (4 * B)) & 31);
      tiles = (L.nvec - 1) / 4 + 1;
    } else {
      stride = (static_cast<int64_t>(L.nvec) * B + 127) / 128 * 4;
      base = L.idx[m] + o * L.rw[m];
      shift = 0;
    }
  }
  __device__ __forceinline__ void load(int kt, uint32_t (&w)[count]) const {
    if constexpr (LAYOUT == VQ_IDX_TILE4) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t* q = base + (2 * kt + t) * stride;
        const bool in = 2 * kt + t < tiles;
        if constexpr (B == 16) {
          const uint2 v = in ? __ldg(reinterpret_cast<const uint2*>(q)) : make_uint2(0u, 0u);
          w[2 * t] = v.x;
          w[2 * t + 1] = v.y;
        } else if constexpr (B == 12) {       // 48 bits from bit 0 or 16 of a word: inside two words of the tile
          w[2 * t] = in ? __ldg(q) : 0u;
          w[2 * t + 1] = in ? __ldg(q + 1) : 0u;
        } else {
          w[t] = in ? __ldg(q) : 0u;
        }
      }
    } else {
      const int64_t at = static_cast<int64_t>(kt) * per;
      if (at + per <= stride) {
        const uint32_t* q = base + at;
        if constexpr (B == 16) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (B == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
          w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
          for (int i = 0; i < per; ++i) w[i] = __ldg(q + i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < per; ++i) w[i] = at + i < stride ? __ldg(base + at + i) : 0u;
      }
    }
  }
  // field of vector v of the step
  __device__ __forceinline__ uint32_t field(const uint32_t (&w)[count], int v) const {
    constexpr uint32_t mask = (1u << B) - 1u;
    if constexpr (LAYOUT == VQ_IDX_TILE4) {
      const int t = v >> 2, f = v & 3;
      if constexpr (B == 16) return (w[2 * t + (f >> 1)] >> (16 * (f & 1))) & mask;
      if constexpr (B == 8) return (w[t] >> (8 * f)) & mask;
      if constexpr (B == 4) return (w[t] >> (shift + 4 * f)) & mask;
      // 12: the record moved down to bit 0
      const uint32_t lo = __funnelshift_r(w[2 * t], w[2 * t + 1], shift), hi = w[2 * t + 1] >> shift;
      if (f == 0) return lo & mask;
      if (f == 1) return (lo >> 12) & mask;
      if (f == 2) return __funnelshift_r(lo, hi, 24) & mask;
      return (hi >> 4) & mask;
    } else {
      const int bit = v * B;
      const int q = bit >> 5;
      return __funnelshift_r(w[q], q + 1 < count ? w[q + 1] : 0u, bit & 31) & mask;
    }
  }
};

// Field j of row o of any width and order.
__device__ __forceinline__ uint32_t any_field(const Layer& L, int m, int64_t o, int j) {
  const int b = L.b[m];
  return L.layout == VQ_IDX_ROWS ? load_field(L.idx[m] + o * L.rw[m], static_cast<int64_t>(j) * b, b)
                                 : load_field(L.idx[m] + (j >> 2) * L.rw[m], (4 * o + (j & 3)) * b, b);
}

// x' comes in boxes of box_rows() rows by xk steps, one box for a tile's half: a
// load's issue takes its warp about 450 clocks, whatever the box holds, longer
// than the other warps take for a step of few rows.
constexpr int kBoxes = 5;
__host__ __device__ constexpr int box_rows(int i, int acc) { return i < 4 ? 16 << i : acc; }
__host__ __device__ constexpr int box_of(int n) { return n <= 16 ? 0 : n <= 32 ? 1 : n <= 64 ? 2 : n <= 128 ? 3 : 4; }
struct Maps {
  CUtensorMap m[kBoxes];
};

// y of one output (its column in y: yo) for `n` of sixteen rows from their
// sums: s v 2^e + t sum x + b, t in units of 1 / kSumUnit.  scales: 2^e and
// kSumUnit sum x of the rows, in shared memory.  s 2^e comes first: v 2^e can
// leave fp32's range where y does not.  The type is a template argument: a
// branch on it per value, with the single warp that each scheduler has for
// this, made the store of a tile take longer than its products.
template <int YT>
__device__ __forceinline__ void store_rows(uint8_t* yo, int64_t ldb, const float (&v)[16], int n, const float4* scales,
                                           float sc, float tb, float ob) {
  using T = typename std::conditional<YT == VQ_FP32, float, uint16_t>::type;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float4 e = scales[i / 2];
    const float a = fmaf(sc * e.x, v[i], fmaf(tb, e.y, ob)), b = fmaf(sc * e.z, v[i + 1], fmaf(tb, e.w, ob));
    T x, y;
    if constexpr (YT == VQ_FP32) {
      x = a;
      y = b;
    } else {
      x = YT == VQ_FP16 ? f2h(a) : f2bf(a);
      y = YT == VQ_FP16 ? f2h(b) : f2bf(b);
    }
    if (i < n) *reinterpret_cast<T*>(yo + i * ldb) = x;
    if (i + 1 < n) *reinterpret_cast<T*>(yo + (i + 1) * ldb) = y;
  }
}

// Where a book is read from.  A staged entry takes 16 bytes a chunk (eight
// values); a small book is kept eight times over, entry i's copies side by
// side, so that the eight lanes of a shared-memory phase read eight different
// bank groups whatever their indices.
struct Book {
  uint32_t smem;            // shared address, with the lane's copy
  int shift;                // log2 of an entry's bytes
  const uint16_t* global;   // not staged: rows of d halves
};

// Chunk q (values 8 q .. 8 q + 7, zeros past d) of entry i of a book of rows of d halves.
__device__ __forceinline__ uint4 global_chunk(const uint16_t* book, int d, uint32_t i, int q) {
  const uint16_t* r = book + static_cast<size_t>(i) * d + 8 * q;
  if (d % 8 == 0) return __ldg(reinterpret_cast<const uint4*>(r));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (d % 2 == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (8 * q + 2 * e < d) w[e] = __ldg(reinterpret_cast<const uint32_t*>(r) + e);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (8 * q + e < d) w[e >> 1] |= static_cast<uint32_t>(__ldg(r + e)) << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same of a book that may be staged.
__device__ __forceinline__ uint4 any_centroid(const Book& b, bool staged, int d, uint32_t i, int q) {
  return staged ? lds128(b.smem + (i << b.shift) + 16 * q) : global_chunk(b.global, d, i, q);
}

// W tiles whose rows pass through registers anyway (books in shared memory) lie
// in tensor memory: a step is 32 columns, and neither the producers' stores nor
// the products' reads of W take shared memory's cycles from the lookups, which
// bound the kernel.  Those that cp.async fills (2^16 books) and those of the
// general kernel lie in shared memory.  Tensor memory holds two accumulators of
// acc_rows() rows and, in the first case, four steps of W.
__host__ __device__ constexpr bool w_in_tmem(int b1) { return b1 > 0 && b1 < 16; }
__host__ __device__ constexpr int acc_rows(bool in_tmem) { return in_tmem ? 192 : 256; }

// B1 > 0: d <= 8, books of 2^B1 and 2^B2 (0: no second) entries; the second
// staged, the first staged or (B1 = 16) read through L2 with d = 8.  B1 = 0:
// any layer, field by field.  Measured (eight 4096 x 4096 experts, cold, ps a
// vector in row order / tiled), 16 rows each: 12 + 8 bits 5.2 / 3.8, 16 bits 5.1 /
// 4.9; B1 = 0: 10 + 6 bits 13.7 / 11.2, 11 bits 7.8, 16 bits of d = 6 11.6 / 10.9, d
// = 16 13 to 15 for twice the values.  256 rows each: 12 + 8 bits 8.3 / 7.3, 10 + 6
// bits 18 / 14, but 12 + 12 and 13 + 13 bits 62 and 84: 128 KB of staged books leave
// room for token tiles of 64 and 32 rows, and W is decoded for each.
template <int LAYOUT, int B1, int B2>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_experts_kernel(const __grid_constant__ Maps maps,
                        const __grid_constant__ Args g) {
  extern __shared__ uint8_t smem_raw[];
  constexpr bool kInTmem = w_in_tmem(B1);
  constexpr int kAcc = acc_rows(kInTmem);
  uint8_t* base = align1024(smem_raw);
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(base);
  uint8_t* aring = base + 1024;
  uint8_t* xring = aring + (kInTmem ? 0 : g.na * kATile);
  uint8_t* books = xring + g.nx * g.xslot;
  const Layer& L0 = g.E.L;
  const int n_experts = g.E.e;
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctrl->abort;
  int* s_off = reinterpret_cast<int*>(books + g.off_table);    // [experts + 1] borders
  int* s_first = s_off + n_experts + 1;                        // [experts + 1] token tiles in front
  int64_t* s_cost = reinterpret_cast<int64_t*>(s_first + n_experts + 1);  // [experts + 1] see share_border
  Place* s_border = reinterpret_cast<Place*>(s_cost + n_experts + 1);     // [CTAs + 1]
  float2* s_scales = reinterpret_cast<float2*>(books + g.off_scales);    // [2][tokens]

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.na; ++s) mbar_init(&ctrl->fulla[s], kProducers / 32 / kGroups);
    for (int s = 0; s < kGroups; ++s) mbar_init(&ctrl->donea[s], 1);
    for (int s = 0; s < g.nx; ++s) {
      mbar_init(&ctrl->fullx[s], 1);
      mbar_init(&ctrl->emptyx[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctrl->accf[b], 1);
      mbar_init(&ctrl->acce[b], 4);
    }
    mbar_init(&ctrl->idle, 1);
    ctrl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem, kTmemCols);
    tmem_relinquish();
  }
  for (int k = threadIdx.x; k <= n_experts; k += kThreads) s_off[k] = min(g.m, max(0, __ldg(g.offsets + k)));
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {                                   // ascending borders and the token tiles before each expert
    const int per = (n_experts + 32) / 32;           // entries of a lane
    const int k0 = min(lane * per, n_experts + 1), k1 = min(k0 + per, n_experts + 1);
    int top = 0;
    for (int k = k0; k < k1; ++k) top = max(top, s_off[k]);
    int before = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before = max(before, v);
    }
    before = __shfl_up_sync(0xffffffffu, before, 1);
    top = lane == 0 ? 0 : before;
    for (int k = k0; k < k1; ++k) s_off[k] = top = max(top, s_off[k]);
    __syncwarp();
    int sum = 0;
    int64_t cost = 0;
    for (int k = k0; k < min(k1, n_experts); ++k) {
      const int count = s_off[k + 1] - s_off[k], tt = (count + g.tokens - 1) / g.tokens;
      sum += tt;
      if (tt) cost += static_cast<int64_t>(tt) * step_cost(tile_rows(count, tt));
    }
    int incl = sum;
    int64_t cincl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      const int64_t w = __shfl_up_sync(0xffffffffu, cincl, o);
      if (lane >= o) {
        incl += v;
        cincl += w;
      }
    }
    sum = incl - sum;
    cost = cincl - cost;
    for (int k = k0; k < k1; ++k) {
      s_first[k] = sum;
      s_cost[k] = cost;
      if (k == n_experts) break;
      const int count = s_off[k + 1] - s_off[k], tt = (count + g.tokens - 1) / g.tokens;
      sum += tt;
      if (tt) cost += static_cast<int64_t>(tt) * step_cost(tile_rows(count, tt));
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(ctrl->tmem);
  Line line;
  line.off = s_off;
  line.first = s_first;
  line.border = s_border;
  line.experts = n_experts;
  line.row_tiles = g.row_tiles;
  line.nkt = g.nkt;
  line.acc = kAcc;
  {
    // a CTA for each tile at least, more where their steps are worth cutting
    const int64_t tiles = static_cast<int64_t>(s_first[n_experts]) * g.row_tiles;
    const int ctas = static_cast<int>(max(
        static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), max(tiles, tiles * g.nkt / kMinSteps))));
    for (int c = threadIdx.x; c <= static_cast<int>(gridDim.x); c += kThreads)
      s_border[c] = share_border(line, s_cost, ctas, c);
  }
  __syncthreads();
  const int cta = blockIdx.x;
  const Place from = s_border[cta], to = s_border[cta + 1];
  const int nbuf = g.tokens <= kAcc ? 2 : 1;         // accumulators in turn
  const uint32_t tmem_a = tmem + 2 * kAcc;           // W steps of 32 columns

  // The loops of the two issuing warps are on the critical path of small tiles,
  // so what can be worked out per tile or once is.
  if (warp == 0) {                                    // x' by TMA
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int q = 0, qp = 0, issued = 0;                    // x slot, its phase, loads issued
    bool stop = false;
    for (Place at = from; at < to && !stop;) {
      const Part t(line, at, to);
      const int n0 = uniform(t.half_rows(0)), n1 = uniform(t.n) - n0, r0 = uniform(t.r0);
      const int kt1 = uniform(t.kt1), b0 = box_of(n0);
      for (int kt = uniform(t.kt0); kt < kt1 && !stop; kt += g.xk) {
        int row = r0, box = b0;
        for (;;) {
          if (!warp_wait(&ctrl->emptyx[q], qp ^ 1, abort_flag, g.status, g.budget)) {
            stop = true;
            break;
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(&ctrl->fullx[q], g.xk * box_rows(box, kAcc) * 128);
            tma_load_3d(xring + q * g.xslot, &maps.m[box], &ctrl->fullx[q], 0, row, kt);
          }
          __syncwarp();
          ++issued;
          if (++q == g.nx) {
            q = 0;
            qp ^= 1;
          }
          if (n1 == 0 || row != r0) break;
          row += n0;
          box = box_of(n1);
        }
      }
    }
    // Loads in flight land before the block ends, whichever warp gives up and
    // when (the products wait for them anyway).
    if (lane == 0)
      for (int i = max(0, issued - g.nx); i < issued; ++i)
        drain_phase(&ctrl->fullx[i % g.nx], (i / g.nx) & 1, kDrain / 16);
    __syncwarp();
  } else if (warp == 1) {                             // products
    const uint64_t adesc0 = sw128_kmajor_desc(smem_addr(aring)), xdesc0 = sw128_kmajor_desc(smem_addr(xring));
    const uint32_t xstep = static_cast<uint32_t>(g.xslot) >> 4;
    // the four products of a step, W from tensor or shared memory
    auto step_products = [](uint32_t d, uint32_t at_, uint64_t ad, uint64_t bd, uint32_t id, uint32_t add) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if constexpr (kInTmem) umma_f16_ta(d, at_ + 8 * kk, bd + 2 * kk, id, kk ? 1u : add);
        else umma_f16(d, ad + 2 * kk, bd + 2 * kk, id, kk ? 1u : add);
      }
    };
    int q = 0, qp = 0, s = 0, sp = 0, it = 0, step = 0;
    bool stop = false;
    for (Place at = from; at < to && !stop; ++it) {
      const Part t(line, at, to);
      // two accumulators in turn, or the halves of one tile after another: `acce`
      // of a half tells that the epilogue has read it
      const int buf = it % nbuf;
      if (it >= nbuf && !warp_wait(&ctrl->acce[buf], ((it / nbuf) & 1) ^ 1, abort_flag, g.status, g.budget)) break;
      tc_fence_after();
      const uint32_t d0 = tmem + buf * kAcc;
      const uint32_t id0 = uniform(f16_idesc(kRowTile, t.half_rows(0)));
      const uint32_t id1 = uniform(t.halves() == 2 ? f16_idesc(kRowTile, t.half_rows(1)) : 0u);
      const int kt0 = uniform(t.kt0), kt1 = uniform(t.kt1);
      uint32_t add = 0;
      // A barrier's test takes longer than a product of a few rows, so the next
      // one's is under way while this step's products are issued.
      bool ready = false, readyx = false;
      if (id1 == 0) {
        const uint32_t kstep = uniform(static_cast<uint32_t>(box_rows(box_of(t.n), kAcc))) * (128 >> 4);
        int kk = 0;                                   // step of the x slot
        uint64_t bd = 0;
        for (int kt = kt0; kt < kt1; ++kt, ++step) {
          if (kk == 0) {
            if (!readyx && !warp_wait(&ctrl->fullx[q], qp, abort_flag, g.status, g.budget)) {
              stop = true;
              break;
            }
            bd = xdesc0 + static_cast<uint32_t>(q) * xstep;
          }
          if (!ready && !warp_wait(&ctrl->fulla[s], sp, abort_flag, g.status, g.budget)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint64_t ad = adesc0 + static_cast<uint32_t>(s * (kATile >> 4));
          const uint32_t at_ = tmem_a + 32 * s;
          if (++s == g.na) {
            s = 0;
            sp ^= 1;
          }
          const bool next = mbar_test_wait(&ctrl->fulla[s], sp), more = kt + 1 < kt1;
          const bool spent = ++kk == g.xk || !more;   // the x slot's last step
          uint64_t* free_bar = &ctrl->emptyx[q];
          bool nextx = false;
          if (spent) {
            kk = 0;
            if (++q == g.nx) {
              q = 0;
              qp ^= 1;
            }
            nextx = mbar_test_wait(&ctrl->fullx[q], qp);
          }
          if (elect_one()) {
            step_products(d0, at_, ad, bd, id0, add);
            umma_commit(&ctrl->donea[step % kGroups]);
            if (spent) umma_commit(free_bar);
          }
          bd += kstep;
          ready = __all_sync(0xffffffffu, next) && more;
          if (spent) readyx = __all_sync(0xffffffffu, nextx) && more;
          add = 1;
        }
      } else {
        const int halves = 2;
        for (int kt = kt0; kt < kt1 && !stop; ++kt, ++step) {
          if (!ready && !warp_wait(&ctrl->fulla[s], sp, abort_flag, g.status, g.budget)) {
            stop = true;
            break;
          }
          const uint64_t ad = adesc0 + static_cast<uint32_t>(s * (kATile >> 4));
          const uint32_t at_ = tmem_a + 32 * s;
          if (++s == g.na) {
            s = 0;
            sp ^= 1;
          }
          for (int h = 0; h < halves; ++h) {
            if ((!readyx && !warp_wait(&ctrl->fullx[q], qp, abort_flag, g.status, g.budget)) ||
                (h == 1 && add == 0 && it > 0 &&
                 !warp_wait(&ctrl->acce[1], (it & 1) ^ 1, abort_flag, g.status, g.budget))) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint64_t bd = xdesc0 + static_cast<uint32_t>(q) * xstep;
            uint64_t* free_bar = &ctrl->emptyx[q];
            if (++q == g.nx) {
              q = 0;
              qp ^= 1;
            }
            const bool last = h + 1 == halves;
            const bool nextx = mbar_test_wait(&ctrl->fullx[q], qp);
            const bool next = mbar_test_wait(&ctrl->fulla[s], sp);
            const uint32_t d = d0 + h * kAcc, id = h ? id1 : id0;
            if (elect_one()) {
              step_products(d, at_, ad, bd, id, add);
              umma_commit(free_bar);
              if (last) umma_commit(&ctrl->donea[step % kGroups]);
            }
            const bool more = !last || kt + 1 < kt1;
            readyx = __all_sync(0xffffffffu, nextx) && more;
            ready = __all_sync(0xffffffffu, next) && last && more;
          }
          add = 1;
        }
      }
      if (!stop && elect_one()) umma_commit(&ctrl->accf[buf]);
      __syncwarp();
    }
    if (elect_one()) {                                // products in flight end before tensor memory is freed, as above
      umma_commit(&ctrl->idle);
      drain_phase(&ctrl->idle, 0, kDrain);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {                 // epilogue: lane quarter warp & 3, one W row per thread
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lq = warp & 3, r = 32 * lq + lane;
    const int64_t slot_size = static_cast<int64_t>(g.tokens) * kRowTile;
    const int64_t ldb = g.ldy * (g.yt == VQ_FP32 ? 4 : 2);
    int it = 0;
    for (Place at = from; at < to; ++it) {
      const Part t(line, at, to);
      const bool whole = t.kt0 == 0 && t.kt1 == g.nkt;
      const int buf = it % nbuf;
      const int o = t.row0 + r;
      const Layer L = expert_layer(g.E, t.expert);
      const bool live = o < L.n;
      const float sc = live && L.scale ? h2f(__ldg(L.scale + o)) : 1.0f;
      const float tb = live && L.bias ? h2f(__ldg(L.bias + o)) * (1.0f / kSumUnit) : 0.0f;
      const float ob = live ? out_bias_of(L.ob, o) : 0.0f;
      // the rows' scales and sums, in the table that the tile before last used
      float2* scales = s_scales + (it & 1) * g.tokens;
      for (int i = r; i < t.n; i += 128)
        scales[i] = i < t.live ? make_float2(g.xe[t.r0 + i], g.xsum[t.r0 + i]) : make_float2(0.0f, 0.0f);
      uint8_t* yo = static_cast<uint8_t*>(g.y) + t.r0 * ldb + static_cast<int64_t>(o) * (g.yt == VQ_FP32 ? 4 : 2);
      auto store16 = [&](const float (&v)[16], int c) {
        const int n = live ? t.live - c : 0;
        const float4* e = reinterpret_cast<const float4*>(scales + c);
        uint8_t* p = yo + c * ldb;
        if (g.yt == VQ_BF16) store_rows<VQ_BF16>(p, ldb, v, n, e, sc, tb, ob);
        else if (g.yt == VQ_FP16) store_rows<VQ_FP16>(p, ldb, v, n, e, sc, tb, ob);
        else store_rows<VQ_FP32>(p, ldb, v, n, e, sc, tb, ob);
      };
      // the four warps go on together or not at all (they meet at barriers below)
      if (!barrier_all(1, 128, warp_wait(&ctrl->accf[buf], (it / nbuf) & 1, abort_flag, g.status, g.budget))) break;
      tc_fence_after();
      const uint32_t acc0 = tmem + buf * kAcc + (static_cast<uint32_t>(32 * lq) << 16);
      const int n0 = t.half_rows(0);
      // a shared tile: the sums to this CTA's slot (1: it starts the tile, 0: it goes on with it)
      float* mine = g.part + (2 * static_cast<int64_t>(cta) + (t.kt0 == 0 ? 1 : 0)) * slot_size + r;
      // rows c .. c + 15 start at tensor-memory column c, or kAcc + c - n0 in the
      // second half; the next ones are read while these are stored
      auto read16 = [&](int c, uint32_t (&acc)[16]) { tmem_ld16(acc0 + (c < n0 ? c : kAcc + c - n0), acc); };
      auto was_read = [&](int c) {                               // rows up to c: maybe the end of a half
        if (c != t.n && !(nbuf == 1 && c == n0)) return;
        tc_fence_before();
        __syncwarp();
        if (lane != 0) return;
        if (nbuf == 2) mbar_arrive(&ctrl->acce[buf]);
        if (nbuf == 1 && c == n0) mbar_arrive(&ctrl->acce[0]);
        if (nbuf == 1 && c == t.n) mbar_arrive(&ctrl->acce[1]);
      };
      uint32_t acc[16];
      read16(0, acc);
      tmem_wait_ld();
      was_read(16);
      for (int c = 0; c < t.n; c += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(acc[i]);
        const bool more = c + 16 < t.n;
        if (more) read16(c + 16, acc);
        if (whole) {
          store16(v, c);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) __stcg(mine + (c + i) * kRowTile, v[i]);
        }
        if (more) {
          tmem_wait_ld();
          was_read(c + 32);
        }
      }
      if (whole) continue;
      // the CTAs of the tile: from the one whose share holds its first step to
      // the one with its last
      int c0 = cta, c1 = cta;
      const Place begin = {t.tile, 0}, end = {t.tile + 1, 0};
      while (c0 > 0 && begin < s_border[c0]) --c0;
      while (s_border[c1 + 1] < end) ++c1;
      __threadfence();
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (r == 0) {
        int parts = 0;                                // shares that are not empty
        for (int c = c0; c <= c1; ++c) parts += s_border[c + 1] == s_border[c] ? 0 : 1;
        ctrl->last = atomicAdd(g.joined + c0, 1) == parts - 1;
        __threadfence();
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (ctrl->last) {
        // sixteen rows at a time, so that their loads are in flight together
        for (int c = 0; c < t.n; c += 16) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.0f;
          for (int k = c0; k <= c1; ++k) {
            if (s_border[k + 1] == s_border[k]) continue;
            const float* part = g.part + (2 * static_cast<int64_t>(k) + (k == c0 ? 1 : 0)) * slot_size + c * kRowTile + r;
            float u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = __ldcg(part + i * kRowTile);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += u[i];
          }
          store16(v, c);
        }
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // `last` is read before the next tile sets it
    }
  } else if (warp >= 8) {                             // producers
    const int pt = threadIdx.x - kProducer0;
    const int group = pt >> 7, r = pt & 127;
    const bool two = L0.nb == 2;
    const int ch = L0.d > 8 ? 2 : 1;                  // chunks of a vector
    Book book[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const bool copies = (g.copies >> m) & 1;
      book[m].shift = (copies ? 7 : 4) + (ch - 1);
      book[m].smem = smem_addr(books) + g.off_book[m] + (copies ? (lane & 7) * 16 * ch : 0);
    }
    int staged_expert = -1;
    int gs = 0;                                       // steps of this CTA's earlier tiles
    bool stop = false;                                // a warp that gave up still meets the others where books change
    for (Place at = from; at < to;) {
      const Part t(line, at, to);
      const Layer L = expert_layer(g.E, t.expert);
      book[0].global = L.book[0];
      book[1].global = L.book[1];
      const int64_t o = min(t.row0 + r, L.n - 1);     // rows past N repeat the last; they are never stored
      int kt = t.kt0 + ((group - gs) & (kGroups - 1));   // the group's first step
      constexpr int W1 = B1 > 0 ? Words<LAYOUT, (B1 > 0 ? B1 : 4)>::count : 1;
      constexpr int W2 = B2 > 0 ? Words<LAYOUT, (B2 > 0 ? B2 : 4)>::count : 1;
      Words<LAYOUT, (B1 > 0 ? B1 : 4)> f1;
      Words<LAYOUT, (B2 > 0 ? B2 : 4)> f2;
      uint32_t w1[W1], w2[W2];                        // words of the group's next step
      if constexpr (B1 > 0) {
        f1.set(L, 0, o);
        if constexpr (B2 > 0) f2.set(L, 1, o);
        if (kt < t.kt1) {
          f1.load(kt, w1);
          if constexpr (B2 > 0) f2.load(kt, w2);
        }
      }
      if (staged_expert != t.expert && g.staged) {
        const bool all = staged_expert < 0;           // books that the experts share are staged once
        staged_expert = t.expert;
        asm volatile("bar.sync 2, 512;" ::: "memory");   // nobody reads the old books any more
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (!(g.staged & (1 << m)) || (!all && g.E.sb[m] == 0)) continue;
          const uint16_t* src = L.book[m];
          const bool copies = (g.copies >> m) & 1;
          const uint32_t dst = smem_addr(books) + g.off_book[m];
          const int chunks = ch << L.b[m];            // 16-byte chunks of the book
          for (int i0 = pt; i0 < chunks; i0 += 4 * kProducers) {
            uint4 v[4];                               // loads in flight together
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = i0 + u * kProducers;
              if (i < chunks) v[u] = global_chunk(src, L.d, i / ch, i & (ch - 1));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = i0 + u * kProducers;
              if (i >= chunks) break;
              if (copies) {
#pragma unroll
                for (int c = 0; c < 8; ++c) sts128(dst + ((i / ch * 8 + c) * ch + (i & (ch - 1))) * 16, v[u]);
              } else {
                sts128(dst + i * 16, v[u]);
              }
            }
          }
        }
        asm volatile("bar.sync 2, 512;" ::: "memory");
      }
      for (; kt < t.kt1 && !stop; kt += kGroups) {
        // Step i writes slot i % na once step i - na is done with it.  That
        // step's barrier is shared with step i - na - 4 alone of the earlier
        // ones, which this group saw done before it wrote step i - 4, so the
        // barrier's phase cannot be mistaken for an older one.
        const int step = gs + (kt - t.kt0), freed = step - g.na;
        const int s = step % g.na;
        auto slot_free = [&] {
          return freed < 0 || warp_wait(&ctrl->donea[freed % kGroups], (freed / kGroups) & 1, abort_flag, g.status, g.budget);
        };
        const uint32_t row = smem_addr(aring + s * kATile) + r * 128;
        if constexpr (B1 == 16) {
          // Straight into the tile: no registers and no lines of L1 (what is
          // left of it beside the rings holds too few for the gathers of a
          // step) wait for the centroids.  The other groups' steps are in flight
          // meanwhile.
          if (!slot_free()) {
            stop = true;
            break;
          }
#pragma unroll
          for (int v = 0; v < 8; ++v)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(row + ((v ^ (r & 7)) << 4)),
                         "l"(reinterpret_cast<const uint4*>(book[0].global) + f1.field(w1, v))
                         : "memory");
          asm volatile("cp.async.commit_group;" ::: "memory");
          uint32_t i2[8];
          if constexpr (B2 > 0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) i2[v] = f2.field(w2, v);
          }
          if (kt + kGroups < t.kt1) {
            f1.load(kt + kGroups, w1);
            if constexpr (B2 > 0) f2.load(kt + kGroups, w2);
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          if constexpr (B2 > 0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              const uint32_t a = row + ((v ^ (r & 7)) << 4);
              sts128(a, hadd8(lds128(a), lds128(book[1].smem + (i2[v] << book[1].shift))));
            }
          }
        } else if constexpr (B1 > 0) {
          uint4 c[8];
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const uint32_t i = f1.field(w1, v);
            c[v] = lds128(book[0].smem + (i << book[0].shift));
          }
          if constexpr (B2 > 0) {
#pragma unroll
            for (int v = 0; v < 8; ++v) c[v] = hadd8(c[v], lds128(book[1].smem + (f2.field(w2, v) << book[1].shift)));
          }
          if (kt + kGroups < t.kt1) {
            f1.load(kt + kGroups, w1);
            if constexpr (B2 > 0) f2.load(kt + kGroups, w2);
          }
          if (!slot_free()) {
            stop = true;
            break;
          }
          tc_fence_after();
          tmem_st32(tmem_a + 32 * s + (static_cast<uint32_t>(32 * (warp & 3)) << 16), c);
          tmem_wait_st();
          tc_fence_before();
        } else {
          if (!slot_free()) {
            stop = true;
            break;
          }
          const int vectors = 8 / ch;
          for (int v = 0; v < vectors; ++v) {
            const int j = kt * vectors + v;
            uint4 c[2];
            c[0] = c[1] = make_uint4(0u, 0u, 0u, 0u);
            if (j < L.nvec) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                if (m == 1 && !two) break;
                const uint32_t i = any_field(L, m, o, j);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  if (q >= ch) break;
                  const uint4 u = any_centroid(book[m], (g.staged >> m) & 1, L.d, i, q);
                  c[q] = m == 0 ? u : hadd8(c[q], u);
                }
              }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (q < ch) sts128(row + (((v * ch + q) ^ (r & 7)) << 4), c[q]);
          }
        }
        if constexpr (!kInTmem) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->fulla[s]);
      }
      gs += t.kt1 - t.kt0;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// y = output bias for experts without inputs.
__global__ void experts_bias_kernel(Experts E, const int32_t* __restrict__ offsets, int m, void* __restrict__ y,
                                    vq_dtype yt, int64_t ldy) {
  int last = 0;
  for (int e = 0; e < E.e; ++e) {
    const int r0 = max(last, min(m, max(0, offsets[e]))), r1 = max(r0, min(m, max(0, offsets[e + 1])));
    last = r1;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
         i < static_cast<int64_t>(r1 - r0) * E.L.n; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
      const int64_t r = i / E.L.n;
      const int o = static_cast<int>(i - r * E.L.n);
      store_out(y, yt, (r0 + r) * ldy + o, E.L.ob ? h2f(E.L.ob[e * E.so + o]) : 0.0f);
    }
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

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Shared memory and workspace of a call.
struct Plan {
  int nkt, row_tiles, tokens, ctas;
  int64_t kp;
  int na, nx, xk, xslot, staged, copies, off_book[2], off_table, off_scales, smem;
  size_t off_xe, off_sum, off_joined, off_xh, off_part, total;
};

// A token tile holds so many times the rows that the experts have on average: an
// expert above it is decoded twice, a larger tile leaves fewer x slots and less
// L1.  Routed unevenly (the most popular of 16 or 64 experts at two to three
// times the average), 2, 3 and 4 took 131 / 119 / 119 us (1000 x 2 of 16, 12 + 8
// bits), 239 / 229 / 237 (2000 x 2 of 16, 16 + 8) and 158 / 149 / 172 (512 x 8 of 64).
constexpr int kSpread = 3;
constexpr int kMaxCopied = 8;      // log2 entries of a book that may be kept eight times (32 KB at d <= 8)

// The kernel that serves a layer with the books of mask `staged` in shared
// memory: its compile-time index widths (0, 0: the general one).
struct Widths {
  int b1, b2;
};
Widths widths_of(const Layer& L, int staged) {
  const int b1 = L.b[0], b2 = L.nb == 2 ? L.b[1] : 0;
  if (L.d <= 8 && staged == (L.nb == 2 ? 3 : 1)) {
    if (b1 == 12 && (b2 == 8 || b2 == 4 || b2 == 0)) return {b1, b2};
    if (b1 == 8 && (b2 == 8 || b2 == 0)) return {b1, b2};
  }
  if (L.d == 8 && b1 == 16 && staged == (L.nb == 2 ? 2 : 0) && (b2 == 0 || b2 == 8)) return {b1, b2};
  return {0, 0};
}

// Whether books (mask `staged`, those of `copies` eight times) and rings fit for
// token tiles of at most `tokens` rows: at least two W slots, and x slots of
// several steps, two at least, or of one step (of a half), three at least.
bool fit(const Experts& E, int m, int staged, int copies, int tokens, Plan* p) {
  const Layer& L = E.L;
  const int ch = L.d > 8 ? 2 : 1;
  int off = 0;
  for (int b = 0; b < 2; ++b) {
    p->off_book[b] = off;
    if (staged & (1 << b)) off += ((1 << L.b[b]) * 16 * ch) << ((copies >> b) & 1 ? 3 : 0);
  }
  p->off_table = off;
  off += 16 * (E.e + 1) + 8 * (device_sm_count() + 1);
  p->off_scales = off = (off + 15) / 16 * 16;
  off += 2 * 8 * std::min((m + 15) / 16 * 16, tokens);
  const int room = device_smem_optin() - 2048 - off;
  const bool in_tmem = w_in_tmem(widths_of(L, staged).b1);
  const int acc = acc_rows(in_tmem), atile = in_tmem ? 0 : kATile;
  p->tokens = std::min((m + 15) / 16 * 16, tokens);
  const int slot = box_rows(box_of(std::min(p->tokens, acc)), acc) * 128;      // bytes of a step of x'
  if (p->tokens <= acc) {
    p->na = kMaxA;
    for (p->xk = 4; p->xk > 1 && (room - p->na * atile) / (slot * p->xk) < 2; p->xk /= 2) {}
    // three slots of several steps are enough to stay ahead; what is left serves
    // the index words as L1
    p->nx = std::min(p->xk > 1 ? 3 : kMaxX, (room - p->na * atile) / (slot * p->xk));
    if (p->nx < (p->xk > 1 ? 2 : 3)) return false;
  } else {
    p->xk = 1;
    p->na = kMaxA;
    while (p->na > 2 && (room - p->na * atile) / slot < 3) --p->na;
    p->nx = std::min(kMaxX, (room - p->na * atile) / slot);
    if (p->nx < 3) return false;
  }
  p->xslot = slot * p->xk;
  p->staged = staged;
  p->copies = copies;
  p->smem = 2048 + p->na * atile + p->nx * p->xslot + off;
  return true;
}

Plan plan_experts(const Experts& E, int m) {
  Plan p{};
  const Layer& L = E.L;
  const int per = L.d > 8 ? 4 : 8;                             // vectors of a step
  p.nkt = (L.nvec - 1) / per + 1;
  p.kp = static_cast<int64_t>(p.nkt) * 64;
  p.row_tiles = (L.n - 1) / kRowTile + 1;
  p.ctas = device_sm_count();
  // What comes first: books in shared memory (both, the first, the second; one
  // of more than 2^13 entries never fits), then the token tile (W is decoded once
  // per token tile), then eight copies of small books (their lookups meet no bank
  // conflicts).  The tile: the smallest of 64, 128, one and two accumulators that
  // holds kSpread times the rows that the experts have on average.
  const int both = L.nb == 2 ? 3 : 1;
  int small = 0;
  for (int b = 0; b < L.nb; ++b) small |= L.b[b] <= kMaxCopied ? 1 << b : 0;
  bool done = false;
  for (int mask : {both, 1, both & 2, 0}) {
    bool ok = true;
    for (int b = 0; b < L.nb; ++b) ok &= !(mask & (1 << b)) || L.b[b] <= 13;
    if (!ok) continue;
    const int acc = acc_rows(w_in_tmem(widths_of(L, mask).b1));
    const int sizes[5] = {2 * acc, acc, 128, 64, 32};
    int first = 3;
    while (first > 0 && static_cast<int64_t>(sizes[first]) * E.e < kSpread * static_cast<int64_t>(m)) --first;
    // short rows of W: smaller tiles where the steps cannot occupy every CTA
    // (9104 rows of 161 x 66: 123 us in tiles of 512 on ten CTAs, 37 us in tiles of 64)
    while (first < 3 && static_cast<int64_t>(p.row_tiles) * ((m + sizes[first] - 1) / sizes[first]) * p.nkt <
                            static_cast<int64_t>(kMinSteps) * p.ctas)
      ++first;
    for (int i = first; i < 5; ++i)
      for (int copies : {mask & small, mask & small & 2, 0})
        if (!done && fit(E, m, mask, copies, sizes[i], &p)) done = true;
  }
  p.off_xe = 256;
  p.off_sum = p.off_xe + round256(static_cast<size_t>(m) * 4);
  p.off_joined = p.off_sum + round256(static_cast<size_t>(m) * 4);
  p.off_xh = p.off_joined + round256(static_cast<size_t>(p.ctas) * 4);
  p.off_part = p.off_xh + round256(static_cast<size_t>(m) * p.kp * 2);
  p.total = p.off_part + static_cast<size_t>(p.ctas) * 2 * p.tokens * kRowTile * 4;
  return p;
}

// Tiles are counted in 31 bits: at most (experts + m / 16) of grouped rows
// (tiles hold 32 rows or all m) times the row tiles of W.
bool too_many_tiles(const Experts& E, int m) {
  const int64_t row_tiles = (static_cast<int64_t>(E.L.n) + kRowTile - 1) / kRowTile;
  return (E.e + static_cast<int64_t>(m) / 16) * row_tiles > 0x7FFFFFFFLL;
}

size_t experts_bytes(const Experts& E, int m) { return E.L.kin == 0 ? 256 : plan_experts(E, m).total; }

long long wait_budget() {
  if (const char* env = std::getenv("VQ_WAIT_BUDGET")) return std::atoll(env);
  return 4000000000LL;
}

template <int LAYOUT>
auto pick_kernel(const Layer& L, int staged) {
  const Widths w = widths_of(L, staged);
  if (w.b1 == 12 && w.b2 == 8) return gemm_experts_kernel<LAYOUT, 12, 8>;
  if (w.b1 == 12 && w.b2 == 4) return gemm_experts_kernel<LAYOUT, 12, 4>;
  if (w.b1 == 12) return gemm_experts_kernel<LAYOUT, 12, 0>;
  if (w.b1 == 8 && w.b2 == 8) return gemm_experts_kernel<LAYOUT, 8, 8>;
  if (w.b1 == 8) return gemm_experts_kernel<LAYOUT, 8, 0>;
  if (w.b1 == 16 && w.b2 == 8) return gemm_experts_kernel<LAYOUT, 16, 8>;
  if (w.b1 == 16) return gemm_experts_kernel<LAYOUT, 16, 0>;
  return gemm_experts_kernel<LAYOUT, 0, 0>;
}

vq_status launch_gemm_experts(const Experts& E, const void* x, bool x_fp16, int x_rows, int64_t ldx,
                              const int32_t* rows, const int32_t* offsets, int m, void* y, vq_dtype yt, int64_t ldy,
                              void* ws, cudaStream_t stream) {
  const Layer& L = E.L;
  if (L.kin == 0) {
    count_launch();
    experts_bias_kernel<<<device_sm_count(), 256, 0, stream>>>(E, offsets, m, y, yt, ldy);
    return cuda_status(cudaGetLastError());
  }
  const Plan p = plan_experts(E, m);
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint16_t* xh = reinterpret_cast<uint16_t*>(w + p.off_xh);
  Args g{};
  g.E = E;
  g.offsets = offsets;
  g.m = m;
  g.nkt = p.nkt;
  g.row_tiles = p.row_tiles;
  g.tokens = p.tokens;
  g.na = p.na;
  g.nx = p.nx;
  g.xk = p.xk;
  g.xslot = p.xslot;
  g.staged = p.staged;
  g.copies = p.copies;
  g.off_book[0] = p.off_book[0];
  g.off_book[1] = p.off_book[1];
  g.off_table = p.off_table;
  g.off_scales = p.off_scales;
  float* xe = reinterpret_cast<float*>(w + p.off_xe);
  float* xsum = reinterpret_cast<float*>(w + p.off_sum);
  g.xe = xe;
  g.xsum = xsum;
  g.y = y;
  g.yt = yt;
  g.ldy = ldy;
  g.part = reinterpret_cast<float*>(w + p.off_part);
  g.joined = reinterpret_cast<int*>(w + p.off_joined);
  g.status = reinterpret_cast<int*>(w);
  g.budget = wait_budget();
  Maps maps;
  const int acc = acc_rows(w_in_tmem(widths_of(L, p.staged).b1));
  for (int i = 0; i < kBoxes; ++i)
    if (!make_map_f16_steps(&maps.m[i], xh, p.nkt, m, p.kp, box_rows(i, acc), p.xk)) return VQ_ERR_CUDA;
  const int vec = aligned(x, 16) && ldx % 8 == 0;
  count_launch();
  experts_prep_kernel<<<m, kPrepThreads, 0, stream>>>(static_cast<const uint16_t*>(x), x_fp16 ? 1 : 0, x_rows, ldx, rows,
                                                      offsets, E.e, L.kin, L.d, p.kp, vec, xh, xe, xsum, g.joined, p.ctas);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  auto k = L.layout == VQ_IDX_TILE4 ? pick_kernel<VQ_IDX_TILE4>(L, p.staged) : pick_kernel<VQ_IDX_ROWS>(L, p.staged);
  e = set_func_attr(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
  if (e != cudaSuccess) return cuda_status(e);
  count_launch();
  return cuda_status(launch_pdl(k, dim3(p.ctas), dim3(kThreads), p.smem, stream, maps, g));
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
  if (m > kMaxGroupedRows || too_many_tiles(E, m)) return VQ_ERR_UNSUPPORTED;
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
  if (m > kMaxGroupedRows || too_many_tiles(E, m)) return VQ_ERR_UNSUPPORTED;
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
