// Low-rank adapters of many requests added to a shared projection's output:
//   out[m][n] = bf16(y[m][n] + s_i * sum_r B_i[n][r] t[m][r]),  t[m][r] = sum_k x[m][k] A_i[r][k]
// with i the adapter of the request that row m belongs to.  The rows of a request are contiguous.
//
// Two kernels.  "Shrink" forms t in binary32 partial sums over slices of K (a workspace
// [slices][M][R]; the second kernel adds the slices in order, so the result does not depend on
// timing).  "Expand" multiplies t, scaled, with B and adds y.  Its products run on bf16 tensor
// cores with t as the sum of two bf16 numbers: t to 2^-17, so the update is off by 2^-17 of the sum of
// its terms' magnitudes (half a step of a bf16 output is 2^-9 to 2^-8 of it: where y and the update, or
// its terms, cancel to less than 2^-8 of their size, the former counts).  Sums in binary32.
//
// Rows go in tiles of BM of one request.  Tile number t -> (request, row) without a prefix sum:
// request s owns the tile numbers from start[s] / BM + s on; as ceil(len / BM) <= (start + len) /
// BM - start / BM + 1, the ranges do not meet, and M / BM + requests numbers cover them all.
//
// Both are bound by HBM: x once, y and out once.
//
// Shrink, tiles of 128 rows (long requests, plan() has the rule): tcgen05 MMAs of 128 x R on
// a ring of TMA stages of 64 k; two CTAs per SM keep 190 KB in flight.  Tiles of 16 rows (a token
// or a few per request): mma.sync, the block's warps share K, operands from global memory straight
// to fragments.  A fragment only needs A and B to use the same order of k, so a thread takes 8
// consecutive k (16 bytes) of a 32-wide slice for two k16 steps, and the four threads of a row
// read 64 consecutive bytes.
//
// Expand, large tiles: t lies in shared memory as tops and rest, y and B come and the result
// leaves by TMA in chunks of 64 columns, the products are tcgen05 MMAs of 128 x 64 into tensor
// memory.  Everything from global memory straight to mma.sync fragments was bound by the L1's line
// accesses (2.1 TB/s; 3.3 with B held in registers).  Small tiles: fragments as above, a warp holds
// t and goes along the columns.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "qs.h"
#include "qs_host.cuh"
#include "qs_launch.cuh"
#include "qs_ops.cuh"
#include "qs_ptx.cuh"

namespace qs {
namespace lora {

using ops::max3_nan;
using ops::mma_ss;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSmallRows = 16, kLargeRows = 128;  // rows of a tile
constexpr int kMaxRank = 128;
constexpr int kGroup = 64;                        // ranks a shrink block forms
constexpr int kSms = 148;
constexpr int kStepK = 64;                        // k of a TMA stage

struct Args {
  const uint16_t *x, *y, *a, *b;
  uint16_t* out;
  const float* scale;       // [adapters] or NULL
  const int32_t *start, *ids;
  float* part;              // [slices][M][R]
  int64_t M;
  int K, N, R, adapters, requests, slices;
};

struct Plan {
  bool large;     // tiles of kLargeRows rows
  int slices;     // of K
  int64_t tiles;  // tile numbers
};

inline Plan plan(int64_t M, int64_t K, int64_t R, int64_t requests) {
  Plan p;
  // Large tiles cost a fixed time each and pay from some rows per request on; small ones form up to 64
  // ranks in registers and read y and B once for each 16 rows.  By rows per request (uneven lengths),
  // large / small, us, M 8192, K and N 5120: R 16: 88 / 79 at 195, 80 / 79 at 256, 66 / 77 at 512; R 32:
  // 133 / 109 at 64, 116 / 109 at 80, 102 / 109 at 96; R 48: 141 / 130 at 64, 121 / 129 at 80; R 64: 172 /
  // 166 at 32, 142 / 163 at 48, 137 / 139 at 64; R 128: 386 / 351 at 24, 263 / 319 at 32.  M 3000, N
  // 13824: R 64: 132 / 116 at 48; R 128: 272 / 233 at 28.  The rule sees the mean only.  One long request
  // and 63 single tokens: 58 / 56 at M 2063 R 64, 113 / 116 at R 128, 65 / 99 at M 4000 R 64; 82 / 113 at M
  // 8000 R 32.  Little x in all: 21 / 15 at M 512 R 32, 42 / 36 at R 128, 18 / 14 at M 1024 K 1536 R 48.
  const int64_t least_rows = R <= 16 ? 256 : R <= 32 ? 96 : R <= 48 ? 72 : R <= 64 ? 56 : 32;
  p.large = M * K >= (1 << 22) && M / requests >= least_rows;
  const int rows = p.large ? kLargeRows : kSmallRows;
  p.tiles = M / rows + requests;
  const int64_t blocks = p.large ? p.tiles : p.tiles * ((R + kGroup - 1) / kGroup);
  // About two blocks per SM; small tiles: 64 k and more for each warp, large ones: 16 stages.  Small
  // tiles, 1, 2, 3, 4 blocks per SM, us: 256 rows of 64 requests, K and N 5120, R 32: 22.3, 16.3, 15.5,
  // 18.1; 64 tokens, N 15360, R 64: 34.8, 32.1, 38.0, 35.4.  32, 64, 128, 256 k a warp: one token, R 16:
  // 6.1, 5.7, 5.6, 7.0.
  int64_t n = 2 * kSms / blocks;
  const int64_t most = p.large ? K / (16 * kStepK) : K / 512;
  if (n > most) n = most;
  // The second kernel reads every slice of t once per column range.  1, 2, 4, 6, 8 slices, us: M 4099
  // of nine requests, K 13824, R 32: 93, 67, 56, 56, 56; M 2048, K 13824, R 64: 85, 57, 43, 45, 46;
  // M 512, R 128: 100, 70, 55, 66, 70.
  if (p.large && n > 4) n = 4;
  p.slices = static_cast<int>(n < 1 ? 1 : n);
  return p;
}

struct Tile {
  int row0, rows, adapter;  // rows == 0: nothing to do
};

// The tile of number t; called by all threads of the block.
__device__ __forceinline__ Tile find_tile(const Args& a, int64_t t, int bm) {
  int s;
  if (a.requests <= static_cast<int>(blockDim.x)) {
    // the ranges' first numbers grow with the request: count those not above t
    const int i = threadIdx.x;
    s = __syncthreads_count(i < a.requests && a.start[i] / bm + static_cast<int64_t>(i) <= t) - 1;
  } else {
    int lo = 0, hi = a.requests;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.start[mid] / bm + static_cast<int64_t>(mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    s = lo;
  }
  if (s < 0) return {0, 0, -1};
  const int64_t first = a.start[s], end = a.start[s + 1];
  const int id = a.ids[s];
  if (first < 0 || end < first || end > a.M || id < -1 || id >= a.adapters) return {0, 0, -1};
  const int64_t row0 = first + (t - (first / bm + s)) * bm;
  if (row0 < first || row0 >= end) return {0, 0, -1};
  return {static_cast<int>(row0), static_cast<int>(min(end - row0, static_cast<int64_t>(bm))), id};
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// Requests that find_tile need not come to (their rows lie behind the tile numbers, or before the
// request in front) are reported too, by one block of the second kernel while it waits for the first
// (in the first it took 0.5 us of 20).
__device__ __forceinline__ void report_bad_requests(const Args& a) {
  if (blockIdx.x != 0 || blockIdx.y != 0) return;
  bool bad = false;
  for (int s = threadIdx.x; s < a.requests; s += blockDim.x) {
    const int first = a.start[s], end = a.start[s + 1], id = a.ids[s];
    bad |= first < 0 || end < first || end > a.M || id < -1 || id >= a.adapters;
  }
  if (bad) atomicOr(&g_error_word, kErrIndex);
}

// The second kernel may be on the GPU before the first has ended (programmatic dependent launch).
// It waits for that end before it reads the sums, and every block of it does so before it leaves:
// what comes after it in the stream must find both done.
__device__ __forceinline__ void let_expand_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_shrink() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// t of a small tile: a block forms 16 rows x up to 64 ranks (NT groups of 8) over one slice of K;
// its warps share the slice's 32-wide steps and add their sums through shared memory in warp order.
template <int NT>
__global__ void __launch_bounds__(kThreads) shrink_small_kernel(const Args a) {
  extern __shared__ float sums[];  // [warps][16][8 * NT]
  const Tile tile = find_tile(a, blockIdx.x, kSmallRows);
  let_expand_start();
  if (tile.rows <= 0 || tile.adapter < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.z * kGroup;
  const int steps = a.K / 32, parts = a.slices * kWarps, part = blockIdx.y * kWarps + warp;
  const int k_begin = static_cast<int>(static_cast<int64_t>(steps) * part / parts) * 32;
  const int k_end = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts) * 32;

  float acc[NT][4] = {};
  const uint16_t* xp = a.x + static_cast<int64_t>(tile.row0 + g) * a.K + 8 * c;
  const uint16_t* ap =
      a.a + (static_cast<int64_t>(tile.adapter) * a.R + r0 + g) * a.K + 8 * c;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (int k = k_begin; k < k_end; k += 32) {
    uint4 xf[2], wf[NT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xf[h] = 8 * h + g < tile.rows ? ldg16(xp + static_cast<int64_t>(8 * h) * a.K + k) : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      wf[n] = r0 + 8 * n < a.R ? ldg16(ap + static_cast<int64_t>(8 * n) * a.K + k) : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma_bf16_16816(acc[n], xf[0].x, xf[1].x, xf[0].y, xf[1].y, wf[n].x, wf[n].y);
      mma_bf16_16816(acc[n], xf[0].z, xf[1].z, xf[0].w, xf[1].w, wf[n].z, wf[n].w);
    }
  }
  constexpr int cols = 8 * NT;
  float* mine = sums + warp * (16 * cols);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mine[(g + 8 * (e >> 1)) * cols + 8 * n + 2 * c + (e & 1)] = acc[n][e];
  __syncthreads();
  float* out = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + tile.row0) * a.R + r0;
  for (int i = threadIdx.x; i < tile.rows * cols; i += kThreads) {
    const int r = i % cols;
    if (r0 + r >= a.R) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * (16 * cols) + i];
    out[static_cast<int64_t>(i / cols) * a.R + r] = v;
  }
}

// t of a large tile: x rows (whoever's they are behind the request: their results are not
// written) times the adapter's R rows of A, one slice of K.  Warp 0 loads, warp 1 issues, warps
// 2-5 carry the sums from tensor memory to the workspace.
template <int RN>  // R rounded up to 16 (an MMA's columns): the rows loaded
struct ShrinkCfg {
  static constexpr int kX = kLargeRows * 128, kA = RN * 128, kStage = kX + kA;
  static constexpr int kStages = 100 * 1024 / kStage;  // two CTAs per SM
  static constexpr int kOffBar = kStages * kStage, kNumBars = 2 * kStages + 1;
  static constexpr int kSmemBytes = kOffBar + 8 * kNumBars + 16 + 1024;
  static constexpr int kTmemCols = RN <= 32 ? 32 : RN <= 64 ? 64 : 128;
  static_assert(kSmemBytes <= 113 * 1024, "two CTAs per SM");
};
constexpr int kShrinkThreads = 32 * 6;

template <int RN>
__global__ void __launch_bounds__(kShrinkThreads)
    shrink_large_kernel(const __grid_constant__ CUtensorMap tmX,
                        const __grid_constant__ CUtensorMap tmA, const Args a) {
  using C = ShrinkCfg<RN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* sp = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + C::kOffBar + 8 * C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const auto full = [&](int s) { return sbase + C::kOffBar + 8u * s; };
  const auto empty = [&](int s) { return full(C::kStages + s); };
  const uint32_t done = full(2 * C::kStages);
  const Tile tile = find_tile(a, blockIdx.x, kLargeRows);
  if (tile.rows <= 0 || tile.adapter < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = a.K / kStepK;
  const int k0 = static_cast<int>(static_cast<int64_t>(steps) * blockIdx.y / a.slices);
  const int n = static_cast<int>(static_cast<int64_t>(steps) * (blockIdx.y + 1) / a.slices) - k0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(full(i), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  let_expand_start();

  if (warp == 0 && lane == 0) {
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % C::kStages;
      if (!mbar_wait_bounded(empty(s), ((i / C::kStages) & 1) ^ 1, abort_flag, kErrWaitProducer))
        break;
      const uint32_t dst = sbase + s * C::kStage;
      mbar_arrive_expect_tx(full(s), C::kStage);
      tma_load_2d(dst, &tmX, (k0 + i) * kStepK, tile.row0, full(s));
      tma_load_2d(dst + C::kX, &tmA, (k0 + i) * kStepK, tile.adapter * a.R, full(s));
    }
    // no copy into this CTA's memory may outlive it
    for (int k = i > C::kStages ? i - C::kStages : 0; k < i; ++k)
      mbar_wait_limit(full(k % C::kStages), (k / C::kStages) & 1, kWaitTimeoutNs, kErrWaitTma);
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = ops::idesc_f16(kLargeRows, RN, false, false);
    for (int i = 0; i < n; ++i) {
      const int s = i % C::kStages;
      if (!mbar_wait_bounded(full(s), (i / C::kStages) & 1, abort_flag, kErrWaitTma)) break;
      tc_fence_after();
      const uint32_t x = sbase + s * C::kStage;
#pragma unroll
      for (int k = 0; k < kStepK / 16; ++k)
        mma_ss(tmem, smem_desc_sw128(x + 32 * k), smem_desc_sw128(x + C::kX + 32 * k), idesc,
                    i != 0 || k != 0);
      mma_commit(empty(s));
    }
    mma_commit(done);
    mbar_wait_limit(done, 0, kWaitTimeoutNs, kErrWaitMma);
  } else if (warp >= 2) {
    const bool ok = mbar_wait_bounded(done, 0, abort_flag, kErrWaitMma);
    __syncwarp();
    tc_fence_after();
    const int quarter = warp & 3, r = 32 * quarter + lane;  // the lanes of tensor memory it may read
    float* out = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + tile.row0 + r) * a.R;
#pragma unroll 1
    for (int c = 0; c < C::kTmemCols / 32; ++c) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 32 * c, v);
      tmem_wait_ld();
      if (r < tile.rows && ok)
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          if (32 * c + e < a.R)  // R is a multiple of 8
            *reinterpret_cast<uint4*>(out + 32 * c + e) =
                make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Eight consecutive ranks of a row of t, scaled, as two bf16 numbers each: their tops and the rest.
__device__ __forceinline__ void load_t(const Args& a, int64_t row, int k, float scale, bool there,
                                       uint4& hi, uint4& lo) {
  float t[8] = {};
  if (there && k < a.R) {
    const float* p = a.part + row * a.R + k;
#pragma unroll 4
    for (int i = 0; i < a.slices; ++i, p += a.M * a.R) {
      const float4 u = *reinterpret_cast<const float4*>(p);
      const float4 v = *reinterpret_cast<const float4*>(p + 4);
      t[0] += u.x, t[1] += u.y, t[2] += u.z, t[3] += u.w;
      t[4] += v.x, t[5] += v.y, t[6] += v.z, t[7] += v.w;
    }
  }
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p = t[2 * e] * scale, q = t[2 * e + 1] * scale;
    const __nv_bfloat162 top = __floats2bfloat162_rn(p, q);
    const float u = __low2float(top), v = __high2float(top);
    // an infinite t stays infinite: its remainder is 0, not inf - inf
    const __nv_bfloat162 rest =
        __floats2bfloat162_rn(isinf(u) ? 0.f : p - u, isinf(v) ? 0.f : q - v);
    h[e] = *reinterpret_cast<const uint32_t*>(&top);
    l[e] = *reinterpret_cast<const uint32_t*>(&rest);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// The sums of `count` columns from n on of one row that came out as NaN, formed again from t in one
// piece: times an infinite element of B the two parts of t give infinities of either sign, or 0 times
// infinity, where t itself gives one infinity.  A sum that is NaN by itself stays so, and the first
// such term ends it.
__device__ __noinline__ void sum_again(const Args& a, int64_t row, int adapter, int n, int count,
                                       float* sums) {
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  for (int e = 0; e < count && n + e < a.N; ++e) {
    if (sums[e] == sums[e]) continue;
    const uint16_t* b = a.b + (static_cast<int64_t>(adapter) * a.N + n + e) * a.R;
    float sum = 0.f;
    for (int r = 0; r < a.R && sum == sum; ++r) {
      float t = 0.f;
      for (int i = 0; i < a.slices; ++i) t += a.part[(i * a.M + row) * a.R + r];
      sum = fmaf(t * scale, __uint_as_float(static_cast<uint32_t>(b[r]) << 16), sum);
    }
    sums[e] = sum;
  }
}

// Two k16 steps of 16 rows x 8 columns: t as tops and rest, rows g (0) and g + 8 (1) of each.
__device__ __forceinline__ void mma_t(float (&acc)[4], const uint4 (&hi)[2], const uint4 (&lo)[2],
                                      const uint4& w) {
  mma_bf16_16816(acc, hi[0].x, hi[1].x, hi[0].y, hi[1].y, w.x, w.y);
  mma_bf16_16816(acc, lo[0].x, lo[1].x, lo[0].y, lo[1].y, w.x, w.y);
  mma_bf16_16816(acc, hi[0].z, hi[1].z, hi[0].w, hi[1].w, w.z, w.w);
  mma_bf16_16816(acc, lo[0].z, lo[1].z, lo[0].w, lo[1].w, w.z, w.w);
}

__device__ __forceinline__ void mma_tops(float (&acc)[4], const uint4 (&hi)[2], const uint4& w) {
  mma_bf16_16816(acc, hi[0].x, hi[1].x, hi[0].y, hi[1].y, w.x, w.y);
  mma_bf16_16816(acc, hi[0].z, hi[1].z, hi[0].w, hi[1].w, w.z, w.w);
}

// Whether one of the thread's sums is NaN.
__device__ __forceinline__ bool has_nan(const float (&acc)[4][4]) {
  float most[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    most[0] = max3_nan(most[0], acc[j][0], acc[j][1]);
    most[1] = max3_nan(most[1], acc[j][2], acc[j][3]);
  }
  return isnan(most[0] + most[1]);
}

// y + the sums of four n8 tiles, as bf16.  The tiles' column order inside their 32 is permuted so
// that a thread's share is 8 consecutive columns: y and out move in 16-byte pieces.
__device__ __forceinline__ uint4 add_y(const uint4& y, const float (&acc)[4][4], int half) {
  const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float u = __uint_as_float(yw[j] << 16), v = __uint_as_float(yw[j] & 0xFFFF0000u);
    const __nv_bfloat162 r = __floats2bfloat162_rn(u + acc[j][2 * half], v + acc[j][2 * half + 1]);
    o[j] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// B of 32 columns: rank group s, tile j, in the permuted order.
template <int KS>
__device__ __forceinline__ void load_b(const Args& a, int adapter, int n0, uint4 (&w)[KS][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = 32 * s + 8 * c, n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
      w[s][j] = k < a.R && n < a.N
                    ? ldg16(a.b + (static_cast<int64_t>(adapter) * a.N + n) * a.R + k)
                    : make_uint4(0, 0, 0, 0);
    }
}

// Large tiles.  KH: 64-wide parts of the rank.  Warp 0 loads, warp 1 issues, warps 2-5 (a row to a
// thread) put t into shared memory, then add y to the products in the place of y; warp 6 sends the
// chunks off and gives their stages back as soon as they have been read.
template <int KH>
struct ExpandCfg {
  static constexpr int kCols = 64;                                   // of a chunk
  static constexpr int kT = KH * kLargeRows * 128;                   // tops or rest
  static constexpr int kY = kLargeRows * 128, kB = KH * kCols * 128, kStage = kY + kB;
  static constexpr int kStages = KH == 1 ? 3 : 4;                    // two CTAs per SM, or one
  static constexpr int kOffStage = 2 * kT, kOffBar = kOffStage + kStages * kStage;
  static constexpr int kFull = 0, kEmpty = kStages, kDFull = 2 * kStages, kDFree = kDFull + 2;
  static constexpr int kSum = kDFree + 2, kTFull = kSum + kStages, kDrain = kTFull + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr int kSmemBytes = kOffBar + 8 * kNumBars + 16 + 1024;
  static_assert(kSmemBytes <= (KH == 1 ? 113 : 227) * 1024, "shared memory per CTA");
};
constexpr int kExpandThreads = 32 * 7;

template <int KH>
__global__ void __launch_bounds__(kExpandThreads)
    expand_large_kernel(const __grid_constant__ CUtensorMap tmY,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmO,
                        const __grid_constant__ Args a, int chunks_each) {
  using C = ExpandCfg<KH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* sp = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + C::kOffBar + 8 * C::kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
  const Tile tile = find_tile(a, blockIdx.x, kLargeRows);
  report_bad_requests(a);
  const bool turned = tile.adapter >= 0;
  const int chunks = (a.N + C::kCols - 1) / C::kCols;
  const int first = blockIdx.y * chunks_each, n = min(chunks_each, chunks - first);
  if (tile.rows <= 0 || n <= 0 || !turned) {
    if (tile.rows > 0 && n > 0 && a.out != a.y) {  // no adapter: y as it is
      const int pieces = min(n * C::kCols, a.N - first * C::kCols) / 8;
      for (int64_t i = threadIdx.x; i < static_cast<int64_t>(tile.rows) * pieces; i += kExpandThreads) {
        const int64_t at = (tile.row0 + i / pieces) * a.N + first * C::kCols + 8 * (i % pieces);
        *reinterpret_cast<uint4*>(a.out + at) = *reinterpret_cast<const uint4*>(a.y + at);
      }
    }
    wait_for_shrink();
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), i >= C::kDFree && i <= C::kTFull ? 4 : 1);  // the four row warps'
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 2 * C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // After a wait that gave up, a thread waits for nothing more and runs its loops out.
  bool ok = true;
  const auto wait = [&](int i, uint32_t parity, unsigned err) {
    if (ok) ok = mbar_wait_bounded(bar(i), parity, abort_flag, err);
  };

  if (warp == 0 && lane == 0) {
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % C::kStages;
      wait(C::kEmpty + s, ((i / C::kStages) & 1) ^ 1, kErrWaitProducer);
      if (!ok) break;
      const uint32_t dst = sbase + C::kOffStage + s * C::kStage;
      const int c0 = (first + i) * C::kCols;
      mbar_arrive_expect_tx(bar(C::kFull + s), C::kStage);
      tma_load_2d(dst, &tmY, c0, tile.row0, bar(C::kFull + s));
      for (int h = 0; h < KH; ++h)
        tma_load_2d(dst + C::kY + h * C::kCols * 128, &tmB, 64 * h, tile.adapter * a.N + c0,
                    bar(C::kFull + s));
    }
    // no copy into this CTA's memory may outlive it
    for (int k = i > C::kStages ? i - C::kStages : 0; k < i; ++k)
      mbar_wait_limit(bar(C::kFull + k % C::kStages), (k / C::kStages) & 1, kWaitTimeoutNs,
                      kErrWaitTma);
  } else if (warp == 1 && lane == 0) {
    constexpr uint32_t idesc = ops::idesc_f16(kLargeRows, C::kCols, false, false);
    const int steps = (a.R + 15) / 16;
    wait(C::kTFull, 0, kErrWaitEpilogue);
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % C::kStages, buf = i & 1;
      wait(C::kFull + s, (i / C::kStages) & 1, kErrWaitTma);
      wait(C::kDFree + buf, ((i >> 1) & 1) ^ 1, kErrWaitEpilogue);
      if (!ok) break;
      tc_fence_after();
      const uint32_t b = sbase + C::kOffStage + s * C::kStage + C::kY;
      for (int part = 0; part < 2; ++part)  // tops, rest
        for (int k = 0; k < steps; ++k)
          mma_ss(tmem + C::kCols * buf,
                      smem_desc_sw128(sbase + part * C::kT + (k / 4) * kLargeRows * 128 + (k % 4) * 32),
                      smem_desc_sw128(b + (k / 4) * C::kCols * 128 + (k % 4) * 32), idesc,
                      part != 0 || k != 0);
      mma_commit(bar(C::kDFull + buf));
    }
    mma_commit(bar(C::kDrain));
    mbar_wait_limit(bar(C::kDrain), 0, kWaitTimeoutNs, kErrWaitMma);
  } else if (warp >= 2 && warp < 6) {
    const int thread = threadIdx.x - 64;
    wait_for_shrink();
    {
      const float scale = a.scale ? a.scale[tile.adapter] : 1.f;
#pragma unroll 4
      for (int i = thread; i < kLargeRows * 8 * KH; i += 128) {
        const int r = i / (8 * KH), p = i % (8 * KH);  // row, piece of 8 ranks
        uint4 hi, lo;
        load_t(a, tile.row0 + r, 8 * p, scale, r < tile.rows, hi, lo);
        uint8_t* at = sp + (p / 8) * kLargeRows * 128 + r * 128 + 16 * ((p & 7) ^ (r & 7));
        *reinterpret_cast<uint4*>(at) = hi;
        *reinterpret_cast<uint4*>(at + C::kT) = lo;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kTFull));
    }
    const int quarter = warp & 3, r = 32 * quarter + lane;  // the lanes of tensor memory it may read
    const bool whole = tile.rows == kLargeRows;
    for (int i = 0; i < n; ++i) {
      const int s = i % C::kStages, buf = i & 1, c0 = (first + i) * C::kCols;
      wait(C::kFull + s, (i / C::kStages) & 1, kErrWaitTma);
      wait(C::kDFull + buf, (i >> 1) & 1, kErrWaitMma);
      __syncwarp();
      tc_fence_after();
      uint8_t* y = sp + C::kOffStage + s * C::kStage + r * 128;
      uint16_t* out = a.out + (static_cast<int64_t>(tile.row0) + r) * a.N + c0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + C::kCols * buf + 32 * h, d);
        tmem_wait_ld();
        float most[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          most[0] = max3_nan(most[0], __uint_as_float(d[e]), __uint_as_float(d[e + 1]));
          most[1] = max3_nan(most[1], __uint_as_float(d[e + 2]), __uint_as_float(d[e + 3]));
        }
        if (isnan(most[0] + most[1]) && r < tile.rows && ok) {
          float sums[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) sums[e] = __uint_as_float(d[e]);
          sum_again(a, tile.row0 + r, tile.adapter, c0 + 32 * h, 32, sums);
#pragma unroll
          for (int e = 0; e < 32; ++e) d[e] = __float_as_uint(sums[e]);
        }
        __syncwarp();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4* at = reinterpret_cast<uint4*>(y + 16 * ((4 * h + p) ^ (r & 7)));
          const uint4 v = *at;
          const uint32_t yw[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 e = __floats2bfloat162_rn(
                __uint_as_float(yw[j] << 16) + __uint_as_float(d[8 * p + 2 * j]),
                __uint_as_float(yw[j] & 0xFFFF0000u) + __uint_as_float(d[8 * p + 2 * j + 1]));
            o[j] = *reinterpret_cast<const uint32_t*>(&e);
          }
          if (whole)
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          else if (r < tile.rows && ok && c0 + 32 * h + 8 * p < a.N)
            *reinterpret_cast<uint4*>(out + 32 * h + 8 * p) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(C::kDFree + buf));
        mbar_arrive(bar(C::kSum + s));
      }
    }
  } else if (warp == 6 && lane == 0) {
    for (int i = 0; i < n && ok; ++i) {
      const int s = i % C::kStages;
      wait(C::kSum + s, (i / C::kStages) & 1, kErrWaitEpilogue);
      if (!ok) break;
      if (tile.rows == kLargeRows) {
        asm volatile(
            "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
            "cp.async.bulk.commit_group;\n\t"
            "cp.async.bulk.wait_group.read 0;" ::"l"(reinterpret_cast<uint64_t>(&tmO)),
            "r"((first + i) * C::kCols), "r"(tile.row0), "r"(sbase + C::kOffStage + s * C::kStage)
            : "memory");
      }
      mbar_arrive(bar(C::kEmpty + s));
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * C::kCols);
}

// Small tiles: the warp's t in registers, 32 columns at a time.
template <int KS>
__global__ void __launch_bounds__(kThreads) expand_small_kernel(const Args a, int cols_per_block) {
  const Tile tile = find_tile(a, blockIdx.x, kSmallRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const bool turned = tile.adapter >= 0;
  report_bad_requests(a);
  wait_for_shrink();
  if (tile.rows <= 0 || (!turned && a.out == a.y)) return;
  const int n_begin = blockIdx.y * cols_per_block + 32 * warp;
  const int n_end = min(a.N, (static_cast<int>(blockIdx.y) + 1) * cols_per_block);
  uint4 hi[KS][2], lo[KS][2];
  const float scale = turned && a.scale ? a.scale[tile.adapter] : 1.f;
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      load_t(a, tile.row0 + g + 8 * h, 32 * s + 8 * c, scale, turned && g + 8 * h < tile.rows,
             hi[s][h], lo[s][h]);
  const auto there = [&](int n0, int h) { return n0 + 8 * c < a.N && g + 8 * h < tile.rows; };
  const auto offset = [&](int n0, int h) {
    return static_cast<int64_t>(tile.row0 + g + 8 * h) * a.N + n0 + 8 * c;
  };
  const auto load_y = [&](int n0, int h) {
    return there(n0, h) ? *reinterpret_cast<const uint4*>(a.y + offset(n0, h)) : make_uint4(0, 0, 0, 0);
  };
  bool again = false;
  // Two groups at a time for every rank, us: 42.7 for 40.3 (64 tokens, R 128), 98.2 for 96.1 (M 4000 of
  // 40 requests, R 8), 12.6 for 13.0 (M 300, N 2048, R 72).
  constexpr int kUnroll = KS == 1 ? 3 : KS == 2 ? 2 : 1;
#pragma unroll kUnroll
  for (int n0 = n_begin; n0 < n_end; n0 += 32 * kWarps) {
    uint4 y[2], w[KS][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) y[h] = load_y(n0, h);
    float acc[4][4] = {};
    if (turned) {
      load_b<KS>(a, tile.adapter, n0, w);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_t(acc[j], hi[s], lo[s], w[s][j]);
    }
    const bool nan = has_nan(acc);
    again |= nan;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (there(n0, h) && !nan)
        *reinterpret_cast<uint4*>(a.out + offset(n0, h)) = turned ? add_y(y[h], acc, h) : y[h];
  }
  // Times an infinite element of B the tops give the infinity that t does, the rest one of its own
  // sign, or 0 times infinity: a sum of both that is NaN is the tops' alone.  Such pieces were left
  // out above, and are formed again here: a branch in the loop cost 2 to 8 us of 20 to 35.
  if (!__any_sync(0xffffffffu, again)) return;
#pragma unroll 1
  for (int n0 = n_begin; n0 < n_end; n0 += 32 * kWarps) {
    uint4 w[KS][4];
    float acc[4][4] = {}, top[4][4] = {};
    load_b<KS>(a, tile.adapter, n0, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        mma_t(acc[j], hi[s], lo[s], w[s][j]);
        mma_tops(top[j], hi[s], w[s][j]);
      }
    }
    const bool nan = has_nan(acc);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!there(n0, h) || !nan) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 2 * h; e < 2 * h + 2; ++e) acc[j][e] = isnan(acc[j][e]) ? top[j][e] : acc[j][e];
      *reinterpret_cast<uint4*>(a.out + offset(n0, h)) = add_y(load_y(n0, h), acc, h);
    }
  }
}

template <int NT>
cudaError_t launch_shrink_small(const Args& a, const Plan& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.tiles), a.slices, (a.R + kGroup - 1) / kGroup);
  const int smem = kWarps * 16 * 8 * NT * static_cast<int>(sizeof(float));  // 32 KB at most
  shrink_small_kernel<NT><<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int RN>
cudaError_t launch_shrink_large(const Args& a, const Plan& p, cudaStream_t stream) {
  CUtensorMap x, w;
  if (!make_tensor_map_2d(&x, a.x, a.K, a.M, kStepK, kLargeRows, true, 2) ||
      !make_tensor_map_2d(&w, a.a, a.K, static_cast<uint64_t>(a.adapters) * a.R, kStepK, RN, true, 2))
    return cudaErrorInvalidValue;
  auto kern = shrink_large_kernel<RN>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             ShrinkCfg<RN>::kSmemBytes);
  if (e != cudaSuccess) return e;
  kern<<<dim3(static_cast<unsigned>(p.tiles), a.slices), kShrinkThreads, ShrinkCfg<RN>::kSmemBytes,
         stream>>>(x, w, a);
  return cudaGetLastError();
}

// A block's t in chunks of y, by bytes.
inline int64_t t_chunks(const Args& a) {
  return (static_cast<int64_t>(a.R) * a.slices * 4 + 127) / 128;
}

// Column chunks of a large tile's block.  A tile's last block may have fewer; the GPU takes the full
// ones first.  The time of `slots` blocks at once is counted in chunks, a block's beginning and end as
// two and two for each of its t's, for one to three rounds of blocks, and the shortest taken.
// One, two, three, four rounds, us: R 64, M 32760, K 5120, N 13824: 426, 428, 423, 429; N 5120: 209,
// 215, 221, 222; R 32, M 8192, N 15360: 112, 121, 133, 142; R 128, M 32760, N 13824: 620, 571, 634,
// 621; R 48, M 20000, N 10240: 261, 223, 216, 228.  The choice is the best of these, or within 1.5 %.
inline int64_t chunks_each(int64_t tiles, int64_t chunks, int64_t t, int64_t slots) {
  const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  int64_t best = 0, least = 0;
  for (int64_t rounds = 1; rounds <= 3; ++rounds) {
    int64_t each = up(tiles * chunks, slots * rounds);
    each = each > chunks ? chunks : each < t ? t : each;  // t is not to be more to read than y
    const int64_t ranges = up(chunks, each), full = tiles * (ranges - 1), begin = 2 + 2 * t;
    const int64_t cost_full = each + begin, cost_last = chunks - each * (ranges - 1) + begin;
    const int64_t used = full % slots;
    int64_t rest;  // the last, partly filled round of full blocks, and the tiles' last ones
    if (used == 0) {
      rest = up(tiles, slots) * cost_last;
    } else {
      // the last ones on the slots left free, or also on the others behind the full ones
      const int64_t alone = up(tiles, slots - used) * cost_last;
      const int64_t left = tiles - (slots - used) * (cost_full / cost_last);
      const int64_t shared = cost_full + (left > 0 ? up(left, slots) * cost_last : 0);
      rest = alone < cost_full ? cost_full : alone < shared ? alone : shared;
    }
    const int64_t cost = full / slots * cost_full + rest;
    if (rounds == 1 || cost < least) best = each, least = cost;
  }
  return best;
}

template <int KH>
cudaError_t launch_expand_large(const Args& a, const Plan& p, cudaStream_t stream) {
  using C = ExpandCfg<KH>;
  CUtensorMap y, w, o;
  if (!make_tensor_map_2d(&y, a.y, a.N, a.M, C::kCols, kLargeRows, true, 2) ||
      !make_tensor_map_2d(&w, a.b, a.R, static_cast<uint64_t>(a.adapters) * a.N, 64, C::kCols, true, 2) ||
      !make_tensor_map_2d(&o, a.out, a.N, a.M, C::kCols, kLargeRows, true, 2))
    return cudaErrorInvalidValue;
  auto kern = expand_large_kernel<KH>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (a.N + C::kCols - 1) / C::kCols;
  const int64_t each = chunks_each(p.tiles, chunks, t_chunks(a), (KH == 1 ? 2 : 1) * kSms);
  const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>((chunks + each - 1) / each));
  return launch_behind(kern, grid, kExpandThreads, C::kSmemBytes, stream, y, w, o, a,
                       static_cast<int>(each));
}

template <int KS>
cudaError_t launch_expand_small(const Args& a, const Plan& p, cudaStream_t stream) {
  // A block's t costs as much as a few column groups: about two blocks per SM, up to sixteen groups.
  // With 2, 5, 8 blocks per SM, us: 64 tokens, N 15360, R 16: 19.1, 20.1, 22.9; N 5120, R 128: 40.4,
  // 59.6, 59.5; 512 rows, R 64: 21.7, 25.8, 30.2.  Up to 8, 16, 32 groups: M 8000 of 64 requests, N
  // 8960, R 16: 104, 98, 98.
  const int64_t groups = (a.N + 32 * kWarps - 1) / (32 * kWarps);
  int64_t each = p.tiles * groups / (2 * kSms);
  each = each < 1 ? 1 : each > 16 ? 16 : each;
  const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>((groups + each - 1) / each));
  return launch_behind(expand_small_kernel<KS>, grid, kThreads, 0, stream, a,
                       static_cast<int>(32 * kWarps * each));
}

inline cudaError_t launch(const Args& a, const Plan& p, cudaStream_t stream) {
  cudaError_t e;
  if (p.large)
    switch ((a.R + 15) / 16) {
      case 1: e = launch_shrink_large<16>(a, p, stream); break;
      case 2: e = launch_shrink_large<32>(a, p, stream); break;
      case 3: e = launch_shrink_large<48>(a, p, stream); break;
      case 4: e = launch_shrink_large<64>(a, p, stream); break;
      case 5: e = launch_shrink_large<80>(a, p, stream); break;
      case 6: e = launch_shrink_large<96>(a, p, stream); break;
      case 7: e = launch_shrink_large<112>(a, p, stream); break;
      default: e = launch_shrink_large<128>(a, p, stream); break;
    }
  else if (a.R <= 8)
    e = launch_shrink_small<1>(a, p, stream);
  else if (a.R <= 16)
    e = launch_shrink_small<2>(a, p, stream);
  else if (a.R <= 32)
    e = launch_shrink_small<4>(a, p, stream);
  else
    e = launch_shrink_small<8>(a, p, stream);
  if (e != cudaSuccess) return e;
  if (p.large)
    return a.R <= 64 ? launch_expand_large<1>(a, p, stream) : launch_expand_large<2>(a, p, stream);
  switch ((a.R + 31) / 32) {
    case 1: return launch_expand_small<1>(a, p, stream);
    case 2: return launch_expand_small<2>(a, p, stream);
    case 3: return launch_expand_small<3>(a, p, stream);
    default: return launch_expand_small<4>(a, p, stream);
  }
}

}  // namespace lora
}  // namespace qs
