// Low-rank adapters of many requests added to a shared projection's output:
//   out[m][n] = bf16(y[m][n] + s_i * sum_r B_i[n][r] t[m][r]),  t[m][r] = sum_k x[m][k] A_i[r][k]
// with i the adapter of the request that row m belongs to.  The rows of a request are contiguous.
//
// Two kernels.  "Shrink" forms t in binary32 partial sums over slices of K (a workspace
// [slices][M][R]; the second kernel adds the slices in order, so the result does not depend on
// timing).  "Expand" multiplies t, scaled, with B and adds y.  Its products run on bf16 tensor
// cores with t as the sum of two bf16 numbers (t to 2^-17, below a bf16 output's half step
// whatever the ratio of the update to y), sums in binary32.
//
// Rows go in tiles of BM of one request.  Tile number t -> (request, row) without a prefix sum:
// request s owns the tile numbers from start[s] / BM + s on; as ceil(len / BM) <= (start + len) /
// BM - start / BM + 1, the ranges do not meet, and M / BM + requests numbers cover them all.
//
// Operands go from global memory straight to mma fragments: a fragment only needs A and B to use
// the same order of k, so a thread takes 8 consecutive k (16 bytes) of a 32-wide slice for two
// k16 steps, and the four threads of a row read 64 consecutive bytes.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "qs.h"
#include "qs_ptx.cuh"

namespace qs {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSmallRows = 16, kLargeRows = 128;  // rows of a tile
constexpr int kMaxRank = 128;
constexpr int kGroup = 64;                        // ranks a shrink block forms
constexpr int kSms = 148;

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
  p.large = M / requests >= kLargeRows / 2;
  const int rows = p.large ? kLargeRows : kSmallRows;
  p.tiles = M / rows + requests;
  const int64_t blocks = p.tiles * ((R + kGroup - 1) / kGroup) * (p.large ? kLargeRows / 32 : 1);
  int64_t s = (2 * kSms + blocks - 1) / blocks;
  const int64_t most = K / 512 > 0 ? K / 512 : 1;  // 64 k and more for each warp
  p.slices = static_cast<int>(s < 1 ? 1 : s > most ? most : s);
  return p;
}

struct Tile {
  int row0, rows, adapter;  // rows == 0: nothing to do
};

// The tile of number t; called by all threads of the block.
__device__ __forceinline__ Tile find_tile(const Args& a, int64_t t, int bm) {
  int s;
  if (a.requests <= kThreads) {
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
  if (first < 0 || end < first || end > a.M || id < -1 || id >= a.adapters) {
    if (threadIdx.x == 0) atomicOr(&g_error_word, kErrIndex);
    return {0, 0, -1};
  }
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

// t: a block forms 16 * MT rows x up to 64 ranks (NT groups of 8) over one slice of K; its warps
// share the slice's 32-wide steps and add their sums through shared memory in warp order.
template <int MT, int NT>
__global__ void __launch_bounds__(kThreads) shrink_kernel(const Args a, int bm) {
  extern __shared__ float sums[];  // [warps][16 * MT][8 * NT]
  const int sub = bm / (16 * MT);  // blocks per tile
  const Tile tile = find_tile(a, blockIdx.x / sub, bm);
  const int skip = (blockIdx.x % sub) * 16 * MT;
  const int rows = min(tile.rows - skip, 16 * MT);
  if (rows <= 0 || tile.adapter < 0) return;
  const int row0 = tile.row0 + skip;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int r0 = blockIdx.z * kGroup;
  const int steps = a.K / 32, parts = a.slices * kWarps, part = blockIdx.y * kWarps + warp;
  const int k_begin = static_cast<int>(static_cast<int64_t>(steps) * part / parts) * 32;
  const int k_end = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / parts) * 32;

  float acc[MT][NT][4] = {};
  const uint16_t* xp = a.x + static_cast<int64_t>(row0 + g) * a.K + 8 * c;
  const uint16_t* ap =
      a.a + (static_cast<int64_t>(tile.adapter) * a.R + r0 + g) * a.K + 8 * c;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int k = k_begin; k < k_end; k += 32) {
    uint4 xf[MT][2], wf[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        xf[m][h] = 16 * m + 8 * h + g < rows
                       ? ldg16(xp + static_cast<int64_t>(16 * m + 8 * h) * a.K + k)
                       : zero;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      wf[n] = r0 + 8 * n < a.R ? ldg16(ap + static_cast<int64_t>(8 * n) * a.K + k) : zero;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_bf16_16816(acc[m][n], xf[m][0].x, xf[m][1].x, xf[m][0].y, xf[m][1].y, wf[n].x,
                       wf[n].y);
        mma_bf16_16816(acc[m][n], xf[m][0].z, xf[m][1].z, xf[m][0].w, xf[m][1].w, wf[n].z,
                       wf[n].w);
      }
  }
  constexpr int cols = 8 * NT;
  float* mine = sums + warp * (16 * MT * cols);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mine[(16 * m + g + 8 * (e >> 1)) * cols + 8 * n + 2 * c + (e & 1)] = acc[m][n][e];
  __syncthreads();
  float* part_out = a.part + (static_cast<int64_t>(blockIdx.y) * a.M + row0) * a.R + r0;
  for (int i = threadIdx.x; i < rows * cols; i += kThreads) {
    const int r = i % cols;
    if (r0 + r >= a.R) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums[w * (16 * MT * cols) + i];
    part_out[static_cast<int64_t>(i / cols) * a.R + r] = v;
  }
}

// out = y + t B: a warp takes 16 rows and 32 columns at a time.  LARGE: the block's warps take
// different rows and the same columns (B then comes from L1 for 7 of the 8); else the same 16 rows
// and different columns.  KS: 32-wide steps of the rank.
// The column order inside the 32 is permuted so that a thread's four n8 tiles hold 8 consecutive
// columns: y and out move in 16-byte pieces.
template <bool LARGE, int KS>
__global__ void __launch_bounds__(kThreads) expand_kernel(const Args a, int cols_per_block) {
  const int bm = LARGE ? kLargeRows : kSmallRows;
  const Tile tile = find_tile(a, blockIdx.x, bm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int skip = LARGE ? 16 * warp : 0;
  const int rows = min(tile.rows - skip, 16);
  if (rows <= 0) return;
  const int64_t row0 = tile.row0 + skip;
  const int n_end = min(a.N, (static_cast<int>(blockIdx.y) + 1) * cols_per_block);
  const int n_begin = blockIdx.y * cols_per_block + (LARGE ? 0 : 32 * warp);
  constexpr int n_step = LARGE ? 32 : 32 * kWarps;
  const bool turned = tile.adapter >= 0;
  if (!turned && a.out == a.y) return;

  uint32_t hi[KS][2][4], lo[KS][2][4];  // [step][row half][pairs of k]
#pragma unroll
  for (int s = 0; s < KS; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t[8] = {};
      const int k = 32 * s + 8 * c;
      if (turned && k < a.R && g + 8 * h < rows) {
        const float* p = a.part + (row0 + g + 8 * h) * a.R + k;
        for (int i = 0; i < a.slices; ++i, p += a.M * a.R) {
          const float4 u = *reinterpret_cast<const float4*>(p);
          const float4 v = *reinterpret_cast<const float4*>(p + 4);
          t[0] += u.x, t[1] += u.y, t[2] += u.z, t[3] += u.w;
          t[4] += v.x, t[5] += v.y, t[6] += v.z, t[7] += v.w;
        }
        const float sc = a.scale ? a.scale[tile.adapter] : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= sc;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 top = __floats2bfloat162_rn(t[2 * e], t[2 * e + 1]);
        const float u = __low2float(top), v = __high2float(top);
        // an infinite t stays infinite: its remainder is 0, not inf - inf
        const __nv_bfloat162 rest =
            __floats2bfloat162_rn(isinf(u) ? 0.f : t[2 * e] - u, isinf(v) ? 0.f : t[2 * e + 1] - v);
        hi[s][h][e] = *reinterpret_cast<const uint32_t*>(&top);
        lo[s][h][e] = *reinterpret_cast<const uint32_t*>(&rest);
      }
    }

  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int n0 = n_begin; n0 < n_end; n0 += n_step) {
    float acc[4][4] = {};
    const bool in = n0 + 8 * c < a.N;  // N is a multiple of 16, a warp's columns are 32
    uint4 yv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      yv[h] = in && g + 8 * h < rows
                  ? *reinterpret_cast<const uint4*>(a.y + (row0 + g + 8 * h) * a.N + n0 + 8 * c)
                  : zero;
    if (turned) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = 32 * s + 8 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
          const uint4 w =
              k < a.R && n < a.N
                  ? ldg16(a.b + (static_cast<int64_t>(tile.adapter) * a.N + n) * a.R + k)
                  : zero;
          mma_bf16_16816(acc[j], hi[s][0][0], hi[s][1][0], hi[s][0][1], hi[s][1][1], w.x, w.y);
          mma_bf16_16816(acc[j], lo[s][0][0], lo[s][1][0], lo[s][0][1], lo[s][1][1], w.x, w.y);
          mma_bf16_16816(acc[j], hi[s][0][2], hi[s][1][2], hi[s][0][3], hi[s][1][3], w.z, w.w);
          mma_bf16_16816(acc[j], lo[s][0][2], lo[s][1][2], lo[s][0][3], lo[s][1][3], w.z, w.w);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!in || g + 8 * h >= rows) continue;
      const uint32_t yw[4] = {yv[h].x, yv[h].y, yv[h].z, yv[h].w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = __uint_as_float(yw[j] << 16), v = __uint_as_float(yw[j] & 0xFFFF0000u);
        const __nv_bfloat162 r = __floats2bfloat162_rn(u + acc[j][2 * h], v + acc[j][2 * h + 1]);
        o[j] = turned ? *reinterpret_cast<const uint32_t*>(&r) : yw[j];
      }
      *reinterpret_cast<uint4*>(a.out + (row0 + g + 8 * h) * a.N + n0 + 8 * c) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int NT>
cudaError_t launch_shrink(const Args& a, const Plan& p, cudaStream_t stream) {
  const int groups = (a.R + kGroup - 1) / kGroup;
  const int MT = p.large ? 2 : 1, bm = p.large ? kLargeRows : kSmallRows;
  const dim3 grid(static_cast<unsigned>(p.tiles * (bm / (16 * MT))), a.slices, groups);
  const int smem = kWarps * 16 * MT * 8 * NT * static_cast<int>(sizeof(float));
  auto kern = p.large ? shrink_kernel<2, NT> : shrink_kernel<1, NT>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, kThreads, smem, stream>>>(a, bm);
  return cudaGetLastError();
}

template <int KS>
cudaError_t launch_expand(const Args& a, const Plan& p, cudaStream_t stream) {
  const int cols = p.large ? 512 : 256;
  const dim3 grid(static_cast<unsigned>(p.tiles), (a.N + cols - 1) / cols);
  if (p.large)
    expand_kernel<true, KS><<<grid, kThreads, 0, stream>>>(a, cols);
  else
    expand_kernel<false, KS><<<grid, kThreads, 0, stream>>>(a, cols);
  return cudaGetLastError();
}

inline cudaError_t launch(const Args& a, const Plan& p, cudaStream_t stream) {
  cudaError_t e;
  if (a.R <= 8)
    e = launch_shrink<1>(a, p, stream);
  else if (a.R <= 16)
    e = launch_shrink<2>(a, p, stream);
  else if (a.R <= 32)
    e = launch_shrink<4>(a, p, stream);
  else
    e = launch_shrink<8>(a, p, stream);
  if (e != cudaSuccess) return e;
  switch ((a.R + 31) / 32) {
    case 1: return launch_expand<1>(a, p, stream);
    case 2: return launch_expand<2>(a, p, stream);
    case 3: return launch_expand<3>(a, p, stream);
    default: return launch_expand<4>(a, p, stream);
  }
}

}  // namespace lora
}  // namespace qs
