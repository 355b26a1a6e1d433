// Rotary positions on the heads of a projection's output.
//
// Pair p of a head at row r turns by the angle a = pos[r][axis[p]] * inv_freq[p]:
//   (u, v) -> s * (u cos a - v sin a, u sin a + v cos a)
// with the pairs interleaved, (x[2p], x[2p+1]), or in halves, (x[p], x[p+n]), over the first
// rot = 2n elements of each head; the elements behind them are copied.
//
// The angle is a binary64 product reduced by 2*pi in binary64: a far position times a high
// frequency has lost the digits that matter in binary32 (at position 10^6 the angle's last place
// is 0.06).  The reduced angle goes through the binary32 sine and cosine with a first-order
// correction for the part of it that binary32 drops, so the factors are good to about 1e-7.
// The products are binary32 and rounded once to the output's type.
//
// Bound by HBM: every element is read once and written once.  A block takes as many rows as give
// one (row, pair) to each of its 256 threads, evaluates each row's factors once into shared
// memory (they serve all heads of the row), then streams the heads with 16-byte accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qs.h"
#include "qs_ptx.cuh"

namespace qs {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxDim = 1024;

struct Args {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;  // strides in elements
  int64_t rows;
  int heads, dim, pairs;
  int axes;
  const int64_t* pos;       // [rows, axes]
  const int32_t* axis;      // [pairs], or NULL: axis 0
  const double* inv_freq;   // [pairs]
  double scale;             // of both factors
  int inverse;
  int rows_per_block, heads_per_block;
  int copy_tail;            // elements behind the pairs are copied (0: y is x)
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32(__half v) {
  return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32(float v) {
  return __float2half_rn(v);
}

// cos and sin of pos * inv_freq times scale.
__device__ __forceinline__ float2 factors(int64_t pos, double inv_freq, double scale,
                                          bool inverse) {
  const double a = static_cast<double>(pos) * inv_freq;
  // a - 2 pi n in two steps: 2 pi as the sum of two binary64 numbers (the second is the first
  // one's rounding error); the fused products are exact up to the result's rounding
  const double n = rint(a * 0.15915494309189533577);
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586477, a));
  const float f = static_cast<float>(r);
  const float d = static_cast<float>(r - static_cast<double>(f));
  float s, c;
  sincosf(f, &s, &c);
  const float c1 = fmaf(-s, d, c), s1 = fmaf(c, d, s);
  const float m = static_cast<float>(scale);
  return make_float2(c1 * m, inverse ? -s1 * m : s1 * m);
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// V elements per access; with V == 1 any stride and any alignment of the elements does.
// INTER: an item is V elements of a head (V/2 pairs; 2 elements for V == 1).  Halves: an item is
// V elements of the first half and their partners.  Items behind the pairs copy V elements.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args a) {
  extern __shared__ float2 table[];  // [rows_per_block][pairs]
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows_per_block;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(a.rows_per_block), a.rows - row0));
  for (int i = threadIdx.x; i < nrows * a.pairs; i += kThreads) {
    const int r = i / a.pairs, p = i - r * a.pairs;
    int ax = a.axis ? a.axis[p] : 0;
    if (ax < 0 || ax >= a.axes) {
      atomicOr(&g_error_word, kErrIndex);
      ax = 0;
    }
    table[i] = factors(a.pos[(row0 + r) * a.axes + ax], a.inv_freq[p], a.scale, a.inverse != 0);
  }
  __syncthreads();

  constexpr int W = INTER && V == 1 ? 2 : V;  // elements an interleaved item covers
  constexpr bool kPartner = !INTER || V == 1;  // a pair's second element comes with another access
  constexpr int kUnits = 4;                    // (row, head) units in flight per thread
  const int turn_items = INTER ? 2 * a.pairs / W : a.pairs / V;
  const int tail_items = a.copy_tail ? (a.dim - 2 * a.pairs) / V : 0;
  const int items = turn_items + tail_items;
  const int h0 = blockIdx.y * a.heads_per_block;
  const unsigned nheads = min(a.heads_per_block, a.heads - h0);
  // thread -> (item, first unit); more items than threads: several passes over the items
  const int lanes = items < kThreads ? kThreads / items : 1;
  const int item_step = items < kThreads ? items : kThreads;
  const int lane = threadIdx.x / item_step;
  if (lane >= lanes) return;
  using P = Vec<T, V>;
  const int other = INTER ? 1 : a.pairs;  // distance of a pair's second element
  const unsigned units = nrows * nheads;
  for (int it = threadIdx.x - lane * item_step; it < items; it += item_step) {
    const bool turn = it < turn_items;
    const int e0 = turn ? it * W : 2 * a.pairs + (it - turn_items) * V;
    const T* x = static_cast<const T*>(a.x) + row0 * a.x_row + h0 * a.x_head + e0;
    T* y = static_cast<T*>(a.y) + row0 * a.y_row + h0 * a.y_head + e0;
    for (unsigned u0 = lane; u0 < units; u0 += kUnits * lanes) {
      // all loads before the first store: x and y may be one, so the compiler keeps their order
      P u[kUnits], w[kUnits];
      unsigned r[kUnits], h[kUnits];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const unsigned i = u0 + k * lanes;
        if (i >= units) continue;
        r[k] = i / nheads, h[k] = i - r[k] * nheads;
        const T* p = x + r[k] * a.x_row + h[k] * a.x_head;
        u[k] = *reinterpret_cast<const P*>(p);
        if (kPartner && turn) w[k] = *reinterpret_cast<const P*>(p + other);
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (u0 + k * lanes >= units) continue;
        T* p = y + r[k] * a.y_row + h[k] * a.y_head;
        if (turn) {
          const float2* cs = table + r[k] * a.pairs + (INTER ? e0 / 2 : e0);
          if (kPartner) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float2 f = cs[j];
              const float m = to_f32(u[k].v[j]), n = to_f32(w[k].v[j]);
              u[k].v[j] = from_f32<T>(m * f.x - n * f.y);
              w[k].v[j] = from_f32<T>(m * f.y + n * f.x);
            }
            *reinterpret_cast<P*>(p + other) = w[k];
          } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
              const float2 f = cs[j];
              const float m = to_f32(u[k].v[2 * j]), n = to_f32(u[k].v[2 * j + 1]);
              u[k].v[2 * j] = from_f32<T>(m * f.x - n * f.y);
              u[k].v[2 * j + 1] = from_f32<T>(m * f.y + n * f.x);
            }
          }
        }
        *reinterpret_cast<P*>(p) = u[k];
      }
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_t(Args a, int sms, cudaStream_t stream) {
  a.rows_per_block = kThreads / a.pairs > 0 ? kThreads / a.pairs : 1;
  if (a.rows_per_block > 8) a.rows_per_block = 8;
  // few rows: one row per block, and the heads over several blocks
  if (a.rows < static_cast<int64_t>(sms) * a.rows_per_block) a.rows_per_block = 1;
  const int64_t gx = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  int split = gx < sms ? static_cast<int>(sms / gx) : 1;
  const int items = INTER ? (2 * a.pairs) / (V == 1 ? 2 : V) : a.pairs / V;
  const int lanes = items < kThreads ? kThreads / items : 1;
  int most = (a.heads + lanes - 1) / lanes;  // blocks that still have a head for every lane
  if (split > most) split = most;
  a.heads_per_block = (a.heads + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(gx), (a.heads + a.heads_per_block - 1) / a.heads_per_block);
  const size_t smem = sizeof(float2) * a.rows_per_block * a.pairs;
  rope_kernel<T, V, INTER><<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const Args& a, bool interleaved, int sms, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  const auto multiple = [](int64_t v) { return v % V == 0; };
  const bool wide = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 &&
                    (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0 && multiple(a.x_row) &&
                    multiple(a.x_head) && multiple(a.y_row) && multiple(a.y_head) &&
                    multiple(interleaved ? 2 * a.pairs : a.pairs) && multiple(a.dim);
  if (interleaved)
    return wide ? launch_t<T, V, true>(a, sms, stream) : launch_t<T, 1, true>(a, sms, stream);
  return wide ? launch_t<T, V, false>(a, sms, stream) : launch_t<T, 1, false>(a, sms, stream);
}

}  // namespace rope
}  // namespace qs
