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

// A thread's way through the (row, head) units of a block: from unit `lane` in steps of `lanes`,
// with the offsets of x and y carried along (a division and two 64-bit products per unit made the
// kernel bound by its instructions: 333 us for 1.34 GB).
struct Walk {
  int64_t x, y;          // offsets of this unit
  int64_t dx, dy;        // of a step
  int64_t wx, wy;        // correction where a step passes the last head
  unsigned row, head, d_row, d_head, heads;
  __device__ Walk(const Args& a, unsigned lane, unsigned lanes, unsigned nheads) : heads(nheads) {
    row = lane / nheads, head = lane - row * nheads;
    d_row = lanes / nheads, d_head = lanes - d_row * nheads;
    x = row * a.x_row + head * a.x_head, y = row * a.y_row + head * a.y_head;
    dx = d_row * a.x_row + d_head * a.x_head, dy = d_row * a.y_row + d_head * a.y_head;
    wx = a.x_row - nheads * a.x_head, wy = a.y_row - nheads * a.y_head;
  }
  __device__ __forceinline__ void step() {
    row += d_row, head += d_head, x += dx, y += dy;
    if (head >= heads) head -= heads, ++row, x += wx, y += wy;
  }
};

// V elements per access; with V == 1 any stride and any alignment of the elements does.
// INTER: an item is V elements of a head (V/2 pairs; 2 elements for V == 1).  Halves: an item is
// V elements of the first half and their partners.  The elements behind the pairs are copied in a
// second pass, V at a time.
// One unit per thread and many blocks: two or four units with all their loads first were slower
// (1.34 GB, interleaved: 254 us against 302 and 376), the memory being read and written in more
// places at once.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads, !INTER || V == 1 ? 4 : 8) rope_kernel(const Args a) {
  extern __shared__ __align__(16) float2 table[];  // [rows_per_block][pairs]
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

  constexpr int W = INTER && V == 1 ? 2 : V;   // elements an interleaved item covers
  constexpr bool kPartner = !INTER || V == 1;  // a pair's second element comes with another access
  const int h0 = blockIdx.y * a.heads_per_block;
  const unsigned nheads = min(a.heads_per_block, a.heads - h0);
  const unsigned units = nrows * nheads;
  const T* x0 = static_cast<const T*>(a.x) + row0 * a.x_row + h0 * a.x_head;
  T* y0 = static_cast<T*>(a.y) + row0 * a.y_row + h0 * a.y_head;
  using P = Vec<T, V>;
  // thread -> (item, first unit); more items than threads: several passes over the items
  const auto each = [&](int items, auto&& body) {
    const int step = items < kThreads ? items : kThreads;
    const unsigned lanes = kThreads / step, lane = threadIdx.x / step;
    if (lane >= lanes) return;
    for (int it = threadIdx.x - lane * step; it < items; it += step) {
      Walk at(a, lane, lanes, nheads);
      for (unsigned u = lane; u < units; u += lanes, at.step()) body(it, at);
    }
  };

  each(INTER ? 2 * a.pairs / W : a.pairs / V, [&](int it, const Walk& at) {
    const T* x = x0 + it * W + at.x;
    T* y = y0 + it * W + at.y;
    const float2* f = table + at.row * a.pairs + (INTER ? it * W / 2 : it * W);
    const int other = INTER ? 1 : a.pairs;  // distance of a pair's second element
    P u = *reinterpret_cast<const P*>(x);
    if (kPartner) {
      P w = *reinterpret_cast<const P*>(x + other);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float m = to_f32(u.v[j]), n = to_f32(w.v[j]);
        u.v[j] = from_f32<T>(m * f[j].x - n * f[j].y);
        w.v[j] = from_f32<T>(m * f[j].y + n * f[j].x);
      }
      *reinterpret_cast<P*>(y + other) = w;
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float m = to_f32(u.v[2 * j]), n = to_f32(u.v[2 * j + 1]);
        u.v[2 * j] = from_f32<T>(m * f[j].x - n * f[j].y);
        u.v[2 * j + 1] = from_f32<T>(m * f[j].y + n * f[j].x);
      }
    }
    *reinterpret_cast<P*>(y) = u;
  });
  const int tail = a.copy_tail ? (a.dim - 2 * a.pairs) / V : 0;
  if (tail > 0)
    each(tail, [&](int it, const Walk& at) {
      const int e0 = 2 * a.pairs + it * V;
      *reinterpret_cast<P*>(y0 + at.y + e0) = *reinterpret_cast<const P*>(x0 + at.x + e0);
    });
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

template <typename T, int V>
bool accesses_fit(const Args& a, bool interleaved) {
  const auto multiple = [](int64_t v) { return v % V == 0; };
  const uintptr_t bytes = V * sizeof(T) - 1;
  return (reinterpret_cast<uintptr_t>(a.x) & bytes) == 0 &&
         (reinterpret_cast<uintptr_t>(a.y) & bytes) == 0 && multiple(a.x_row) &&
         multiple(a.x_head) && multiple(a.y_row) && multiple(a.y_head) &&
         multiple(interleaved ? 2 * a.pairs : a.pairs) && multiple(a.dim);
}

// The widest accesses that the views allow: 16 bytes, two elements, one.
template <typename T>
cudaError_t launch(const Args& a, bool interleaved, int sms, cudaStream_t stream) {
  constexpr int V = 16 / sizeof(T);
  if (accesses_fit<T, V>(a, interleaved))
    return interleaved ? launch_t<T, V, true>(a, sms, stream) : launch_t<T, V, false>(a, sms, stream);
  if (accesses_fit<T, 2>(a, interleaved))
    return interleaved ? launch_t<T, 2, true>(a, sms, stream) : launch_t<T, 2, false>(a, sms, stream);
  return interleaved ? launch_t<T, 1, true>(a, sms, stream) : launch_t<T, 1, false>(a, sms, stream);
}

}  // namespace rope
}  // namespace qs
