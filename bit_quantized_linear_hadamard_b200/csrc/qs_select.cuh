// Which key blocks each block of queries attends to, by a cheap score.
//
//   mean(x, j)  = the mean of the valid rows of block j (QS_BLOCK_K keys, QS_BLOCK_Q queries),
//                 rounded once to binary32 from a binary64 sum
//   score(i, j) = <mean(q, i), mean(k, j)> in binary64
//   blocks(i)   = the T visible key blocks of the highest score, the lowest index first among
//                 equals, listed in ascending order; -1 behind the last
//
// The answer is whole numbers, so a score that is off in its last place can change it: over the
// 10^7 scores of a video layer binary32 sums meet a near tie at the border of some list, binary64
// ones do not.  Sums of bf16 or fp16 values are exact in binary64 for all practical ranges, the
// products of two binary32 means are exact, and 128 of them are summed.
//
// Bound by HBM: queries and keys are read once; the scores stay in shared memory.  The query means
// have a kernel of their own (62 us for the 335 MB of a video's queries; formed by the blocks that
// go on to the scores, whose registers leave room for few warps, 150), but for few of them: there
// a launch costs more.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qs.h"
#include "qs_ops.cuh"

namespace qs {
namespace select {

using ops::checked_len;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;                 // query blocks of a CTA (the M of the binary64 mma)
constexpr int kMaxBlocks = 24576;        // key blocks: one row of scores fits shared memory
constexpr int kMaxSmem = 220 * 1024;

struct Strides {
  int64_t batch, row, head;  // in elements
};

struct MeanArgs {
  const uint16_t* x;
  Strides st;
  const int32_t* len;  // [B] or NULL
  float* means;        // [B, H, blocks, D]
  int64_t L;
  int B, H, blocks, first;
  int size;            // rows of a block
};

struct SelectArgs {
  const uint16_t* q;
  Strides st;
  const float* means;  // [B, Hkv, nk, D]
  const int32_t *q_len, *k_len;
  int32_t* blocks;     // [B, Hq, nq, T]
  int64_t Lq, Lk;
  int B, Hq, Hkv, nq, nk, T;
  int first, last;     // blocks always kept at the two ends of the visible ones
  int causal;
  int rows;            // query blocks per CTA, <= kRows
  const float* q_means; // [B, Hq, nq, D], or NULL: the CTAs form them
};

template <bool F16>
__device__ __forceinline__ double2 unpack(uint32_t w) {
  float u, v;
  if (F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    u = f.x, v = f.y;
  } else {
    u = __uint_as_float(w << 16), v = __uint_as_float(w & 0xFFFF0000u);
  }
  return make_double2(u, v);
}

// A warp's sum of `rows` rows of D elements: D / 8 lanes take 16 bytes of a row each, the warp
// 256 / D rows at a time.  Every lane ends with the sums of its 8 columns.
template <int D, bool F16>
__device__ __forceinline__ void warp_row_sum(const uint16_t* x, int64_t row_stride, int rows,
                                             double (&sum)[8]) {
  constexpr int kLanes = D / 8, kAt = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane / kLanes;
  const uint16_t* p = x + (lane % kLanes) * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0;
#pragma unroll 8
  for (int r = sub; r < rows; r += kAt) {
    const uint4 d = __ldg(reinterpret_cast<const uint4*>(p + r * row_stride));
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double2 v = unpack<F16>(w[e]);
      sum[2 * e] += v.x;
      sum[2 * e + 1] += v.y;
    }
  }
#pragma unroll
  for (int off = kLanes; off < 32; off <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], off);
}

// A warp forms one mean: heads vary fastest, so that neighbouring warps read neighbouring bytes
// of the same rows.
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) means_kernel(const MeanArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int count = a.blocks - a.first;
  if (i >= static_cast<int64_t>(a.B) * count * a.H) return;
  const int h = static_cast<int>(i % a.H), j = static_cast<int>(i / a.H % count) + a.first;
  const int b = static_cast<int>(i / a.H / count);
  const int64_t len = checked_len(a.len, b, a.L), row0 = static_cast<int64_t>(j) * a.size;
  const int rows = static_cast<int>(max(int64_t{0}, min(len - row0, static_cast<int64_t>(a.size))));
  double sum[8];
  warp_row_sum<D, F16>(a.x + b * a.st.batch + h * a.st.head + row0 * a.st.row, a.st.row, rows, sum);
  const int lane = threadIdx.x & 31;
  if (lane >= D / 8) return;
  const double n = rows > 0 ? rows : 1;
  float* out = a.means + ((static_cast<int64_t>(b) * a.H + h) * a.blocks + j) * D + lane * 8;
#pragma unroll
  for (int e = 0; e < 8; ++e) out[e] = static_cast<float>(sum[e] / n);
}

// D[8x8] += A[8x4] B[4x8] in binary64.
__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(d[0]), "+d"(d[1])
               : "d"(a), "d"(b));
}

// Scores as whole numbers of the same order; NaN is below all others.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return 0ull;
  if (s == 0.0) s = 0.0;  // -0 and 0 are equal
  const long long v = __double_as_longlong(s);
  const unsigned long long u = static_cast<unsigned long long>(v);
  return v < 0 ? ~u : u | 0x8000000000000000ull;
}

// OWN: the query means are formed here, in blocks of more threads: with few query blocks it is the
// way of one of them that counts.
template <bool OWN>
constexpr int kSelectThreads = OWN ? 512 : kThreads;

template <int D, bool F16, bool OWN>
__global__ void __launch_bounds__(kSelectThreads<OWN>, OWN ? 1 : 3)
    select_kernel(const SelectArgs a) {
  constexpr int kThreads = kSelectThreads<OWN>, kWarps = kThreads / 32;
  extern __shared__ __align__(16) double qm[];  // query means [8][D], behind them the keys [rows][nk]
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(qm + kRows * D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int i0 = blockIdx.x * a.rows;
  const int64_t ql = checked_len(a.q_len, b, a.Lq), kl = checked_len(a.k_len, b, a.Lk);

  // query means, rounded to binary32 as the keys' are
  if (OWN) {
    for (int r = warp; r < kRows; r += kWarps) {
      const int64_t row0 = static_cast<int64_t>(i0 + r) * QS_BLOCK_Q;
      const int rows =
          r < a.rows ? static_cast<int>(max(int64_t{0}, min(ql - row0, int64_t{QS_BLOCK_Q}))) : 0;
      double sum[8];
      warp_row_sum<D, F16>(a.q + b * a.st.batch + h * a.st.head + row0 * a.st.row, a.st.row, rows,
                           sum);
      const double n = rows > 0 ? rows : 1;
      if (lane < D / 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) qm[r * D + lane * 8 + e] = static_cast<float>(sum[e] / n);
    }
  } else {
    const float* src = a.q_means + ((static_cast<int64_t>(b) * a.Hq + h) * a.nq + i0) * D;
    const int have = min(a.rows, a.nq - i0) * D;
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) qm[i] = i < have ? src[i] : 0.f;
  }
  __syncthreads();

  // scores: a warp takes 8 key blocks; a thread's four columns of a 16-wide slice serve as k of
  // four m8n8k4 steps (the order of k is free as long as both operands share it), each with sums
  // of its own: 32 steps on one would wait for each other
  const int g = lane >> 2, c = lane & 3;
  const float* km = a.means +
                    (static_cast<int64_t>(b) * a.Hkv + h / (a.Hq / a.Hkv)) * a.nk * D;
  const double2* aq = reinterpret_cast<const double2*>(qm + g * D + 4 * c);
  for (int j0 = 8 * warp; j0 < a.nk; j0 += 8 * kWarps) {
    const int j = min(j0 + g, a.nk - 1);
    double d4[4][2] = {};
#pragma unroll
    for (int s0 = 0; s0 < D / 16; s0 += 4) {
      float4 f[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        f[s] = __ldg(reinterpret_cast<const float4*>(km + static_cast<int64_t>(j) * D +
                                                     16 * (s0 + s) + 4 * c));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const double2 q01 = aq[8 * (s0 + s)], q23 = aq[8 * (s0 + s) + 1];
        mma_f64(d4[0], q01.x, f[s].x);
        mma_f64(d4[1], q01.y, f[s].y);
        mma_f64(d4[2], q23.x, f[s].z);
        mma_f64(d4[3], q23.y, f[s].w);
      }
    }
    const double d[2] = {(d4[0][0] + d4[1][0]) + (d4[2][0] + d4[3][0]),
                         (d4[0][1] + d4[1][1]) + (d4[2][1] + d4[3][1])};
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (g < a.rows && j0 + 2 * c + e < a.nk)
        keys[static_cast<int64_t>(g) * a.nk + j0 + 2 * c + e] = score_key(d[e]);
  }
  __syncthreads();

  // the T highest of each row's visible blocks: the largest threshold that T keys reach, found
  // from its top bits down, ended as soon as exactly T reach it
  if (warp >= a.rows || i0 + warp >= a.nq) return;
  const int i = i0 + warp;
  const int64_t row0 = static_cast<int64_t>(i) * QS_BLOCK_Q;
  const int64_t end = min(row0 + QS_BLOCK_Q, ql);
  const int64_t seen = row0 >= ql ? 0 : max(int64_t{0}, min(a.causal ? end + kl - ql : kl, kl));
  const int n = static_cast<int>((seen + QS_BLOCK_K - 1) / QS_BLOCK_K);
  unsigned long long* key = keys + static_cast<int64_t>(warp) * a.nk;
  for (int j = lane; j < n; j += 32)
    if (j < a.first || j >= n - a.last) key[j] = ~0ull;
  __syncwarp();
  unsigned long long least = 0ull;
  int ties = -1;  // blocks with exactly `least` that are taken; -1: all
  if (n > a.T) {
    int above = 0;  // keys above `least` at the end
    bool exact = false;
    for (int bit = 62; bit >= 0 && !exact; bit -= 2) {  // two bits at a time
      int count[3] = {0, 0, 0};  // of the three numbers that the two bits may become besides 0
      for (int j = lane; j < n; j += 32) {
        const unsigned long long v = key[j];
#pragma unroll
        for (unsigned long long c = 0; c < 3; ++c) count[c] += v >= (least | ((c + 1) << bit));
      }
#pragma unroll
      for (int c = 0; c < 3; ++c) count[c] = __reduce_add_sync(0xffffffffu, count[c]);
      const unsigned long long most = count[2] >= a.T ? 3 : count[1] >= a.T ? 2 : count[0] >= a.T ? 1 : 0;
      if (most < 3) above = count[most];
      exact = most > 0 && count[most - 1] == a.T;
      least |= most << bit;
    }
    if (!exact) ties = a.T - above;
  }
  int32_t* out = a.blocks + ((static_cast<int64_t>(b) * a.Hq + h) * a.nq + i) * a.T;
  int filled = 0, tied = 0;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    const unsigned long long v = j < n ? key[j] : 0ull;
    const bool equal = j < n && ties >= 0 && v == least;
    const unsigned eq = __ballot_sync(0xffffffffu, equal);
    const unsigned before = (1u << lane) - 1u;
    const bool take = j < n && v >= least && (!equal || tied + __popc(eq & before) < ties);
    const unsigned got = __ballot_sync(0xffffffffu, take);
    if (take) out[filled + __popc(got & before)] = j;
    filled += __popc(got);
    tied += __popc(eq);
  }
  for (int j = filled + lane; j < a.T; j += 32) out[j] = -1;
}

template <int D, bool F16>
cudaError_t launch_means(const MeanArgs& a, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.B) * (a.blocks - a.first) * a.H;
  means_kernel<D, F16>
      <<<static_cast<unsigned>((n + kWarps - 1) / kWarps), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Query means formed on the way: up to this many query blocks in all.  Formed on the way / apart,
// us, D 128: 32.5 / 43.2 at 256 blocks, 36.5 / 43.3 at 1024, 74.3 / 68.1 at 2048.
constexpr int64_t kOwnMeans = 1024;

template <int D, bool F16>
cudaError_t launch_select(SelectArgs a, float* workspace, cudaStream_t stream) {
  a.rows = kRows;
  const auto smem = [&] {
    return static_cast<int64_t>(a.rows) * a.nk * 8 + kRows * D * static_cast<int>(sizeof(double));
  };
  while (a.rows > 1 && (smem() > kMaxSmem || a.rows / 2 >= a.nq)) a.rows /= 2;
  const bool own = workspace == nullptr;
  if (!own) {
    MeanArgs m{a.q, a.st, a.q_len, workspace, a.Lq, a.B, a.Hq, a.nq, 0, QS_BLOCK_Q};
    const cudaError_t e = launch_means<D, F16>(m, stream);
    if (e != cudaSuccess) return e;
    a.q_means = workspace;
  }
  auto kern = own ? select_kernel<D, F16, true> : select_kernel<D, F16, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.nq + a.rows - 1) / a.rows, a.Hq, a.B);
  kern<<<grid, own ? kSelectThreads<true> : kSelectThreads<false>, static_cast<size_t>(smem()),
         stream>>>(a);
  return cudaGetLastError();
}

}  // namespace select
}  // namespace qs
