// Attention of each block of 128 queries over its list of 64-key blocks:
//   out[i] = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * (<q_i, k_j> - m_i)),
//   lse[i] = scale * m_i + log(sum_j p_ij)
// over the keys j of the listed blocks that row i sees (below the key length; with `causal` not
// behind the row's own place).  A row that sees none gets 0 and -inf.
//
// Bound by the tensor cores and the exponentials together: a pair of a query row and a key costs
// 4 D multiply-adds' worth of tensor work and one exponential, and at D = 128 both take about the
// same time on an SM.  One CTA holds one query block; two CTAs share an SM, so that one's
// products run while the other takes exponentials.
//
// A CTA's tile is two list entries, 128 keys.  Warps 0-3 own one query row per thread (lane of
// the tensor memory): the row's maximum and sum need no exchange between threads.  Warp 4 loads
// K and V by TMA (one 128-key tile of each in shared memory; K of the next tile is fetched as
// soon as this tile's scores are formed, V as soon as its product is), warp 5 issues the MMAs:
//   S = Q K^T into tensor memory (binary32), P (bf16 or fp16) written over S by the row threads,
//   O += P V with P read from tensor memory and V as the MN-major operand.
// O stays in tensor memory.  The running maximum only moves when a row's scores exceed it by
// 2^8: until then the old one serves (P stays below 2^8, in range of both types), and most tiles
// need no pass over O.  P is rounded to the operands' type (the tensor cores take no other);
// the row's sum is of the unrounded values in binary32.
//
// Long lists with few query blocks (a single token) are cut into `splits` ranges that run on CTAs
// of their own and leave normalised binary32 parts with their lse; a second kernel joins them in
// order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qs.h"
#include "qs_host.cuh"
#include "qs_ptx.cuh"

namespace qs {
namespace attn {

constexpr int kBQ = QS_BLOCK_Q, kBK = QS_BLOCK_K, kTileK = 2 * kBK;
constexpr int kRowWarps = 4;
constexpr int kThreads = 32 * (kRowWarps + 2);
constexpr int kMaxList = 2048;  // list entries of one CTA
constexpr int kTmemCols = 256;  // S (128) and O (up to 128)
constexpr int kSms = 148;
constexpr float kLazy = 8.f;    // log2 of the factor a row may exceed its running maximum by

enum { kQFull, kKFull, kKEmpty, kVFull, kVEmpty, kSFull, kPFull, kOFull, kDrain, kNumBars };

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;               // 128-byte wide operand columns
  static constexpr int kHalf = 128 * 128;              // bytes of 128 rows of one of them
  static constexpr int kOp = kHalves * kHalf;
  static constexpr int kOffQ = 0, kOffK = kOp, kOffV = 2 * kOp, kOffList = 3 * kOp;
  static constexpr int kOffBar = kOffList + 4 * kMaxList;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  // two CTAs per SM and no more (each holds half of the tensor memory), whatever D
  static constexpr int kNeed = kOffMisc + 32 + 1024;
  static constexpr int kSmemBytes = kNeed > 100 * 1024 ? kNeed : 100 * 1024;
  static_assert(kSmemBytes <= 113 * 1024, "two CTAs per SM");
};

struct Args {
  void* out;
  int64_t o_batch, o_row, o_head;  // strides in elements
  float* lse;                      // [B, Hq, Lq] or NULL
  const int32_t* blocks;           // [B, Hq, nq, T]
  const int32_t *q_len, *k_len;    // [B] or NULL
  float* part;                     // splits > 1: [splits][B, Hq, Lq][D], then the parts' lse
  int64_t Lq, Lk;
  int B, Hq, Hkv, nq, T;
  int splits, chunk;               // list entries per split
  int causal;
  float scale;
  // 0 where all heads (batches) share one tensor: its coordinate stays 0
  int q_by_head, q_by_batch, k_by_head, k_by_batch, v_by_head, v_by_batch;
};

// Instruction descriptor: kind::f16, binary32 D, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool f16, bool b_mn) {
  return (1u << 4)                                 // D format: F32
         | ((f16 ? 0u : 1u) << 7)                  // A: F16 or BF16
         | ((f16 ? 0u : 1u) << 10)                 // B: the same
         | ((b_mn ? 1u : 0u) << 16)                // B: N contiguous
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A from tensor memory: row = lane, two consecutive k per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand with the 128-byte swizzle: rows of 64 N elements (128 bytes), one per k; the
// next 64 N elements `lead` bytes on, the next 8 k 1024 bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two binary32 numbers in one 64-bit register pair: one instruction for two operations.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A length given on the device, held to [0, most]; outside it the error word is raised.
__device__ __forceinline__ int checked_len(const int32_t* len, int b, int64_t most) {
  if (!len) return static_cast<int>(most);
  const int n = len[b];
  if (n < 0 || n > most) {
    atomicOr(&g_error_word, kErrIndex);
    return n < 0 ? 0 : static_cast<int>(most);
  }
  return n;
}

// A row's 128 scores.
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&s)[4][32]) {
  uint32_t r[4][32];
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(taddr + 32 * q, r[q]);
  tmem_wait_ld();
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 32; ++e) s[q][e] = __uint_as_float(r[q][e]);
}

// -inf for the keys of the two entries from the first that the row does not see.
__device__ __forceinline__ void mask_scores(float (&s)[4][32], int seen0, int seen1) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (32 * (q & 1) + e >= (q < 2 ? seen0 : seen1)) s[q][e] = -INFINITY;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 2)
    attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* sp = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  int* list = reinterpret_cast<int*>(sp + C::kOffList);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + C::kOffMisc + 4);
  int* list_len = reinterpret_cast<int*>(sp + C::kOffMisc + 8);
  const auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qb = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hq / a.Hkv);
  const int ql = checked_len(a.q_len, b, a.Lq), kl = checked_len(a.k_len, b, a.Lk);
  const int row0 = qb * kBQ;
  if (row0 >= ql) return;  // rows behind the sequence stay as they are
  const int off = kl - ql;  // causal: row i sees keys up to i + off
  const int rows = min(kBQ, ql - row0);
  const int seen = a.causal ? min(kl, row0 + rows + off) : kl;  // keys the last row sees

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) mbar_init(bar(i), i == kPFull ? 32 * kRowWarps : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4) {  // the list's entries that some row of the block sees
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int32_t* src = a.blocks + ((static_cast<int64_t>(b) * a.Hq + h) * a.nq + qb) * a.T;
    const int end = min(a.T, (split + 1) * a.chunk);
    const int64_t nk = (a.Lk + kBK - 1) / kBK;
    int n = 0;
    for (int i0 = split * a.chunk; i0 < end; i0 += 32) {
      const int j = i0 + lane < end ? src[i0 + lane] : -1;
      if (j < -1 || j >= nk) atomicOr(&g_error_word, kErrIndex);
      const bool take = j >= 0 && j < nk && j * kBK < seen;
      const unsigned got = __ballot_sync(0xffffffffu, take);
      if (take) list[n + __popc(got & ((1u << lane) - 1u))] = j;
      n += __popc(got);
    }
    if (lane == 0) *list_len = n;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n = *list_len, tiles = (n + 1) / 2;
  const uint32_t tS = tmem, tO = tmem + 128;

  if (warp == 4) {
    if (lane == 0 && tiles > 0) {
      mbar_arrive_expect_tx(bar(kQFull), C::kOp);
      for (int d = 0; d < C::kHalves; ++d)
        tma_load_4d(sbase + C::kOffQ + d * C::kHalf, &tmQ, 64 * d, row0, h * a.q_by_head,
                    b * a.q_by_batch, bar(kQFull));
      const int kh = hk * a.k_by_head, kb = b * a.k_by_batch;
      const int vh = hk * a.v_by_head, vb = b * a.v_by_batch;
      int k_loads = 0, v_loads = 0;
      for (int t = 0; t < tiles; ++t) {
        // a missing second entry is loaded from behind the last key: zeros
        const int r0 = list[2 * t] * kBK;
        const int r1 = 2 * t + 1 < n ? list[2 * t + 1] * kBK : static_cast<int>(a.Lk);
        if (!mbar_wait_bounded(bar(kKEmpty), (t & 1) ^ 1u, abort_flag, kErrWaitProducer)) break;
        mbar_arrive_expect_tx(bar(kKFull), C::kOp);
        for (int d = 0; d < C::kHalves; ++d) {
          const uint32_t dst = sbase + C::kOffK + d * C::kHalf;
          tma_load_4d(dst, &tmK, 64 * d, r0, kh, kb, bar(kKFull));
          tma_load_4d(dst + C::kHalf / 2, &tmK, 64 * d, r1, kh, kb, bar(kKFull));
        }
        ++k_loads;
        if (!mbar_wait_bounded(bar(kVEmpty), (t & 1) ^ 1u, abort_flag, kErrWaitProducer)) break;
        mbar_arrive_expect_tx(bar(kVFull), C::kOp);
        for (int d = 0; d < C::kHalves; ++d) {
          const uint32_t dst = sbase + C::kOffV + d * C::kHalf;
          tma_load_4d(dst, &tmV, 64 * d, r0, vh, vb, bar(kVFull));
          tma_load_4d(dst + C::kHalf / 2, &tmV, 64 * d, r1, vh, vb, bar(kVFull));
        }
        ++v_loads;
      }
      // no copy into this CTA's memory may outlive it
      mbar_wait_limit(bar(kQFull), 0, kWaitTimeoutNs, kErrWaitTma);
      if (k_loads) mbar_wait_limit(bar(kKFull), (k_loads - 1) & 1, kWaitTimeoutNs, kErrWaitTma);
      if (v_loads) mbar_wait_limit(bar(kVFull), (v_loads - 1) & 1, kWaitTimeoutNs, kErrWaitTma);
    }
  } else if (warp == 5) {
    if (lane == 0 && tiles > 0) {
      constexpr uint32_t idesc_s = idesc_f16(128, 128, F16, false);
      constexpr uint32_t idesc_o = idesc_f16(128, D, F16, true);
      if (mbar_wait_bounded(bar(kQFull), 0, abort_flag, kErrWaitTma)) {
        for (int t = 0; t < tiles; ++t) {
          const uint32_t ph = t & 1;
          if (!mbar_wait_bounded(bar(kKFull), ph, abort_flag, kErrWaitTma)) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t at = (s / 4) * C::kHalf + (s % 4) * 32;
            mma_ss(tS, smem_desc_sw128(sbase + C::kOffQ + at),
                   smem_desc_sw128(sbase + C::kOffK + at), idesc_s, s != 0);
          }
          mma_commit(bar(kSFull));
          mma_commit(bar(kKEmpty));
          if (!mbar_wait_bounded(bar(kVFull), ph, abort_flag, kErrWaitTma)) break;
          if (!mbar_wait_bounded(bar(kPFull), ph, abort_flag, kErrWaitMma)) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < kTileK / 16; ++s)
            mma_ts(tO, tS + 8 * s, smem_desc_mn(sbase + C::kOffV + s * 2048, C::kHalf), idesc_o,
                   t != 0 || s != 0);
          mma_commit(bar(kVEmpty));
          if (t + 1 == tiles) mma_commit(bar(kOFull));
        }
      }
      // the tensor memory is given back only when nothing writes it any more
      mma_commit(bar(kDrain));
      mbar_wait_limit(bar(kDrain), 0, kWaitTimeoutNs, kErrWaitMma);
    }
  } else {
    const int r = 32 * warp + lane, row = row0 + r;
    const uint32_t mine = static_cast<uint32_t>(32 * warp) << 16;  // the warp's lanes
    const int limit = a.causal ? min(kl, row + off + 1) : kl;      // keys this row sees
    const int full = a.causal ? min(kl, row0 + off + 1) : kl;      // keys every row sees
    const float scale2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      const uint32_t ph = t & 1;
      const int j0 = list[2 * t] * kBK;
      const int j1 = 2 * t + 1 < n ? list[2 * t + 1] * kBK : 0x40000000;
      const bool masked = j0 + kBK > full || j1 + kBK > full;
      ok = mbar_wait_bounded(bar(kSFull), ph, abort_flag, kErrWaitEpilogue);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      float s[4][32];
      load_scores(tS + mine, s);
      const int seen0 = limit - j0, seen1 = limit - j1;  // of each entry's keys
      if (masked) mask_scores(s, seen0, seen1);
      float top4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        top4[q] = fmaxf(s[q][0], s[q][1]);
#pragma unroll
        for (int e = 2; e < 32; e += 2) top4[q] = max3(top4[q], s[q][e], s[q][e + 1]);
      }
      const float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
      // moves the running maximum (and O and l with it) only when the row outgrows it
      const bool move = top > m && (m == -INFINITY || (top - m) * scale2 > kLazy);
      if (__any_sync(0xffffffffu, move)) {
        const float to = move ? top : m;
        const float f = m == -INFINITY ? 0.f : exp2_approx((m - to) * scale2);
        l *= f;
        if (t > 0) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + mine + 32 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_32(tO + mine + 32 * q, o);
          }
          // the scores are read again rather than held meanwhile
          load_scores(tS + mine, s);
          if (masked) mask_scores(s, seen0, seen1);
        }
        m = to;
      }
      const float shift = m == -INFINITY ? 0.f : -m * scale2;
      const uint64_t scale22 = pair(scale2, scale2), shift2 = pair(shift, shift);
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float u, v;
          unpair(fma2(pair(s[q][2 * e], s[q][2 * e + 1]), scale22, shift2), u, v);
          u = exp2_approx(u), v = exp2_approx(v);
          sum[e & 1] = add2(sum[e & 1], pair(u, v));
          p[e] = pack2<F16>(u, v);
        }
        tmem_st_16(tS + mine + 16 * q, p);
      }
      float l0, l1;
      unpair(add2(sum[0], sum[1]), l0, l1);
      l += l0 + l1;
      // rows of V behind the keys may hold anything, and 0 times a NaN is one: they become 0
      if (masked && (j0 + kBK > kl || (j1 < kl && j1 + kBK > kl))) {
        ok = mbar_wait_bounded(bar(kVFull), ph, abort_flag, kErrWaitTma);
        const int key = (r < kBK ? j0 : j1 - kBK) + r;  // this thread's row of the V tile
        if (ok && key >= kl)
          for (int d = 0; d < C::kHalves; ++d)
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(sp + C::kOffV + d * C::kHalf + r * 128 + 16 * e) =
                  make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(kPFull));
    }
    if (tiles > 0 && __all_sync(0xffffffffu, ok))
      ok = mbar_wait_bounded(bar(kOFull), 0, abort_flag, kErrWaitEpilogue);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const float lse = l > 0.f ? (m * scale2 + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
    const int64_t flat = (static_cast<int64_t>(b) * a.Hq + h) * a.Lq + row;
    const bool write = r < rows && ok;
    if (a.splits == 1 && write && a.lse) a.lse[flat] = lse;
    const int64_t parts = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
    if (a.splits > 1 && write) a.part[parts * D * a.splits + split * parts + flat] = lse;
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld_32x32b_x32(tO + mine + 32 * q, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e)
        o[e] = tiles > 0 && inv != 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
      if (write && a.splits > 1) {
        uint4* dst = reinterpret_cast<uint4*>(a.part + (split * parts + flat) * D + 32 * q);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      } else if (write) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + b * a.o_batch +
                                              row * a.o_row + h * a.o_head + 32 * q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack2<F16>(__uint_as_float(o[8 * e + 2 * k]),
                              __uint_as_float(o[8 * e + 2 * k + 1]));
          dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

// Joins the parts of each row, in the order of the splits: a warp takes a row.
template <int D, bool F16>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  const int64_t parts = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  const int64_t flat = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (flat >= parts) return;
  const int lane = threadIdx.x & 31;
  const int64_t row = flat % a.Lq;
  const int h = static_cast<int>(flat / a.Lq % a.Hq), b = static_cast<int>(flat / a.Lq / a.Hq);
  if (row >= checked_len(a.q_len, b, a.Lq)) return;
  const float* lses = a.part + parts * D * a.splits + flat;
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, lses[s * parts]);
  constexpr int V = D / 32;
  float o[V] = {}, total = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float z = lses[s * parts];
    const float w = z == -INFINITY ? 0.f : exp2_approx((z - top) * kLog2e);
    total += w;
    const float* src = a.part + (s * parts + flat) * D + V * lane;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] += w * src[e];
  }
  const float inv = total > 0.f ? 1.f / total : (total == total ? 0.f : total);
  uint16_t* dst = static_cast<uint16_t*>(a.out) + b * a.o_batch + row * a.o_row + h * a.o_head;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t*>(dst + V * lane + e) = pack2<F16>(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[flat] = total > 0.f ? top + logf(total) : (total == total ? -INFINITY : total);
}

struct Plan {
  int splits, chunk;
};

// Few query blocks: the lists are cut so that the CTAs fill the GPU's 2 per SM once, in pieces of
// at least two tiles; and in any case so that a piece fits a CTA's list.
inline Plan plan(int64_t B, int64_t Hq, int64_t Lq, int64_t T) {
  const int64_t ctas = B * Hq * ((Lq + kBQ - 1) / kBQ);
  int64_t splits = 2 * kSms / ctas;
  const int64_t most = (T + 3) / 4, least = (T + kMaxList - 1) / kMaxList;
  if (splits > most) splits = most;
  if (splits < least) splits = least;
  if (splits < 1) splits = 1;
  int64_t chunk = (T + splits - 1) / splits;
  chunk += chunk & 1;  // whole tiles
  splits = (T + chunk - 1) / chunk;
  return {static_cast<int>(splits), static_cast<int>(chunk)};
}

// [B][H][L][D] view of 16-bit elements with strides in elements, as boxes of 64 columns.  A
// dimension of size 1 or stride 0 becomes one of size 1 (its stride is then any legal one).
inline bool make_map(CUtensorMap* map, const void* base, int64_t D, int64_t L, int64_t H,
                     int64_t B, int64_t row, int64_t head, int64_t batch, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  if (L == 1) row = D;
  if (H == 1 || head == 0) H = 1, head = D;
  if (B == 1 || batch == 0) B = 1, batch = D;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(L),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row) * 2,
                                 static_cast<cuuint64_t>(head) * 2,
                                 static_cast<cuuint64_t>(batch) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box,
             ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F16>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   const Args& a, cudaStream_t stream) {
  auto kern = attn_kernel<D, F16>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.nq) * a.splits, a.Hq, a.B);
  kern<<<grid, kThreads, Cfg<D>::kSmemBytes, stream>>>(q, k, v, a);
  const cudaError_t l = cudaGetLastError();
  if (l != cudaSuccess || a.splits == 1) return l;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  join_kernel<D, F16><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace qs
