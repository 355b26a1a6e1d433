// Attention of each block of 128 queries over its list of 64-key blocks:
//   out[i] = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale * (<q_i, k_j> - m_i)),
//   lse[i] = scale * m_i + log(sum_j p_ij)
// over the keys j of the listed blocks that row i sees (below the key length; with `causal` not
// behind the row's own place).  A row that sees none gets 0 and -inf.
//
// Bound by the tensor cores and the exponentials together: a pair of a query row and a key costs
// 4 D operations on the tensor cores and one exponential, and at D = 128 both take about the same
// time on an SM.  So the row threads must never wait for a product, nor the products for them.
//
// One persistent CTA per SM works through the (batch, head, query block, split) items.  A tile is
// two of an item's listed blocks, 128 keys: an MMA of 64 columns takes as long as one of 128
// (measured 70 and 75 cycles at K = 16), so blocks go in pairs.  Three groups of 128 threads own
// one query row per thread (lane of the tensor memory) and take the tiles in turn, each with a
// score buffer of its own; O fills the rest of the tensor memory:
//   S = Q K^T (binary32), P (bf16 or fp16) written over S by the row threads, O += P V.
// While one group takes its exponentials, the products of the other two run, and a group has the
// time of two tiles to get through its part.
//
// A row's running maximum goes from group to group in the order of the tiles, before the
// exponentials.  It only moves when the scores exceed it by 2^8: until then the old one serves (P
// stays below 2^8, in range of both types), and O, which all groups share, is hardly ever
// rescaled.  P is rounded to the operands' type (the tensor cores take no other); a row's sums,
// one per group, are of the unrounded values in binary32.
// Warps 0-11 the three groups; 12 and 14 read the lists and load Q and K, and V, by TMA; 13 and
// 15 issue the MMAs of S and of O.
//
// With few items (a single token) the lists are cut into `splits` ranges that are items of their
// own and leave normalised binary32 parts with their lse; a second kernel joins them in order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "qs.h"
#include "qs_host.cuh"
#include "qs_launch.cuh"
#include "qs_ops.cuh"
#include "qs_ptx.cuh"

namespace qs {
namespace attn {

using ops::checked_len;
using ops::idesc_f16;
using ops::max3_nan;
using ops::mma_ss;

constexpr int kBQ = QS_BLOCK_Q, kBK = QS_BLOCK_K, kTileK = 2 * kBK;
constexpr int kGroups = 3, kGroupWarps = 4;
constexpr int kTmaWarp = kGroups * kGroupWarps, kMmaWarp = kTmaWarp + 1, kTmaVWarp = kMmaWarp + 1,
              kPvWarp = kTmaVWarp + 1;
constexpr int kThreads = 32 * 16;  // 128 registers each
constexpr int kSms = 148;
constexpr float kLazy = 8.f;  // log2 of the factor a row may exceed its running maximum by
constexpr int kTileRing = 8, kItemRing = 4;

// Tensor memory, columns of 32 bits: O, then the groups' score buffers.
constexpr int kTmemCols = 512, kColO = 0, kColS = 128;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;         // 128-byte wide operand columns
  static constexpr int kHalf = kTileK * 128;     // bytes of 128 rows in one of them
  static constexpr int kOp = kHalves * kHalf;
  static constexpr int kStages = 256 / D;        // of the K and V rings: 64 KB each
  static constexpr int kOffQ = 0, kOffK = 2 * kOp, kOffV = kOffK + kStages * kOp;
  static constexpr int kOffM = kOffV + kStages * kOp;              // running maxima, per group
  static constexpr int kOffMl = kOffM + kGroups * kBQ * 4;         // (m, l) per group, two items
  static constexpr int kOffTiles = kOffMl + 2 * kGroups * kBQ * 8; // first keys of a tile's blocks
  static constexpr int kOffItems = kOffTiles + 8 * kTileRing;      // announced items
  static constexpr int kOffBar = kOffItems + 32 * kItemRing;
  // barriers
  static constexpr int kKFull = 0, kKEmpty = kStages, kVFull = 2 * kStages, kVEmpty = 3 * kStages;
  static constexpr int kQFull = 4 * kStages, kQFree = kQFull + 2, kSFull = kQFree + 2;
  static constexpr int kPFull = kSFull + kGroups;      // per group and half of the tile
  static constexpr int kPvDone = kPFull + 2 * kGroups;
  static constexpr int kMReady = kPvDone + kGroups;    // per group and warp
  static constexpr int kMlFull = kMReady + kGroups * kGroupWarps;
  static constexpr int kOFree = kMlFull + 1;
  static constexpr int kItemFull = kOFree + 1, kItemEmpty = kItemFull + kItemRing;
  static constexpr int kDrain = kItemEmpty + kItemRing, kNumBars = kDrain + 2;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffMisc + 32 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  __device__ static int arrivals(int i) {
    const auto in = [&](int first, int n) { return i >= first && i < first + n; };
    if (in(kPFull, 2 * kGroups)) return kGroupWarps;
    if (in(kSFull, kGroups)) return 2;                            // formed, and its keys known
    if (i == kMlFull) return kGroups * kGroupWarps;
    if (i == kOFree) return kHalves * kGroupWarps;                // the writers' warps only
    if (in(kQFree, 2)) return 1 + kHalves;                        // scores formed, output staged
    if (in(kItemEmpty, kItemRing)) return kGroups * kGroupWarps + 2;
    return 1;
  }
};

struct View {
  const uint16_t* p;
  int64_t batch, row, head;  // strides in elements
};

struct Args {
  View q, k, v;  // as the tensor maps have them
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

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
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

// The scores of a row go through registers 32 at a time, in rolled loops: unrolled over the tile,
// the three groups' code did not stay in the instruction caches and waited for its fetches.

// -inf for the keys from `seen` on, which the row does not see.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], int seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e >= seen) s[e] = 0xff800000u;
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32], float top) {
  float t[2] = {top, top};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    t[0] = max3(t[0], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
    t[1] = max3(t[1], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
  }
  return max3(t[0], t[1], t[1]);
}

// P = exp2(scale2 * s + shift) of 32 scores into tensor memory; their sum is added to `sum`.
template <bool F16>
__device__ __forceinline__ void exp32(uint32_t taddr, const uint32_t (&s)[32], uint64_t scale2,
                                      uint64_t shift2, uint64_t (&sum)[2]) {
  uint32_t p[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float u, v;
    unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), scale2, shift2), u,
           v);
    u = exp2_approx(u), v = exp2_approx(v);
    sum[e & 1] = add2(sum[e & 1], pair(u, v));
    p[e] = pack2<F16>(u, v);
  }
  tmem_st_16(taddr, p);
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One item: a range of the list of one query block.  The warp that reads the lists announces it
// to the others through a ring in shared memory.
struct alignas(16) Item {
  int b, h, row0, split;
  int ql, kl;  // lengths
  int tiles;   // -1: no further item
  int pad_;
};

__device__ __forceinline__ Item item_at(const Args& a, unsigned i) {
  Item it;
  it.split = static_cast<int>(i % static_cast<unsigned>(a.splits));
  i /= static_cast<unsigned>(a.splits);
  it.row0 = static_cast<int>(i % static_cast<unsigned>(a.nq)) * kBQ;
  i /= static_cast<unsigned>(a.nq);
  it.h = static_cast<int>(i % static_cast<unsigned>(a.Hq));
  it.b = static_cast<int>(i / static_cast<unsigned>(a.Hq));
  it.ql = static_cast<int>(checked_len(a.q_len, it.b, a.Lq));
  it.kl = static_cast<int>(checked_len(a.k_len, it.b, a.Lk));
  it.tiles = 0;
  return it;
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Rows whose output has a NaN although their sum is finite, formed again from the keys that they see
// alone, in binary32: in the matrix products a key that a row does not see has P = 0, and 0 times an
// infinity or a NaN of that key's v is a NaN.  The block's four groups of 128 threads go through its
// items once more, a row and 64 columns to a thread.  Only blocks that met such a row come here.  In
// the loop over the items this code cost 2 to 9 %, here 1 to 3 % where items are short (causal, 2 x
// 4099 rows, 32 / 8 heads, D 128: 197.8 -> 200.4 us) and nothing where they are long.
template <int D, bool F16>
__device__ __noinline__ void rows_again(const Args& a, unsigned items) {
  const int half = threadIdx.x / kBQ, r = threadIdx.x % kBQ;
  if (half >= D / 64) return;
  const int64_t nk = (a.Lk + kBK - 1) / kBK, parts = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  const float scale2 = a.scale * kLog2e;
  float o[64];
  for (unsigned i = blockIdx.x; i < items; i += gridDim.x) {
    const Item it = item_at(a, i);
    const int row = it.row0 + r, off = it.kl - it.ql, limit = min(it.kl, row + off + 1);
    if (row >= it.ql || limit >= min(it.kl, it.row0 + kBQ + off)) continue;
    const int64_t flat = (static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Lq + row;
    float4* part = reinterpret_cast<float4*>(a.part + (it.split * parts + flat) * D + 64 * half);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + it.b * a.o_batch + row * a.o_row +
                                          it.h * a.o_head + 64 * half);
    bool nan = false;
    for (int k = 0; k < 16; ++k) {
      if (a.splits > 1) {
        const float4 v = part[k];
        nan |= isnan(v.x) || isnan(v.y) || isnan(v.z) || isnan(v.w);
      } else {
        const uint2 v = reinterpret_cast<const uint2*>(out)[k];
        const float2 x = unpack2<F16>(v.x), y = unpack2<F16>(v.y);
        nan |= isnan(x.x) || isnan(x.y) || isnan(y.x) || isnan(y.y);
      }
    }
    if (!nan) continue;
    const int hk = it.h / (a.Hq / a.Hkv);
    const uint4* q = reinterpret_cast<const uint4*>(a.q.p + it.b * a.q.batch + row * a.q.row + it.h * a.q.head);
    const int32_t* list = a.blocks + ((static_cast<int64_t>(it.b) * a.Hq + it.h) * a.nq + it.row0 / kBQ) * a.T +
                          static_cast<int64_t>(it.split) * a.chunk;
    const int len = min(a.chunk, a.T - it.split * a.chunk);
    float m = -INFINITY, l = 0.f;
    bool some = true;  // columns that are not NaN yet
    for (int e = 0; e < 64; ++e) o[e] = 0.f;
    for (int n = 0; n < 64 * len && some; ++n) {
      const int entry = list[n / 64], j = entry * kBK + n % 64;
      if (entry < 0 || entry >= nk || j >= limit) continue;
      const uint4* k = reinterpret_cast<const uint4*>(a.k.p + it.b * a.k.batch + j * a.k.row + hk * a.k.head);
      float s = 0.f;
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = q[c], y = k[c];
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 u = unpack2<F16>(xw[w]), t = unpack2<F16>(yw[w]);
          s = fmaf(u.x, t.x, fmaf(u.y, t.y, s));
        }
      }
      s *= scale2;
      if (s == -INFINITY) continue;  // p = 0
      if (s > m) {
        const float f = exp2f(m - s);
        for (int e = 0; e < 64; ++e) o[e] *= f;
        l *= f, m = s;
      }
      const float p = exp2f(s - m);
      l += p;
      const uint4* v =
          reinterpret_cast<const uint4*>(a.v.p + it.b * a.v.batch + j * a.v.row + hk * a.v.head + 64 * half);
      some = false;
      for (int c = 0; c < 8; ++c) {
        const uint4 y = v[c];
        const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
        for (int w = 0; w < 4; ++w) {
          const float2 t = unpack2<F16>(yw[w]);
          float &x0 = o[8 * c + 2 * w], &x1 = o[8 * c + 2 * w + 1];
          x0 = fmaf(p, t.x, x0), x1 = fmaf(p, t.y, x1);
          some |= !isnan(x0) || !isnan(x1);
        }
      }
    }
    if (!some || !(l > 0.f)) continue;  // NaN throughout: as it is
    const float inv = 1.f / l;
    for (int e = 0; e < 64; e += 4) {
      const float4 v = make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv, o[e + 3] * inv);
      if (a.splits > 1)
        part[e / 4] = v;
      else
        reinterpret_cast<uint2*>(out)[e / 4] = make_uint2(pack2<F16>(v.x, v.y), pack2<F16>(v.z, v.w));
    }
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                const __grid_constant__ Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  uint8_t* sp = smem_raw + pad;
  const uint32_t sbase = raw + pad;
  float* maxima = reinterpret_cast<float*>(sp + C::kOffM);  // [group][row]
  float2* ml = reinterpret_cast<float2*>(sp + C::kOffMl);   // [item parity][group][row]
  int2* tile_ring = reinterpret_cast<int2*>(sp + C::kOffTiles);
  Item* item_ring = reinterpret_cast<Item*>(sp + C::kOffItems);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sp + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sp + C::kOffMisc + 4);
  int* staged_warps = reinterpret_cast<int*>(sp + C::kOffMisc + 8);  // per 64 columns, modulo 4
  volatile int* rows_left = reinterpret_cast<volatile int*>(sp + C::kOffMisc + 16);  // for rows_again
  const auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned items = static_cast<unsigned>(a.B) * a.Hq * a.nq * a.splits;  // below 2^31

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(bar(i), C::arrivals(i));
    *abort_flag = 0;
    staged_warps[0] = staged_warps[1] = 0;
    *rows_left = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmO);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the kernel that joins the parts may come onto the GPU; it waits for this one's end
  if (a.splits > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // After a wait that gave up, a thread waits for nothing more and leaves its loops; no barrier
  // but the block's last one is unbounded.
  bool ok = true;
  const auto wait = [&](int i, uint32_t parity, unsigned err) {
    if (ok) ok = mbar_wait_bounded(bar(i), parity, abort_flag, err);
  };

  if (warp < kTmaWarp) {
    // ---- row groups.  A barrier of parity p is only ever waited on when its phase before the
    // awaited one is known to be complete: S of tile g is formed when P V of tile g - 3 is done (and
    // so V of tile g - 3 was there; of g - 2 it need not be).
    const int group = warp / kGroupWarps, quarter = warp % kGroupWarps;
    const int r = threadIdx.x % kBQ;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t tS = tmem + kColS + kTileK * group + lanes, tO = tmem + kColO + lanes;
    const float scale2 = a.scale * kLog2e;
    const uint64_t scale22 = pair(scale2, scale2);
    unsigned g0 = 0;      // tiles of the items so far
    unsigned q_items = 0; // items with tiles
    int staged = -1;      // Q buffer whose output store this thread has yet to see off
    const auto see_off = [&] {
      if (staged < 0) return;
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      mbar_arrive(bar(C::kQFree + staged));
      staged = -1;
    };
    for (unsigned e = 0;; ++e) {
      const int item_slot = e % kItemRing;
      wait(C::kItemFull + item_slot, (e / kItemRing) & 1, kErrWaitProducer);
      if (!__all_sync(0xffffffffu, ok)) break;
      const Item it = item_ring[item_slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kItemEmpty + item_slot));
      const int n = it.tiles;
      if (n < 0) break;
      const int row = it.row0 + r;
      const int off = it.kl - it.ql;  // causal: row i sees keys up to i + off
      const int limit = a.causal ? min(it.kl, row + off + 1) : it.kl;    // keys this row sees
      const int full = a.causal ? min(it.kl, it.row0 + off + 1) : it.kl; // keys every row sees
      // a warp without a valid row only keeps step: with one query token three of four are
      const bool idle = it.row0 + 32 * quarter >= it.ql;
      float m = -INFINITY, l = 0.f;
      // tiles of this group: those with (g0 + t) % 3 == group
      for (int t = (group + kGroups - static_cast<int>(g0 % kGroups)) % kGroups; t < n; t += kGroups) {
        const unsigned g = g0 + t;
        const uint32_t ph = (g / kGroups) & 1;
        // the running maximum from the tile before, there before this tile's scores as a rule
        const int from = (group + kGroups - 1) % kGroups;
        if (g > 0)
          wait(C::kMReady + from * kGroupWarps + quarter, ((g - 1) / kGroups) & 1, kErrWaitEpilogue);
        __syncwarp();
        const float old = t > 0 ? maxima[from * kBQ + r] : -INFINITY;
        wait(C::kSFull + group, ph, kErrWaitEpilogue);
        __syncwarp();
        const int2 tile = tile_ring[g % kTileRing];
        // rows of V behind the keys may hold anything, and 0 times a NaN is one: they become 0
        // (behind the tensor's end the copies have filled in zeros already)
        if (it.kl < a.Lk &&
            (tile.x + kBK > it.kl || (tile.y < it.kl && tile.y + kBK > it.kl))) {
          const int slot = static_cast<int>(g % C::kStages);
          // The stage may still wait for, or hold, the V of the tile that had it before, which S of
          // this tile says nothing about where there are fewer stages than groups.
          if (C::kStages < kGroups && g >= C::kStages)
            wait(C::kPvDone + (g - C::kStages) % kGroups, ((g - C::kStages) / kGroups) & 1,
                 kErrWaitEpilogue);
          wait(C::kVFull + slot, (g / C::kStages) & 1, kErrWaitTma);
          const int key = r < kBK ? tile.x + r : tile.y + r - kBK;  // this thread's row of V
          if (ok && key >= it.kl)
            for (int d = 0; d < C::kHalves; ++d)
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(sp + C::kOffV + slot * C::kOp + d * C::kHalf + r * 128 +
                                          16 * k) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          // a warp's arrival for the first block of P says that its rows are done
        }
        if (idle) {  // its rows of P and O stay what they are, and are not written out
          if (lane == 0) {
            mbar_arrive(bar(C::kMReady + group * kGroupWarps + quarter));
            mbar_arrive(bar(C::kPFull + 2 * group));
            mbar_arrive(bar(C::kPFull + 2 * group + 1));
          }
          continue;
        }
        tc_fence_after();
        const bool masked = tile.x + kBK > full || tile.y + kBK > full;
        // two sets of registers: the next 32 scores are on their way while these are looked at
        uint32_t sa[32], sb[32];
        float top = -INFINITY;
        tmem_ld_32x32b_x32(tS, sa);
        tmem_wait_ld();
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int seen = limit - (c == 0 ? tile.x : tile.y);
          tmem_ld_32x32b_x32(tS + kBK * c + 32, sb);
          if (masked) mask32(sa, seen);
          top = max32(sa, top);
          tmem_wait_ld();
          tmem_ld_32x32b_x32(tS + kBK * (c ^ 1), sa);  // at the end: the first ones again
          if (masked) mask32(sb, seen - 32);
          top = max32(sb, top);
          tmem_wait_ld();
        }
        // it moves only when the row outgrows it
        const bool move = top > old && (old == -INFINITY || (top - old) * scale2 > kLazy);
        const float now = move ? top : old;
        maxima[group * kBQ + r] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kMReady + group * kGroupWarps + quarter));
        if (t > 0 && __any_sync(0xffffffffu, move)) {
          wait(C::kPvDone + (g - 1) % kGroups, ((g - 1) / kGroups) & 1, kErrWaitEpilogue);
          __syncwarp();
          tc_fence_after();
          const float f = !move ? 1.f : old == -INFINITY ? 0.f : exp2_approx((old - now) * scale2);
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            tmem_ld_16(tO + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st_16(tO + 16 * q, o);
          }
        }
        if (m != now) {  // this group's sum moves with it; before any maximum it is 0, or NaN
          if (m != -INFINITY) l *= exp2_approx((m - now) * scale2);
          m = now;
        }
        // P of a block goes to the second product as soon as it is written
        const auto give_half = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kPFull + 2 * group + half));
        };
        const float shift = m == -INFINITY ? 0.f : -m * scale2;
        const uint64_t shift2 = pair(shift, shift);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int seen = limit - (c == 0 ? tile.x : tile.y);
          tmem_ld_32x32b_x32(tS + kBK * c + 32, sb);
          if (masked) mask32(sa, seen);
          exp32<F16>(tS + 32 * c, sa, scale22, shift2, sum);
          tmem_wait_ld();
          if (c == 0) tmem_ld_32x32b_x32(tS + kBK, sa);
          if (masked) mask32(sb, seen - 32);
          exp32<F16>(tS + 32 * c + 16, sb, scale22, shift2, sum);
          tmem_wait_ld();
          give_half(c);
        }
        float l0, l1;
        unpair(add2(sum[0], sum[1]), l0, l1);
        l += l0 + l1;
        see_off();
      }
      g0 += n;
      see_off();  // the item after this one needs that buffer, wherever this thread then waits
      // the item's end: the groups' sums meet.  The group of the last tile and the one before it
      // write out 64 columns of O each (one of them, for D = 64); the third, whose tile is next,
      // goes on.  The sums' slots alternate: all groups have read the item before the last when
      // the last one's sums are complete.
      if (e > 0) wait(C::kMlFull, (e - 1) & 1, kErrWaitEpilogue);
      ml[((e & 1) * kGroups + group) * kBQ + r] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kMlFull));
      const int last = static_cast<int>((g0 + kGroups - 1) % kGroups);  // any, for n == 0
      const int half = (last + kGroups - group) % kGroups;
      const int qb = q_items & 1;
      q_items += n > 0;
      if (half < C::kHalves) {
        wait(C::kMlFull, e & 1, kErrWaitEpilogue);
        if (n > 0) wait(C::kPvDone + last, ((g0 - 1) / kGroups) & 1, kErrWaitEpilogue);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        // O into registers first: the next item's products wait for its place.  Only the writers
        // give it back: a group that does not read O may be an item ahead, and its arrival would
        // then stand for one that is still to come
        uint32_t o[2][32];
        tmem_ld_32x32b_x32(tO + 64 * half, o[0]);
        tmem_ld_32x32b_x32(tO + 64 * half + 32, o[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (n > 0 && lane == 0) mbar_arrive(bar(C::kOFree));
        float mm = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) mm = fmaxf(mm, ml[((e & 1) * kGroups + k) * kBQ + r].x);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          // in the order of the item's tiles, so that it does not matter where a CTA meets it
          const float2 v = ml[((e & 1) * kGroups + (g0 - n + k) % kGroups) * kBQ + r];
          sum += v.x == -INFINITY ? v.y : v.y * exp2_approx((v.x - mm) * scale2);  // 0 or NaN
        }
        // a sum of 0: no key seen; NaN goes on into the row
        const float inv = sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
        const int64_t flat = (static_cast<int64_t>(it.b) * a.Hq + it.h) * a.Lq + row;
        const int64_t parts = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
        const bool write = row < it.ql;
        // A whole block goes through shared memory (its Q is done with) and out by TMA: single
        // rows from the threads would take 2048 line accesses of the L1.
        const bool whole = n > 0 && it.row0 + kBQ <= it.ql && a.splits == 1;
        const auto value = [&](int k) {
          return inv == 0.f ? 0.f : __uint_as_float(o[k / 32][k % 32]) * inv;
        };
        // a finite sum beside a NaN: of a key that only other rows of the block see, or one that this does
        if (a.causal && write && inv > 0.f && limit < min(it.kl, it.row0 + kBQ + off)) {
          float most = 0.f;
#pragma unroll
          for (int k = 0; k < 64; k += 2)
            most = max3_nan(most, __uint_as_float(o[k / 32][k % 32]), __uint_as_float(o[k / 32][k % 32 + 1]));
          if (isnan(most)) *rows_left = 1;
        }
        if (a.splits > 1) {
          if (write) {
            float4* part = reinterpret_cast<float4*>(a.part + (it.split * parts + flat) * D + 64 * half);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              part[k] = make_float4(value(4 * k), value(4 * k + 1), value(4 * k + 2), value(4 * k + 3));
          }
        } else {
          uint8_t* stage = sp + C::kOffQ + qb * C::kOp + half * C::kHalf + r * 128;
          uint4* direct = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + it.b * a.o_batch +
                                                   row * a.o_row + it.h * a.o_head + 64 * half);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = pack2<F16>(value(8 * k + 2 * j), value(8 * k + 2 * j + 1));
            const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
            if (whole)
              *reinterpret_cast<uint4*>(stage + 16 * (k ^ (r & 7))) = v;
            else if (write)
              direct[k] = v;
          }
        }
        if (whole) fence_proxy_async_smem();
        __syncwarp();
        if (n > 0 && lane == 0) {
          // the last of the group's warps sends the 64 columns off, or gives the buffer back
          __threadfence_block();
          if ((atomicAdd(&staged_warps[half], 1) & (kGroupWarps - 1)) == kGroupWarps - 1) {
            if (whole) {
              __threadfence_block();
              fence_proxy_async_smem();
              see_off();
              asm volatile(
                  "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group"
                  " [%0, {%1, %2, %3, %4}], [%5];\n\tcp.async.bulk.commit_group;" ::"l"(
                      reinterpret_cast<uint64_t>(&tmO)),
                  "r"(64 * half), "r"(it.row0), "r"(it.h), "r"(it.b),
                  "r"(sbase + C::kOffQ + qb * C::kOp + half * C::kHalf)
                  : "memory");
              staged = qb;
            } else {
              mbar_arrive(bar(C::kQFree + qb));
            }
          }
        }
        if (write && half == 0) {
          const float lse =
              sum > 0.f ? (mm * scale2 + log2f(sum)) * kLn2 : (sum == sum ? -INFINITY : sum);
          if (a.splits > 1)
            a.part[parts * D * a.splits + it.split * parts + flat] = lse;
          else if (a.lse)
            a.lse[flat] = lse;
        }
        __syncwarp();
      }
    }
    see_off();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp == kTmaWarp || warp == kTmaVWarp) {
    // ---- the lists, and Q, K and V by TMA: one warp announces the items and loads Q and K, the
    // other V, as K is wanted up to three tiles before V.  The tiles of an item are pairs of its
    // entries that some row of the block sees; a warp looks at 32 entries at a time.
    const bool is_v = warp == kTmaVWarp;
    const int64_t nk = (a.Lk + kBK - 1) / kBK;
    const CUtensorMap* map = is_v ? &tmV : &tmK;
    const uint32_t ring = sbase + (is_v ? C::kOffV : C::kOffK);
    const int bar_full = is_v ? C::kVFull : C::kKFull, bar_empty = is_v ? C::kVEmpty : C::kKEmpty;
    unsigned g = 0, e = 0, loaded_q = 0, loaded = 0;
    struct List {
      const int32_t* at;
      int len, seen;  // entries of the item's range; keys that the block's last row sees
    };
    const auto list_of = [&](const Item& it) {
      const int last = min(it.row0 + kBQ, it.ql) + it.kl - it.ql;
      return List{a.blocks + ((static_cast<int64_t>(it.b) * a.Hq + it.h) * a.nq + it.row0 / kBQ) * a.T +
                      static_cast<int64_t>(it.split) * a.chunk,
                  min(a.chunk, a.T - it.split * a.chunk), a.causal ? min(it.kl, last) : it.kl};
    };
    const auto fetch = [&](const List& list, int i0) {
      return i0 + lane < list.len ? __ldg(list.at + i0 + lane) : -1;
    };
    const auto steps = [&](const List& list, int entry) {
      const bool bad = entry < -1 || entry >= nk;
      if (bad) atomicOr(&g_error_word, kErrIndex);
      return __ballot_sync(0xffffffffu, entry >= 0 && !bad && entry * kBK < list.seen);
    };
    const auto agree = [&] { ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0; };
    const auto announce = [&](const Item& it) {
      const int slot = e % kItemRing;
      if (lane == 0) {
        wait(C::kItemEmpty + slot, ((e / kItemRing) & 1) ^ 1, kErrWaitProducer);
        item_ring[slot] = it;
        mbar_arrive(bar(C::kItemFull + slot));
      }
      ++e;
      agree();
    };
    // The item after the current one is looked up and its list counted bit by bit while the
    // current one's tiles are loaded, never with a load from memory to wait for.
    unsigned next = blockIdx.x;
    Item nit;
    List nlist{};
    int n_count = 0, n_i0 = 0, n_first = -1, n_entry = -1;
    const auto look_up = [&] {  // next: the next item with rows
      for (; next < items; next += gridDim.x) {
        nit = item_at(a, next);
        if (nit.row0 >= nit.ql) continue;  // behind the sequence: such rows stay as they are
        nlist = list_of(nit);
        n_count = n_i0 = 0;
        n_first = n_entry = fetch(nlist, 0);
        break;
      }
    };
    const auto count_part = [&] {
      if (next >= items || n_i0 >= nlist.len) return;
      n_count += __popc(steps(nlist, n_entry));
      n_i0 += 32;
      n_entry = fetch(nlist, n_i0);
    };
    look_up();
    while (ok && next < items) {
      if (!is_v)
        while (n_i0 < nlist.len) count_part();
      Item it = nit;
      const List list = nlist;
      int entry = n_first, ahead = 0;
      next += gridDim.x;
      if (!is_v) {
        it.tiles = (n_count + 1) / 2;
        announce(it);
        if (lane == 0 && it.tiles > 0) {
          const int qb = loaded_q & 1;
          wait(C::kQFree + qb, ((loaded_q >> 1) & 1) ^ 1, kErrWaitProducer);
          if (ok) {
            mbar_arrive_expect_tx(bar(C::kQFull + qb), C::kOp);
            for (int d = 0; d < C::kHalves; ++d)
              tma_load_4d(sbase + C::kOffQ + qb * C::kOp + d * C::kHalf, &tmQ, 64 * d, it.row0,
                          it.h * a.q_by_head, it.b * a.q_by_batch, bar(C::kQFull + qb));
            ++loaded_q;
          }
        }
        agree();
      }
      const int hk = it.h / (a.Hq / a.Hkv);
      const int hc = hk * (is_v ? a.v_by_head : a.k_by_head);
      const int bc = it.b * (is_v ? a.v_by_batch : a.k_by_batch);
      const auto load_tile = [&](int j0, int j1) {
        if (lane == 0) {
          const int slot = static_cast<int>(g % C::kStages);
          wait(bar_empty + slot, ((g / C::kStages) & 1) ^ 1, kErrWaitProducer);
          if (ok) {
            if (!is_v) {
              // a missing second block: no key of it is seen, and it is loaded from behind the
              // last key, as zeros
              tile_ring[g % kTileRing] = make_int2(j0, j1 < a.Lk ? j1 : 0x40000000);
            }
            const uint32_t full = bar(bar_full + slot), dst = ring + slot * C::kOp;
            mbar_arrive_expect_tx(full, C::kOp);
            for (int d = 0; d < C::kHalves; ++d) {
              tma_load_4d(dst + d * C::kHalf, map, 64 * d, j0, hc, bc, full);
              tma_load_4d(dst + d * C::kHalf + C::kHalf / 2, map, 64 * d, j1, hc, bc, full);
            }
            ++loaded;
          }
        }
        __syncwarp();
        ++g;
        if (++ahead == 2)
          look_up();
        else if (!is_v && ahead > 2)
          count_part();
      };
      int first = -1;  // a tile's first block, waiting for its second
      for (int i0 = 0; i0 < list.len && ok; i0 += 32) {
        const int now = entry;
        entry = fetch(list, i0 + 32);
        for (unsigned bits = steps(list, now); bits; bits &= bits - 1) {
          const int j = __shfl_sync(0xffffffffu, now, __ffs(bits) - 1) * kBK;
          if (first < 0) {
            first = j;
          } else {
            load_tile(first, j);
            first = -1;
          }
        }
        agree();
      }
      if (first >= 0 && ok) load_tile(first, static_cast<int>(a.Lk));
      if (ahead < 2) look_up();
      agree();
    }
    if (!is_v) {
      nit.tiles = -1;
      announce(nit);
    }
    // no copy into this CTA's memory may outlive it
    if (lane == 0) {
      for (unsigned k = loaded_q > 2 ? loaded_q - 2 : 0; k < loaded_q; ++k)
        mbar_wait_limit(bar(C::kQFull + (k & 1)), (k >> 1) & 1, kWaitTimeoutNs, kErrWaitTma);
      for (unsigned k = loaded > C::kStages ? loaded - C::kStages : 0; k < loaded; ++k)
        mbar_wait_limit(bar(bar_full + k % C::kStages), (k / C::kStages) & 1, kWaitTimeoutNs,
                        kErrWaitTma);
    }
  } else if (lane == 0) {
    // ---- MMAs: one thread issues the scores, another the second products.  An issuing thread
    // stands still while the tensor cores catch up, and what it has to look at between two tiles
    // would leave them idle; two threads cover for each other.
    const bool is_pv = warp == kPvWarp;
    unsigned g = 0, q = 0;  // tiles, items with tiles
    for (unsigned e = 0; ok; ++e) {
      const int item_slot = e % kItemRing;
      wait(C::kItemFull + item_slot, (e / kItemRing) & 1, kErrWaitMma);
      if (!ok) break;
      const int n = item_ring[item_slot].tiles;
      mbar_arrive(bar(C::kItemEmpty + item_slot));
      if (n < 0) break;
      if (n == 0) continue;
      const int qb = q & 1;
      if (!is_pv) {
        constexpr uint32_t idesc = idesc_f16(128, kTileK, F16, false);
        wait(C::kQFull + qb, (q >> 1) & 1, kErrWaitTma);
        const uint32_t aq = sbase + C::kOffQ + qb * C::kOp;
        for (int t = 0; t < n && ok; ++t, ++g) {
          const int slot = static_cast<int>(g % C::kStages), buf = static_cast<int>(g % kGroups);
          // the buffer is free when P V of the tile three before is done
          wait(C::kKFull + slot, (g / C::kStages) & 1, kErrWaitTma);
          wait(C::kPvDone + buf, ((g / kGroups) & 1) ^ 1, kErrWaitMma);
          if (!ok) break;
          tc_fence_after();
          const uint32_t bk = sbase + C::kOffK + slot * C::kOp;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t at = (s / 4) * C::kHalf + (s % 4) * 32;
            mma_ss(tmem + kColS + kTileK * buf, smem_desc_sw128(aq + at), smem_desc_sw128(bk + at),
                   idesc, s != 0);
          }
          mbar_arrive(bar(C::kSFull + buf));  // hands on the tile ring's entry, which came before K
          mma_commit(bar(C::kSFull + buf));
          mma_commit(bar(C::kKEmpty + slot));
        }
        mma_commit(bar(C::kQFree + qb));
      } else {
        constexpr uint32_t idesc = idesc_f16(128, D, F16, true);
        // O is free when the item before has been written out
        wait(C::kOFree, (q & 1) ^ 1, kErrWaitEpilogue);
        for (int t = 0; t < n && ok; ++t, ++g) {
          const int slot = static_cast<int>(g % C::kStages), buf = static_cast<int>(g % kGroups);
          const uint32_t bv = sbase + C::kOffV + slot * C::kOp;
          wait(C::kVFull + slot, (g / C::kStages) & 1, kErrWaitTma);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            wait(C::kPFull + 2 * buf + half, (g / kGroups) & 1, kErrWaitMma);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int s = half * kBK / 16; s < (half + 1) * kBK / 16; ++s)
              mma_ts(tmem + kColO, tmem + kColS + kTileK * buf + 8 * s,
                     smem_desc_mn(bv + s * 2048, C::kHalf), idesc, t != 0 || s != 0);
          }
          if (!ok) break;
          mma_commit(bar(C::kPvDone + buf));
          mma_commit(bar(C::kVEmpty + slot));
        }
      }
      ++q;
    }
    // the tensor memory is given back only when nothing writes it any more
    const int drain = C::kDrain + (is_pv ? 1 : 0);
    mma_commit(bar(drain));
    mbar_wait_limit(bar(drain), 0, kWaitTimeoutNs, kErrWaitMma);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  if (*rows_left) rows_again<D, F16>(a, items);
}

// Joins the parts of each row, in the order of the splits: a warp takes a row.  (Four parts at a
// time cost more than they hid: 24.5 against 22.6 us for 32 heads of 64 rows.)
template <int D, bool F16>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  const int64_t parts = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  const int64_t flat = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
    float src[V];
    const float* at = a.part + (s * parts + flat) * D + V * lane;
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(src) = *reinterpret_cast<const float4*>(at);
    } else {
      static_assert(V == 2, "a lane takes two or four elements");
      *reinterpret_cast<float2*>(src) = *reinterpret_cast<const float2*>(at);
    }
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

// The lists are cut (in pairs of entries) where that shortens the longest CTA's work: rounds of
// items times the tiles of an item, of which about two more go to its beginning and end.  Parts
// cost a second kernel, worth two tiles, and to be written and read in binary32, a tile's time for
// 2048 of their rows.  Whole / cut, us, D 128: 40 heads, 1 row, 256 entries 128 / 69; 32 heads,
// 300 rows, 256 entries 134 / 112; 8 heads, 1024 rows, 16 entries 16.7 / 22.6; 40 heads, 512 rows,
// 64 entries 75 / 82.
inline Plan plan(int64_t B, int64_t Hq, int64_t Lq, int64_t T) {
  const int64_t items = B * Hq * ((Lq + kBQ - 1) / kBQ);
  Plan best{1, static_cast<int>(T)};
  const int64_t tiles = (T + 1) / 2;
  int64_t least = 0;
  const int64_t most = 1 + 2 * kSms / items;  // more than two items per CTA gain nothing
  for (int64_t s = 1; s <= tiles && s <= most; ++s) {
    const int64_t chunk = (tiles + s - 1) / s, splits = (tiles + chunk - 1) / chunk;
    const int64_t cost = (items * splits + kSms - 1) / kSms * (chunk + 2) +
                         (splits > 1 ? 2 + B * Hq * Lq * splits / 2048 : 0);
    if (s == 1 || cost < least)
      least = cost, best = {static_cast<int>(splits), static_cast<int>(2 * chunk)};
  }
  return best;
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
                   const CUtensorMap& o, const Args& a, int sms, cudaStream_t stream) {
  auto kern = attn_kernel<D, F16>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Cfg<D>::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hq * a.nq * a.splits;
  const int grid = static_cast<int>(items < sms ? items : sms);
  kern<<<grid, kThreads, Cfg<D>::kSmemBytes, stream>>>(q, k, v, o, a);
  const cudaError_t l = cudaGetLastError();
  if (l != cudaSuccess || a.splits == 1) return l;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq * a.Lq;
  return launch_behind(join_kernel<D, F16>, dim3(static_cast<unsigned>((rows + 7) / 8)), 256, 0,
                       stream, a);
}

}  // namespace attn
}  // namespace qs
