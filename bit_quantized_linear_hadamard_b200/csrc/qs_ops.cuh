// What the operators around the projections share on the device.
#pragma once

#include <cstdint>

#include "qs_ptx.cuh"

namespace qs {
namespace ops {

// A length given on the device, held to [0, most]; outside it the error word is raised.
__device__ __forceinline__ int64_t checked_len(const int32_t* len, int b, int64_t most) {
  if (!len) return most;
  const int64_t n = len[b];
  if (n < 0 || n > most) {
    atomicOr(&g_error_word, kErrIndex);
    return n < 0 ? 0 : most;
  }
  return n;
}

// The largest, or NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Instruction descriptor: kind::f16, binary32 D, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool f16, bool b_mn) {
  return (1u << 4)                                 // D format: F32
         | ((f16 ? 0u : 1u) << 7)                  // A: F16 or BF16
         | ((f16 ? 0u : 1u) << 10)                 // B: the same
         | ((b_mn ? 1u : 0u) << 16)                // B: N contiguous
         | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

// Both operands from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace ops
}  // namespace qs
