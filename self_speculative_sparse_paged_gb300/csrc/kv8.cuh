// The 8-bit cache's element format, shared by the kernels that write and read it.
//
// A block is one page (16 positions) of one KV head.  An element is an e4m3 code c (four bits of
// exponent, three of fraction, largest 448) and stands for c * 2^e, with one exponent a block for K
// and one for V, held as the byte e + 127.  Powers of two, because then a block's exponent can be
// raised when a later row is larger and the codes it holds stay exact (but for those that become
// subnormal), every c * 2^e is exact in bf16, and applying a scale never rounds.
#pragma once

#include <cuda_fp16.h>

#include "vegas_common.cuh"

namespace vegas {

constexpr int kKv8MinExp = -60, kKv8MaxExp = 60, kKv8Bias = 127;

// The exponent of a scale byte.  The append writes bytes within the range; others are clamped,
// so that no content makes an infinite or zero scale.
__device__ __forceinline__ int kv8_exponent(uint8_t byte) {
  return max(kKv8MinExp, min(kKv8MaxExp, int(byte) - kKv8Bias));
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Row sums over blocks whose scales lie far apart.  With x a logit in binades and e_v the block's exponent,
// P = 2^(x + e_v - r) multiplies the codes and P 2^-e_v goes into the row's sum.  References r follow
// x + e_v, so they lie up to 120 binades above what a term of the sum alone would need, and what weighs in
// the sum may have a P that fp32 does not hold (the exponential gives 0 below 2^-126).  Hence
//  - a sum that moves from one reference to another takes 2^(d / 2) twice for 2^d: after the first its own
//    2^-e_v has it in range;
//  - blocks of e_v < kKv8Deep take their terms of the sum from an exponential that is 2^kKv8Lift larger.
// As r <= max(x + e_v) - 7, a term is lost 45 binades below the row's heaviest (126 + kKv8Deep - 60 + 7), one
// of a deep block 77 below it.
constexpr int kKv8Deep = -28, kKv8Lift = 64;

// The least exponent whose block holds a magnitude of these bf16 bits (sign removed, finite):
// x = 1.f * 2^n <= 1.75 * 2^8 * 2^e.
__device__ __forceinline__ int kv8_exponent_for(uint32_t bf16_bits) {
  const int n = int(bf16_bits >> 7) - 127;
  const int e = bf16_bits < 0x80u ? kKv8MinExp : n - 8 + ((bf16_bits & 0x7fu) > 0x60u ? 1 : 0);
  return max(kKv8MinExp, min(kKv8MaxExp, e));
}

// Two codes, lo in the lower byte; round to nearest even, beyond 448 saturates, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Codes 0, 1 (lo) and 2, 3 (hi) of a word as f16 pairs; exact.
__device__ __forceinline__ void f16x2_from_e4m3x4(uint32_t word, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(word));
}
__device__ __forceinline__ float2 f32x2_from_f16x2(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace vegas
