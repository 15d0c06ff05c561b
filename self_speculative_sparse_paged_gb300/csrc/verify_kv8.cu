// Verify attention with captured scores over the 8-bit cache, on the 5th-generation tensor cores
// (compiled once per head_dim, VEGAS_KV8_D).
//
// The work is that of verify_tc.cu on half the bytes, laid out so that its length goes by what the
// sequences hold, not by what their tables could: the 128-position tiles of all (sequence, KV
// head) units stand in one row, and each CTA (one an SM) takes an equal run of it, whole units or
// pieces, with the K/V stream going on from one unit to the next.  Twelve
// warps:
//   0-7   two softmax groups of four warps that alternate tiles; a thread owns a position of a tile,
//         and a head dimension of O^T.  They also build the query operand of a unit and finish it.
//   8, 9  TMA producers: 8 pages a tile into K and V rings, block-table entries prefetched
//   10    issues the MMAs
//
//   S^T[128 pos x N] = K Q^T   kind::f8f6f4, M = 128: K's codes go to the tensor cores as the
//       TMA left them.  A query row, scaled by a power of two 2^k, is the sum of two e4m3
//       parts (4 + 4 bits of bf16's 8), so the products are exact.  Captured scores take the
//       summed captured query (fp32) in six parts, two and two 2^8 apart.  (kind::f8f6f4
//       sums e4m3 products to fp32's precision here: 2.3e-7 of the terms' sum at worst, measured
//       over random codes.)
//   z = S 2^(e_k - k) scale log2(e) + e_v,  P = 2^(z - r) with r a reference for the column:
//       e_k costs nothing (a thread's one factor), and 2^e_v goes into P instead of V.  Row sums
//       take P 2^-e_v in fp32.
//   O^T[D x N] += V^T P^T   kind::f8f6f4, M = D: V's codes as they lie (read MN-major), P as the
//       sum of three e5m2 parts.  e5m2 is the upper byte of f16, so the parts are cut off P's f16
//       (each takes three bits or more, the last is rounded: with f16's own rounding 1.1 * 2^-9 of P at
//       most, just below 1.1426 * 2^e), with f16's range.
//       Turning V into f16 instead moved 1200-1300 clocks' worth of a tile's 1425 through
//       shared memory at head_dim 128, which bounded that kernel (172-179 us on a batch of eight
//       of 49K-64K); this one moves about 750.
//
// Parts lie side by side in N where tensor memory holds their columns (one pass over the A
// operand; an MMA takes 45 clocks up to N = 64 and 64 at 128), else they share an accumulator.
// P <= 2^15 (f16 ends at 65504) and the largest P is 2^11 or more when r was raised, so P's grid
// reaches 2^-28 below the largest.  e_v spans 120 binades, and row sums keep what weighs in them all the
// same (kv8.cuh).
//
// A unit that one CTA covers is written by it; the pieces of a shared one go to the workspace
// (fp32 O, maximum and sum of each row), and the CTA that arrives last on the unit's ticket merges
// them.  No CTA waits for another.
//
// What bounds it.  Long batches of 24 columns at head_dim 128: the DRAM stream (a tile's 735 ns at
// the copy peak, of which the softmax needs about 300).  One long sequence: what comes before and
// behind the stream (launch, division of the work 1.2 us, queries 0.9, first tile 1.5, end 1, partial state
// and ticket 1.8, merge 1.6-3).  Many short sequences: 5 us a unit beside the stream (queries 1800 clocks,
// first S 1300, first reference 1600, end 2500).  56 columns at head_dim 64: the softmax's latency, 1900
// clocks a tile with two warps a scheduler (no step above 550; without the row sums 8 us of 224 less, with P
// in one f16 part and V turned by four more warps 29 us more).
//   8 x 49K-64K, 24 columns of 128    158 us (0.90 of the copy peak)     32K: 23.4     64 x 1000: 44.4
//   4 x 128K, 56 columns of 64        197 us (0.42)    one token each of 12 up to 8K: 17.6    2K, 20 of 64: 10.2
#include "attn_core.cuh"
#include "kernels.h"
#include "kv8.cuh"
#include "lengths.h"

#ifndef VEGAS_KV8_D
#error "compile with -DVEGAS_KV8_D=64 or -DVEGAS_KV8_D=128"
#endif

namespace vegas {

namespace {
constexpr float kTop = 15.f, kRaise = 11.f;   // log2 of the largest P, and of P at a raised reference
constexpr int kCapParts = 6;
constexpr int kSoftWarps = 8, kWarps = 12, kSoft = 32 * kSoftWarps, kThreads = 32 * kWarps;
// In the division of the work a unit counts kUnitTiles tiles more than it has (its queries, first
// reference and end; with 5, 6, 7: 12 ragged single tokens 17.2, 17.5, 17.9 us, 8 x 2K 17.6, 17.2, 17.0,
// 4 x 128K of 64 196.6, 195.9, 195.0), and a CTA takes part for kLeastRun tiles or more (1, 4, 8, by an
// earlier kernel: one of 4K 15.3, 14.1, 15.4 us, one of 2K 11.8, 12.0, 14.3).
constexpr int kUnitTiles = 6, kLeastRun = 4;
constexpr int kMixed = 1000;   // (in place of the rows' common exponent) rows have their own

// Instruction descriptor, kind::f8f6f4 (K = 32), fp32 accumulator: A e4m3, B e4m3 or e5m2, both
// K-major or both MN-major (N in whole 16-byte units then).
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, int b_e5m2, int mn_major) {
  return (1u << 4) | (uint32_t(b_e5m2) << 10) | (uint32_t(mn_major) << 15) |
         (uint32_t(mn_major) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Consecutive fp32 columns of this thread's lane as pairs; complete on return.
template <int N>
__device__ __forceinline__ void tmem_ld_pairs(uint32_t a, uint64_t* v) {
  static_assert(N == 8 || N == 16 || N == 24 || N == 32, "columns");
  if constexpr (N == 8) {
    asm volatile(
        "{\n .reg .b32 t<8>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7}, [%4];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3])
        : "r"(a)
        : "memory");
  }
  if constexpr (N == 16) {
    asm volatile(
        "{\n .reg .b32 t<16>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15}, [%8];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7])
        : "r"(a)
        : "memory");
  }
  if constexpr (N == 24) {
    asm volatile(
        "{\n .reg .b32 t<24>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15}, [%12];\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t16, t17, t18, t19, t20, t21, t22, t23}, [%13];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        " mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11])
        : "r"(a), "r"(a + 16)
        : "memory");
  }
  if constexpr (N == 32) {
    asm volatile(
        "{\n .reg .b32 t<32>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15, "
        "t16, t17, t18, t19, t20, t21, t22, t23, "
        "t24, t25, t26, t27, t28, t29, t30, t31}, [%16];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        " mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n"
        " mov.b64 %12, {t24, t25}; mov.b64 %13, {t26, t27}; mov.b64 %14, {t28, t29}; mov.b64 %15, {t30, t31};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(v[12]),
          "=l"(v[13]), "=l"(v[14]), "=l"(v[15])
        : "r"(a)
        : "memory");
  }
}
// The same of two column ranges at once.
template <int N>
__device__ __forceinline__ void tmem_ld_pairs(uint32_t a, uint64_t* v, uint32_t b, uint64_t* w) {
  if constexpr (N == 8) {
    asm volatile(
        "{\n .reg .b32 t<16>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7}, [%8];\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t8, t9, t10, t11, t12, t13, t14, t15}, [%9];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(w[0]), "=l"(w[1]), "=l"(w[2]),
          "=l"(w[3])
        : "r"(a), "r"(b)
        : "memory");
  }
  if constexpr (N == 16) {
    asm volatile(
        "{\n .reg .b32 t<32>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15}, [%16];\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t16, t17, t18, t19, t20, t21, t22, t23, "
        "t24, t25, t26, t27, t28, t29, t30, t31}, [%17];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        " mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n"
        " mov.b64 %12, {t24, t25}; mov.b64 %13, {t26, t27}; mov.b64 %14, {t28, t29}; mov.b64 %15, {t30, t31};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7]), "=l"(w[0]), "=l"(w[1]), "=l"(w[2]), "=l"(w[3]), "=l"(w[4]), "=l"(w[5]),
          "=l"(w[6]), "=l"(w[7])
        : "r"(a), "r"(b)
        : "memory");
  }
  if constexpr (N == 24) {
    asm volatile(
        "{\n .reg .b32 t<48>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15}, [%24];\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t16, t17, t18, t19, t20, t21, t22, t23}, [%25];\n"
        " tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "t24, t25, t26, t27, t28, t29, t30, t31, "
        "t32, t33, t34, t35, t36, t37, t38, t39}, [%26];\n"
        " tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "t40, t41, t42, t43, t44, t45, t46, t47}, [%27];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        " mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n"
        " mov.b64 %12, {t24, t25}; mov.b64 %13, {t26, t27}; mov.b64 %14, {t28, t29}; mov.b64 %15, {t30, t31};\n"
        " mov.b64 %16, {t32, t33}; mov.b64 %17, {t34, t35}; mov.b64 %18, {t36, t37}; mov.b64 %19, {t38, t39};\n"
        " mov.b64 %20, {t40, t41}; mov.b64 %21, {t42, t43}; mov.b64 %22, {t44, t45}; mov.b64 %23, {t46, t47};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(w[0]),
          "=l"(w[1]), "=l"(w[2]), "=l"(w[3]), "=l"(w[4]), "=l"(w[5]), "=l"(w[6]), "=l"(w[7]),
          "=l"(w[8]), "=l"(w[9]), "=l"(w[10]), "=l"(w[11])
        : "r"(a), "r"(a + 16), "r"(b), "r"(b + 16)
        : "memory");
  }
  if constexpr (N == 32) {
    asm volatile(
        "{\n .reg .b32 t<64>;\n"
        " tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "t0, t1, t2, t3, t4, t5, t6, t7, "
        "t8, t9, t10, t11, t12, t13, t14, t15, "
        "t16, t17, t18, t19, t20, t21, t22, t23, "
        "t24, t25, t26, t27, t28, t29, t30, t31}, [%32];\n"
        " tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "t32, t33, t34, t35, t36, t37, t38, t39, "
        "t40, t41, t42, t43, t44, t45, t46, t47, "
        "t48, t49, t50, t51, t52, t53, t54, t55, "
        "t56, t57, t58, t59, t60, t61, t62, t63}, [%33];\n"
        " tcgen05.wait::ld.sync.aligned;\n"
        " mov.b64 %0, {t0, t1}; mov.b64 %1, {t2, t3}; mov.b64 %2, {t4, t5}; mov.b64 %3, {t6, t7};\n"
        " mov.b64 %4, {t8, t9}; mov.b64 %5, {t10, t11}; mov.b64 %6, {t12, t13}; mov.b64 %7, {t14, t15};\n"
        " mov.b64 %8, {t16, t17}; mov.b64 %9, {t18, t19}; mov.b64 %10, {t20, t21}; mov.b64 %11, {t22, t23};\n"
        " mov.b64 %12, {t24, t25}; mov.b64 %13, {t26, t27}; mov.b64 %14, {t28, t29}; mov.b64 %15, {t30, t31};\n"
        " mov.b64 %16, {t32, t33}; mov.b64 %17, {t34, t35}; mov.b64 %18, {t36, t37}; mov.b64 %19, {t38, t39};\n"
        " mov.b64 %20, {t40, t41}; mov.b64 %21, {t42, t43}; mov.b64 %22, {t44, t45}; mov.b64 %23, {t46, t47};\n"
        " mov.b64 %24, {t48, t49}; mov.b64 %25, {t50, t51}; mov.b64 %26, {t52, t53}; mov.b64 %27, {t54, t55};\n"
        " mov.b64 %28, {t56, t57}; mov.b64 %29, {t58, t59}; mov.b64 %30, {t60, t61}; mov.b64 %31, {t62, t63};\n"
        "}"
        : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
          "=l"(v[7]), "=l"(v[8]), "=l"(v[9]), "=l"(v[10]), "=l"(v[11]), "=l"(v[12]),
          "=l"(v[13]), "=l"(v[14]), "=l"(v[15]), "=l"(w[0]), "=l"(w[1]), "=l"(w[2]),
          "=l"(w[3]), "=l"(w[4]), "=l"(w[5]), "=l"(w[6]), "=l"(w[7]), "=l"(w[8]), "=l"(w[9]),
          "=l"(w[10]), "=l"(w[11]), "=l"(w[12]), "=l"(w[13]), "=l"(w[14]), "=l"(w[15])
        : "r"(a), "r"(b)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_ld4(uint32_t a, float (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(a));
}
// Behind the wait for loads of v (of its first Used elements): the wait does not name them, and no use of
// them may move ahead of it.
template <int Used = 0, int N>
__device__ __forceinline__ void loaded(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < (Used ? Used : N); ++i) asm volatile("" : "+f"(v[i]));
}
// Whether the phase with the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Takes a ticket, with everything before it released and everything after it acquired.
__device__ __forceinline__ int ticket_acq_rel(int* t) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(t) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// sum += 2^(y + kKv8Lift) f, of a pair.  (In one piece: as separate steps their temporaries cost the
// registers of the whole loop, 8 x 50K with 64 columns of 64: 207 -> 222 us.)
__device__ __forceinline__ void add_lifted(uint64_t& sum, uint64_t y, float f) {
  asm volatile(
      "{\n .reg .f32 a, b, c, d;\n mov.b64 {a, b}, %1;\n mov.b64 {c, d}, %0;\n"
      " add.f32 a, a, %3;\n add.f32 b, b, %3;\n ex2.approx.ftz.f32 a, a;\n ex2.approx.ftz.f32 b, b;\n"
      " fma.rn.f32 c, a, %2, c;\n fma.rn.f32 d, b, %2, d;\n mov.b64 %0, {c, d};\n}"
      : "+l"(sum)
      : "l"(y), "f"(f), "f"(float(kKv8Lift)));
}
// op over the warp's lanes of each of eight columns: lane l gets column l / 4's.  In three steps a
// lane exchanges half of the columns it still holds for the other half of another lane's.
template <class Op>
__device__ __forceinline__ float reduce_chunk(const float* x, Op op) {
  const int lane = threadIdx.x & 31;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x[j];
#pragma unroll
  for (int w = 16; w >= 4; w >>= 1) {
    const bool upper = lane & w;
#pragma unroll
    for (int j = 0; j < w / 4; ++j) {
      const float give = upper ? v[j] : v[j + w / 4], keep = upper ? v[j + w / 4] : v[j];
      v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
}  // namespace

template <int D, int NQC, bool CAPTURE>
struct Kv8Cfg {
  // S: [high parts | low parts | capture parts] side by side, or the two parts of NQC + 3 columns
  // one after the other.
  static constexpr bool kSideS = NQC <= 40;
  static constexpr int kCap = CAPTURE ? (kSideS ? kCapParts : kCapParts / 2) : 0;
  static constexpr int kCap0 = kSideS ? 2 * NQC : NQC;    // first capture column
  static constexpr int NS = (kCap0 + kCap + 15) / 16 * 16;   // N of S
  // PV: three parts side by side, or one after the other (NQC = 64)
  static constexpr bool kSideP = NQC <= 56;
  // columns from one part to the next: whole 16-byte chunks, where P's room holds them
  static constexpr int PS = !kSideP ? 128 : NQC == 40 ? 40 : (NQC + 15) / 16 * 16;
  static constexpr int kParts = kSideP ? 3 : 1;       // accumulators
  static constexpr int kPCols = kSideP ? 3 * PS : NQC;
  static constexpr int NP = (kPCols + 15) / 16 * 16;  // N of PV
  static constexpr int kTile = 128 * D;               // one K tile (and one V tile): 8 pages
  // P of a position: rows of 128 bytes in blocks of 128 positions, [part][PS] over the blocks, or a
  // block a part
  static constexpr int kBlocks = kSideP ? (NP + 127) / 128 : 3;
  static constexpr int kP = kBlocks * 128 * 128;
  // Ring slots of K and V (16 KB at head_dim 128, 8 KB at 64).  Few: what more of them ask for ahead only
  // disturbs the memory (128, K and V slots 5 + 6, 4 + 5, 3 + 5, 2 + 5: batch of eight 163.8, 161.5, 156.3,
  // 169.9 us, 32K 23.4, 22.7, 23.0, 23.3; 64, 8 + 10, 6 + 6, 5 + 5, 4 + 4: 4 x 128K 202, 196, 195, 194, 8 x 50K
  // with 24 columns -, -, 111.9, 114.0).
  static constexpr int KS = D == 128 ? 3 : 5, VS = 5;
  static constexpr int kQ = NS * D;                   // Q^T operand, one a pass
  static constexpr int kPasses = kSideS ? 1 : 2;
  static constexpr int kSCol = (NS + 31) / 32 * 32, kOCol = (NP + 31) / 32 * 32;
  static constexpr uint32_t kTmemCols =
      2 * (kSCol + kOCol) <= 128 ? 128 : 2 * (kSCol + kOCol) <= 256 ? 256 : 512;
  static_assert(2 * (kSCol + kOCol) <= 512, "tensor memory");
  static constexpr int kOffV = KS * kTile;
  static constexpr int kOffP = kOffV + VS * kTile;
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffBar = kOffQ + kPasses * kQ;
  static constexpr int kNumBars = 2 * KS + 2 * VS + 4 * 2 + 2;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
  // misc: 16 words; votes[2][2][4]; warp sums[12] (64 bits); colmax[2][4][NQC], colsum[2][4][NQC],
  // colfac[NQC], nref[2][NQC], fac[2][NQC], wgt[2][NQC], colM[NQC], colL[NQC]; tlim[NQC]; rowexp[NQC];
  // rowat[NQC]
  static constexpr size_t kMisc = 64 + 64 + 96 + 4 * size_t(16 + 1 + 2 + 2 + 2 + 2 + 2 + 1) * NQC;
  static constexpr size_t kSmem = size_t(kOffMisc) + kMisc + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(8 * D * 4 <= kP, "partial sums of the captured query (P's buffer)");
};

// A place in the row of tiles: tile t of KV head g of sequence b.
struct Place {
  long long left;          // of the CTA's run from here on
  int b, g, t, tiles, L;   // tiles: of each unit of sequence b; L: its context length
  int pre;                 // of the run, before tile t
  // tiles of the unit in the run; 0: the run is over
  __device__ int here() const {
    return left > pre ? int(min((long long)(tiles - t), left - pre)) : 0;
  }
};

template <int D, int NQC, bool CAPTURE>
__global__ void __launch_bounds__(kThreads, 1)
    verify_kv8_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const VerifyKv8Params p) {
  using Cfg = Kv8Cfg<D, NQC, CAPTURE>;
  constexpr int KS = Cfg::KS, VS = Cfg::VS, NS = Cfg::NS, NP = Cfg::NP;
  constexpr bool kSideS = Cfg::kSideS, kSideP = Cfg::kSideP;
  constexpr int kAllBar = 3;   // named barriers: 1 + group, and all softmax threads
  static_assert(NQC % 8 == 0 && (D == 64 || D == 128), "columns, head_dim");

  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::kOffBar;
  // barriers: K full/free (per K slot), V full/free (per V slot); S full, S read, P ready, PV done
  // (per softmax group); queries ready, MMA drain
  auto kfull = [&](int s) { return bar0 + 8 * s; };
  auto kfree = [&](int s) { return bar0 + 8 * (KS + s); };
  auto vfull = [&](int s) { return bar0 + 8 * (2 * KS + s); };
  auto vfree = [&](int s) { return bar0 + 8 * (2 * KS + VS + s); };
  constexpr int B1 = 2 * KS + 2 * VS;
  auto sfull = [&](int g2) { return bar0 + 8 * (B1 + g2); };
  auto sread = [&](int g2) { return bar0 + 8 * (B1 + 2 + g2); };
  auto pready = [&](int g2) { return bar0 + 8 * (B1 + 4 + g2); };
  auto pvdone = [&](int g2) { return bar0 + 8 * (B1 + 6 + g2); };
  const uint32_t qready = bar0 + 8 * (B1 + 8), drain = bar0 + 8 * (B1 + 9);
  uint8_t* misc = smem + Cfg::kOffMisc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  int* flag = reinterpret_cast<int*>(misc + 4);
  int* capexp = reinterpret_cast<int*>(misc + 8);
  int* uniform = reinterpret_cast<int*>(misc + 12);
  int* votes = reinterpret_cast<int*>(misc + 64);                // [2][2][4]
  long long* wsum = reinterpret_cast<long long*>(misc + 128);    // [12] a warp's sequences
  float* colmax = reinterpret_cast<float*>(misc + 224);          // [2][4][NQC]
  float* colsum = colmax + 8 * NQC;                              // [2][4][NQC]
  float* colfac = colsum + 8 * NQC;                              // [NQC] 2^-k of rows of unlike size
  float* nrefs = colfac + NQC;                                   // [2][NQC] -reference
  float* facs = nrefs + 2 * NQC;                                 // [2][NQC] factors of a raise
  float* wgt = facs + 2 * NQC;                                   // [2][NQC] weights of the groups
  float* colM = wgt + 2 * NQC;                                   // [NQC] maximum, and sum, of a piece
  float* colL = colM + NQC;
  int* tlim = reinterpret_cast<int*>(colL + NQC);                // [NQC]
  int* rowexp = tlim + NQC;                                      // [NQC]
  int* rowat = rowexp + NQC;   // [NQC] where a column's row of q and out is, from the unit's first
  float* qsum = reinterpret_cast<float*>(smem + Cfg::kOffP);     // [softmax warps][D] of the captured sum

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int T = p.gamma + 1;
  const int cap = p.max_pages * 16;

  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kfree(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(vfull(s), 1);
      mbar_init(vfree(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull(i), 1);
      mbar_init(sread(i), 128);
      mbar_init(pready(i), 128);
      mbar_init(pvdone(i), 1);
    }
    mbar_init(qready, kSoft);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == kSoftWarps + 2) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  // (once, and not in every unit: quotients by a number known at run time take a hundred clocks)
  for (int n2 = tid; n2 < NQC; n2 += kThreads) {
    const int t = n2 / p.group, hl = n2 - t * p.group;
    tlim[n2] = n2 < p.nq ? t : -1;
    rowat[n2] = (t * p.hq + hl) * D;
  }
  tc_fence_before();
  __syncthreads();   // (the barriers are initialised, and tensor memory is there)
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Nothing above reads or writes global memory, so it overlaps the tail of
  // the previous kernel of the stream.
  griddep_wait();

  // ---- this CTA's run.  A sequence's units have ceil((L + T) / 128) tiles each.
  auto length = [&](int b) { return nearest_length(p.ctx_lens[b], T, cap); };   // (recorded below)
  auto tiles_of = [&](int L) { return (L + T + 127) >> 7; };
  auto span_of = [&](int L) { return (long long)(tiles_of(L) + kUnitTiles) * p.hkv; };
  // Up to 32 sequences every warp scans by itself; else warp w first counts [w * chunk, (w + 1) *
  // chunk).
  const int chunk = (p.batch + kThreads - 1) / kThreads * 32;
  long long all = 0;
  int first_chunk = 0;
  if (p.batch > 32) {
    long long sum = 0;
    for (int b = warp * chunk + lane; b < min(p.batch, (warp + 1) * chunk); b += 32)
      sum += span_of(length(b));
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
    if (lane == 0) wsum[warp] = sum;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) all += wsum[w];
  }
  long long upto = 0;    // this lane's sequence and those before it, of 32
  int mylen = 0;
  auto scan = [&](int b0) {
    const int b = b0 + lane;
    mylen = b < p.batch ? length(b) : 0;
    upto = b < p.batch ? span_of(mylen) : 0;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o2);
      if (lane >= o2) upto += v;
    }
  };
  if (p.batch <= 32) {
    scan(0);
    all = __shfl_sync(0xffffffffu, upto, 31);
  }
  if (cta == 0)   // lengths out of range are recorded once
    for (int b = tid; b < p.batch; b += kThreads)
      if (!length_fits(p.ctx_lens[b], T, cap)) set_error(p.err, kErrDeviceFault);
  // CTAs that take part
  const int n = int(max(1ll, min((long long)gridDim.x, all / kLeastRun)));
  // (64-bit quotients take a few hundred clocks: 32-bit ones while they do)
  const bool small = all < (1 << 24);   // (n < 2^8)
  auto quotient = [&](long long a, long long d) {
    return small ? (long long)(uint32_t(a) / uint32_t(d)) : a / d;
  };
  auto run_begin = [&](int c) { return quotient(c * all, n); };
  const long long begin = cta < n ? run_begin(cta) : 0, end = cta < n ? run_begin(cta + 1) : 0;
  // the CTA that holds place x: the last c with run_begin(c) <= x
  auto cta_of = [&](long long x) { return int(quotient((x + 1) * n - 1, all)); };
  Place start{end - begin, 0, 0, 0, 1, 0, 0};
  long long base = 0;   // where sequence start.b begins
  if (begin < end) {
    int b0 = 0;
    if (p.batch > 32) {
      for (; first_chunk < kWarps - 1 && base + wsum[first_chunk] <= begin; ++first_chunk)
        base += wsum[first_chunk];
      b0 = first_chunk * chunk;
    }
    for (;; b0 += 32) {
      if (p.batch > 32) scan(b0);
      const unsigned beyond = __ballot_sync(0xffffffffu, base + upto > begin);
      if (beyond || b0 + 32 >= p.batch) {
        const int l = beyond ? __ffs(beyond) - 1 : 31;   // (there is one: begin < end <= all)
        start.b = min(b0 + l, p.batch - 1);
        start.L = __shfl_sync(0xffffffffu, mylen, l);
        base += __shfl_sync(0xffffffffu, upto, l) - span_of(start.L);
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    start.tiles = tiles_of(start.L);
    const int span = start.tiles + kUnitTiles;
    start.g = int(quotient(begin - base, span));
    const int off = int((begin - base) - (long long)start.g * span);   // in the unit's span
    start.t = max(0, off - kUnitTiles);
    start.pre = max(0, kUnitTiles - off);
  }
  auto next_unit = [&](Place& q, int done) {   // (done: tiles of the unit that were here)
    q.left -= q.pre + done;
    q.t = 0;
    q.pre = kUnitTiles;
    if (++q.g == p.hkv) {
      q.g = 0;
      if (q.left > 0) {
        q.L = length(++q.b);
        q.tiles = tiles_of(q.L);
      }
    }
  };
  bool ok = true;

  // 384 threads launch with 168 registers each: 2 x 128 x 216 + 128 x 72 are that.
  if (warp >= kSoftWarps) {
    leave_registers<72>();
    if (warp < kSoftWarps + 2) {
      // ---------------------------------------------------------- producers: K, V
      // Lane j < 8 loads page j of a tile; a page past the sequence's last is that one again (its
      // positions are masked).
      const bool is_k = warp == kSoftWarps;
      const int depth = is_k ? KS : VS;
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      const uint32_t ring = sbase + (is_k ? 0 : Cfg::kOffV);
      // The cache is streamed once per pass: its lines leave L2 first.
      const uint64_t stream_pol = l2_evict_first_policy();
      const int j8 = lane & 7;
      Place ahead = start;
      int rest = ahead.here(), done = rest;   // tiles of the unit still to be requested, and of them all
      // a tile's table entry, requested four tiles before its use, and its KV head (-1: no tile)
      int held[4], head[4];
      auto request = [&](int j) {
        held[j] = 0;
        head[j] = -1;
        if (rest > 0) {
          const int page = min(8 * ahead.t + j8, (ahead.L + T - 1) >> 4);
          held[j] = __ldg(&p.block_table[size_t(ahead.b) * p.max_pages + page]);
          head[j] = ahead.g;
          ++ahead.t;
          if (--rest == 0) {
            next_unit(ahead, done);
            rest = done = ahead.here();
          }
        }
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) request(j);
      int issued = 0;
      int s = 0, round = 0;
      bool more = true;
      while (more && ok) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (head[j] < 0) {
            more = false;
            break;
          }
          const uint32_t full = is_k ? kfull(s) : vfull(s);
          const uint32_t freed = is_k ? kfree(s) : vfree(s);
          if (round > 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(freed, (round - 1) & 1))) {
            ok = false;
            break;
          }
          int phys = held[j];
          const int g = head[j];
          request(j);
          if (phys < 0 || phys >= p.num_pages) {
            set_error(p.err, kErrDeviceFault);
            phys = 0;
          }
          if (lane == 0) mbar_arrive_expect_tx(full, Cfg::kTile);
          __syncwarp();
          if (lane < 8)
            tma_load_2d_hint(ring + s * Cfg::kTile + j8 * 16 * D, map, 0, (phys * p.hkv + g) * 16,
                             full, stream_pol);
          __syncwarp();
          if (issued < depth) ++issued;
          if (++s == depth) {
            s = 0;
            ++round;
          }
        }
      }
      if (!ok) {   // what is in flight lands before the CTA ends
        if (lane == 0) set_error(p.err, kErrDeviceTimeout);
        for (int k = 0; k < issued; ++k) {
          if (--s < 0) {
            s = depth - 1;
            --round;
          }
          (void)mbar_wait_bounded(is_k ? kfull(s) : vfull(s), round & 1);
        }
      }
    } else if (warp == kSoftWarps + 2) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idS = idesc_f8(128, NS, 0, 0);
      constexpr uint32_t idPV = idesc_f8(D, NP, 1, 1);
      const bool leader = elect_one();
      // K, Q and V rows of 128 bytes with the 128-byte swizzle, or of 64 with the 64-byte one (V
      // MN-major: the stride leads from 8 positions to the next 8); P MN-major, rows of 128 bytes
      const uint64_t dKQV = smem_desc(0, 16, 8 * D, D == 128 ? 2 : 4);
      const uint64_t dP = smem_desc(0, 16384, 1024, 2);
      auto with_addr = [](uint64_t d, uint32_t a16) { return d | uint64_t(a16 & 0x3FFFu); };
      const uint32_t qb = (sbase + Cfg::kOffQ) >> 4;
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
      };
      int vs = 0, vround = 0;
      // PV of the CTA's tile it (first: its group's first tile of the unit)
      auto issue_pv = [&](uint32_t it, bool first) -> bool {
        const int gg = it & 1;
        if (!wait_all(vfull(vs), vround & 1)) return false;
        if (!wait_all(pready(gg), (it >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t vb = (sbase + Cfg::kOffV + vs * Cfg::kTile) >> 4;
        const uint32_t pb = (sbase + Cfg::kOffP + gg * Cfg::kP) >> 4;
        if (leader) {
          constexpr int Passes = kSideP ? 1 : 3;
#pragma unroll
          for (int j = 0; j < 4 * Passes; ++j)   // 32 positions an MMA
            tc_mma_f8(tmem + 2 * Cfg::kSCol + Cfg::kOCol * gg, with_addr(dKQV, vb + (j & 3) * 2 * D),
                      with_addr(dP, pb + (j >> 2) * 1024 + (j & 3) * 256), idPV, !first || j > 0);
          tc_commit(pvdone(gg));
          tc_commit(vfree(vs));
        }
        __syncwarp();
        if (++vs == VS) {
          vs = 0;
          ++vround;
        }
        return true;
      };
      Place at = start;
      uint32_t it = 0;
      int s = 0, round = 0, seg = 0;
      for (int tiles = at.here(); tiles > 0 && ok; tiles = at.here()) {
        if (!wait_all(qready, seg++ & 1)) {
          ok = false;
          break;
        }
        auto issue_s = [&]() {
          const int gg = it & 1;
          const uint32_t kb = (sbase + s * Cfg::kTile) >> 4;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int j = 0; j < Cfg::kPasses * (D / 32); ++j) {
              const int pass = j / (D / 32), ks = j % (D / 32);
              tc_mma_f8(tmem + Cfg::kSCol * gg, with_addr(dKQV, kb + 2 * ks),
                        with_addr(dKQV, qb + pass * (Cfg::kQ / 16) + 2 * ks), idS, j > 0);
            }
            tc_commit(sfull(gg));
            tc_commit(kfree(s));
          }
          __syncwarp();
          if (++s == KS) {
            s = 0;
            ++round;
          }
        };
        for (int t = 0; t < tiles && ok; ++t, ++it) {
          // S of tile t overwrites that of tile t - 2, whose P (if of this unit) waits for its PV.  S
          // goes first when its K tile is there: the group waits for nothing else.
          if (it >= 2 && !wait_all(sread(it & 1), ((it >> 1) - 1) & 1)) { ok = false; break; }
          const bool early = __all_sync(0xffffffffu, mbar_test(kfull(s), round & 1));
          if (early) issue_s();
          if (t >= 2 && !issue_pv(it - 2, t - 2 < 2)) { ok = false; break; }
          if (!early) {
            if (!wait_all(kfull(s), round & 1)) { ok = false; break; }
            issue_s();
          }
        }
        // the unit's last PVs, before the next unit's queries are waited for
        if (ok && tiles >= 2 && !issue_pv(it - 2, tiles - 2 < 2)) ok = false;
        if (ok && !issue_pv(it - 1, tiles - 1 < 2)) ok = false;
        next_unit(at, tiles);
      }
      if (!ok && leader) set_error(p.err, kErrDeviceTimeout);
      // every MMA issued has completed before tensor memory is released
      if (leader) tc_commit(drain);
      __syncwarp();
      (void)mbar_wait_bounded(drain, 0);
    }
  } else {
    take_registers<216>();
    // ------------------------------------------------------------ softmax groups
    const int grp = warp >> 2;                // 0: even tiles, 1: odd tiles
    const int q4 = warp & 3;                  // tensor-memory lane quarter of this warp
    const int i = 32 * q4 + lane;             // tile position owned
    // head dimension owned: M = 64 puts 16 rows in each quarter of the lanes
    const int dim = D == 128 ? i : lane < 16 ? 16 * q4 + lane : -1;
    const uint32_t tl = tmem + (uint32_t(32 * q4) << 16);
    const uint32_t s_col = Cfg::kSCol * grp, o_col = 2 * Cfg::kSCol + Cfg::kOCol * grp;
    // Column references r (P = 2^(z - r)) are kept as -r in shared memory, up to 32 columns in
    // registers too; 0 while `hollow` says that the column has seen no unmasked logit.
    constexpr bool kSmemRef = NQC > 32;
    constexpr int QPER = (NQC + kSoftWarps - 1) / kSoftWarps;
    uint8_t* qs = smem + Cfg::kOffQ;
    // Element (n, k) of a query part: n * D + the 16-byte chunk k / 16 swizzled with the row.
    auto qoff = [](int n2, int k) {
      const int c = k >> 4, sw = D == 128 ? n2 & 7 : (n2 >> 1) & 3;
      return n2 * D + ((c ^ sw) << 4) + (k & 15);
    };
    const __nv_bfloat16* qbase = reinterpret_cast<const __nv_bfloat16*>(p.q);
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out);
    float* nrg = nrefs + grp * NQC;
    // (pages outside the pool: the producers record and clamp them)
    // (volatile: the compiler may not move the loads down to their uses)
    auto load_page = [&](const int32_t* row, int last, int t) {
      int v;
      asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(row + min(8 * t + (i >> 4), last)));
      return v;
    };
    auto load_scale = [&](const uint8_t* scales, int phys) {   // scales: of the unit's KV head
      uint32_t v;
      const uint32_t block = uint32_t(uint32_t(phys) < uint32_t(p.num_pages) ? phys : 0) * p.hkv;
      asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(scales + block));
      return v;
    };
    // group gg's O^T of columns 4 c .. 4 c + 3, part by part: there after a wait
    auto load_o = [&](int gg, int c, float (&v)[Cfg::kParts][4]) {
      const uint32_t at = tl + 2 * Cfg::kSCol + Cfg::kOCol * gg + 4 * c;
#pragma unroll
      for (int part = 0; part < Cfg::kParts; ++part) tmem_ld4(at + part * Cfg::PS, v[part]);
    };
    // S of all columns in pairs, the parts added
    auto load_all = [&](uint32_t at, uint64_t (&y2)[NQC / 2]) {
      constexpr int kFirst = NQC < 32 ? NQC : 32, kRest = NQC > 32 ? NQC - 32 : 8;
      if constexpr (kSideS) {
        uint64_t low[16];
        tmem_ld_pairs<kFirst>(at, y2, at + NQC, low);
#pragma unroll
        for (int j = 0; j < kFirst / 2; ++j) y2[j] = add_f32x2(y2[j], low[j]);
        if constexpr (NQC > 32) {
          tmem_ld_pairs<kRest>(at + 32, y2 + 16, at + NQC + 32, low);
#pragma unroll
          for (int j = 0; j < kRest / 2; ++j) y2[16 + j] = add_f32x2(y2[16 + j], low[j]);
        }
      } else {   // (more than 40 columns)
        tmem_ld_pairs<kRest>(at, y2, at + kRest, y2 + kRest / 2);
        if constexpr (NQC - 2 * kRest > 0)
          tmem_ld_pairs<NQC - 2 * kRest>(at + 2 * kRest, y2 + kRest);
      }
    };

    Place at = start;
    long long unit0 = base + (long long)start.g * (start.tiles + kUnitTiles);   // its span's begin
    uint32_t it0 = 0;             // the CTA's tile with which the unit begins
    // A unit's first requests: its queries, and the table entries of this thread's position in the
    // group's first two tiles.  Up to 32 columns they are made under the end of the unit before (256 x 100:
    // 73.9 -> 71.4 us, 64 x 4000 99.8 -> 98.5; with 56 columns they cost registers, 4 x 128K 195 -> 202).
    constexpr bool kAhead = !kSmemRef;
    uint32_t qnext[kAhead ? QPER : 1][D / 64];
    int pnext[2];
    // (from: the CTA's tile with which the unit begins)
    auto request = [&](const Place& u, uint32_t from, uint32_t (*q)[D / 64], int* pages) {
      const int32_t* row = p.block_table + size_t(u.b) * p.max_pages;
      const int last_page = (u.L + p.gamma) >> 4, t0 = u.t + int((from ^ uint32_t(grp)) & 1);
      pages[0] = load_page(row, last_page, t0);
      pages[1] = load_page(row, last_page, t0 + 2);
      const __nv_bfloat16* qunit = qbase + (size_t(u.b) * T * p.hq + u.g * p.group) * D;
#pragma unroll
      for (int k = 0; k < QPER; ++k) {
        const int n2 = warp + kSoftWarps * k;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint32_t* from_row = reinterpret_cast<const uint32_t*>(qunit + rowat[n2]) + 32 * h + lane;
          q[k][h] = 0;
          if constexpr (kAhead) {   // (volatile: asked for here)
            if (n2 < p.nq) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(q[k][h]) : "l"(from_row));
          } else {
            if (n2 < p.nq) q[k][h] = *from_row;
          }
        }
      }
    };
    if (kAhead && at.here() > 0) request(at, 0, qnext, pnext);
    for (int tiles = at.here(); tiles > 0; tiles = at.here()) {
      const int L = at.L, g = at.g, b = at.b;
      const int32_t* row = p.block_table + size_t(b) * p.max_pages;
      const int last_page = (L + p.gamma) >> 4;
      const uint8_t *k_scales = p.k_scale + g, *v_scales = p.v_scale + g;
      const uint32_t first = it0 + ((it0 ^ uint32_t(grp)) & 1);   // this group's first tile

      // ---------------------------------------------------------- the unit's queries
      int phys1 = 0;
      uint32_t ekb, evb;
      {
        uint32_t qreg[QPER][D / 64];
        int pages[2];
        if constexpr (kAhead) {
          pages[0] = pnext[0];
          pages[1] = pnext[1];
#pragma unroll
          for (int u = 0; u < QPER; ++u)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) qreg[u][h] = qnext[u][h];
        } else {
          request(at, it0, qreg, pages);
        }
        const int phys0 = pages[0];
        phys1 = pages[1];
        // a row's exponent: its largest element lies in [2^n, 2^(n + 1))
#pragma unroll
        for (int u = 0; u < QPER; ++u) {
          uint32_t most = 0;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) most = __vmaxu2(most, qreg[u][h] & 0x7fff7fffu);
          most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
          if (lane == 0 && warp + kSoftWarps * u < NQC)
            rowexp[warp + kSoftWarps * u] = most ? max(-100, int(most >> 7) - 127) : -1000;
        }
        ekb = load_scale(k_scales, phys0);
        evb = load_scale(v_scales, phys0);
        if (CAPTURE) {
          // the captured query, summed over its rows and heads: this warp's rows
          float acc[D / 64][2] = {};
#pragma unroll
          for (int u = 0; u < QPER; ++u) {
            const int n2 = warp + kSoftWarps * u;
            if (n2 < p.nq && ((p.row_mask >> tlim[n2]) & 1u)) {
#pragma unroll
              for (int h = 0; h < D / 64; ++h) {
                acc[h][0] += __uint_as_float(qreg[u][h] << 16);
                acc[h][1] += __uint_as_float(qreg[u][h] & 0xffff0000u);
              }
            }
          }
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<float2*>(qsum + warp * D + 64 * h + 2 * lane) =
                make_float2(acc[h][0], acc[h][1]);
        }
        named_bar(kAllBar, kSoft);
        // One exponent for all rows while they are within 2^4 of each other (a part's grid then
        // reaches 2^-13 of the smallest row's largest element, and 2^-17 of the unit's), else one a
        // row.
        int most = -1000, least = 1000;
        for (int n2 = lane; n2 < NQC; n2 += 32) {
          const int e = rowexp[n2];
          most = max(most, e);
          if (e > -1000) least = min(least, e);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        const bool one = most - least <= 4;
        if (most == -1000) most = 0;
        // The next e4m3 part of (x0, x1), |x| < 2^8, to row n2 of a pass; x keeps the rest.
        auto put_part = [&](int pass, int n2, int k, float& x0, float& x1) {
          const uint32_t c = e4m3x2_from_f32(x0, x1);
          *reinterpret_cast<uint16_t*>(qs + pass * Cfg::kQ + qoff(n2, k)) = uint16_t(c);
          uint32_t h, unused;
          f16x2_from_e4m3x4(c, h, unused);
          const float2 v = f32x2_from_f16x2(h);
          x0 -= v.x;
          x1 -= v.y;
        };
#pragma unroll
        for (int u = 0; u < QPER; ++u) {
          const int n2 = warp + kSoftWarps * u;
          if (n2 >= NQC) continue;
          const int e = rowexp[n2], k = 7 - (one ? most : e == -1000 ? 0 : e);
          const float f = two_to(k);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            float x0 = __uint_as_float(qreg[u][h] << 16) * f;
            float x1 = __uint_as_float(qreg[u][h] & 0xffff0000u) * f;
            put_part(0, n2, 64 * h + 2 * lane, x0, x1);
            put_part(kSideS ? 0 : 1, kSideS ? NQC + n2 : n2, 64 * h + 2 * lane, x0, x1);
          }
          if (lane == 0) colfac[n2] = one ? 1.f : two_to(-k);
        }
        if (CAPTURE && warp == 7) {
          float x[D / 64][2];
          float top = 0.f;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kSoftWarps; ++j) {
              const float2 w = *reinterpret_cast<const float2*>(qsum + j * D + 64 * h + 2 * lane);
              v.x += w.x;
              v.y += w.y;
            }
            x[h][0] = v.x;
            x[h][1] = v.y;
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
          const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
          const int k = 7 - max(-100, int(bits >> 23) - 127);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            float x0 = x[h][0] * two_to(k), x1 = x[h][1] * two_to(k);
#pragma unroll
            for (int j = 0; j < kCapParts; ++j) {
              put_part(kSideS ? 0 : j & 1, Cfg::kCap0 + (kSideS ? j : j >> 1), 64 * h + 2 * lane, x0, x1);
              if (j & 1) {   // two parts leave less than 2^-8 of the largest: the next start 2^8 lower
                x0 *= 256.f;
                x1 *= 256.f;
              }
            }
          }
          if (lane == 0) *capexp = -k;
        }
        if (warp == 6) {   // rows that fill up N
          constexpr int row = Cfg::kCap0 + Cfg::kCap;
          for (int j = lane; j < (NS - row) * D / 4; j += 32)
#pragma unroll
            for (int pass = 0; pass < Cfg::kPasses; ++pass)
              reinterpret_cast<uint32_t*>(qs + pass * Cfg::kQ + row * D)[j] = 0;
          if (lane == 0) *uniform = one ? most - 7 : kMixed;
        }
        if (i < NQC) nrg[i] = 0.f;
        // Generic-proxy writes of Q must be visible to the tensor cores (async proxy).
        fence_proxy_async_smem();
        mbar_arrive(qready);
        named_bar(kAllBar, kSoft);   // (what was written above is read by all)
      }

      // ---------------------------------------------------------- its tiles
      uint64_t nr2[kSmemRef ? 1 : NQC / 2];
      uint64_t ls2[NQC / 2];   // row sums
#pragma unroll
      for (int c = 0; c < NQC / 2; ++c) {
        if constexpr (!kSmemRef) nr2[c] = 0;
        ls2[c] = 0;
      }
      uint64_t hollow = NQC == 64 ? ~0ull : (1ull << NQC) - 1;   // columns without a reference
      const int uni = *uniform;
      const bool mixed = uni == kMixed;
      const float scale0 = mixed ? p.scale_log2 : p.scale_log2 * two_to(uni);
      const float cap_scale = CAPTURE ? p.scale * two_to(*capexp) : 0.f;
      float* srow = CAPTURE ? p.scores + (size_t(b) * p.hkv + g) * p.score_stride : nullptr;
      int Lcap = L;
      if (CAPTURE && L > p.score_stride) {
        if (tid == 0) set_error(p.err, kErrDeviceFault);
        Lcap = p.score_stride;
      }
      bool any = false;   // this group has a tile of the unit
      // A failed (timed-out) wait is carried to the group vote below, so the 128
      // threads of a group always leave the loop together.
      for (uint32_t it = first; it < it0 + uint32_t(tiles); it += 2) {
        const uint32_t k = it >> 1;
        const int t = at.t + int(it - it0);
        const int pos = 128 * t + i;
        // this position's scales (the next tile's are requested below)
        const int e_k = kv8_exponent(uint8_t(ekb)), e_v = kv8_exponent(uint8_t(evb));
        const bool deep = e_v < kKv8Deep;   // (its part of the row sums is made beside a raise, not from P)
        const float f_k = two_to(e_k), un = deep ? 0.f : two_to(-e_v), f = scale0 * f_k, add = float(e_v);
        const uint64_t f2 = pair_f32(f, f), add2 = pair_f32(add, add), un2 = pair_f32(un, un);
        // (wide: half of the references come to registers while S is on its way, the other half under
        // the first one's arithmetic; all of them do not fit)
        constexpr int kPre = kSmemRef ? NQC / 4 : 1;   // pairs
        uint64_t pre[kPre];
        auto load_refs = [&](int from) {
#pragma unroll
          for (int c = 0; c < kPre; c += 2) {
            const ulonglong2 r = reinterpret_cast<const ulonglong2*>(nrg)[(from + c) / 2];
            pre[c] = r.x;
            pre[c + 1] = r.y;
          }
        };
        if constexpr (kSmemRef) load_refs(0);
        bool okt = ok && mbar_wait_bounded(sfull(grp), k & 1);
        tc_fence_after();
        // z of all columns less their references, two to a register pair
        uint64_t y2[NQC / 2];
        float cx[8] = {};   // the capture columns
        bool left = false, need = hollow != 0 || deep;
        if (okt) {
          if constexpr (CAPTURE) tmem_ld8(tl + s_col + Cfg::kCap0, cx);
          load_all(tl + s_col, y2);   // (waits for both)
          if constexpr (CAPTURE) {
            loaded<Cfg::kCap>(cx);
            if constexpr (kSideS) {
#pragma unroll
              for (int j = 0; j < 3; ++j) cx[j] = cx[2 * j] + cx[2 * j + 1];
            }
          }
          if (mixed) {
#pragma unroll
            for (int c = 0; c < NQC / 2; ++c)
              y2[c] = mul_f32x2(y2[c], reinterpret_cast<const uint64_t*>(colfac)[c]);
          }
#pragma unroll
          for (int c = 0; c < NQC / 2; ++c) {
            if (kSmemRef && c == NQC / 4) load_refs(NQC / 4);
            y2[c] = add_f32x2(fma_f32x2(y2[c], f2, add2), kSmemRef ? pre[kSmemRef ? c % kPre : 0] : nr2[kSmemRef ? 0 : c]);
          }
          if (pos > L) {   // window positions that a row may not see yet, and what lies behind them
#pragma unroll
            for (int c = 0; c < NQC / 2; ++c) {
              float a, d;
              unpair_f32(y2[c], a, d);
              y2[c] = pair_f32(pos > L + tlim[2 * c] ? -INFINITY : a,
                               pos > L + tlim[2 * c + 1] ? -INFINITY : d);
            }
          }
          float ym[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < NQC / 2; ++c) {
            float a, d;
            unpair_f32(y2[c], a, d);
            ym[c & 1] = fmaxf(fmaxf(ym[c & 1], a), d);
          }
          need |= fmaxf(ym[0], ym[1]) > kTop;
        }
        // PV of the group's last tile is done with P's buffer, and with O^T
        okt = okt && (it < 2 || mbar_wait_bounded(pvdone(grp), (k - 1) & 1));
        const bool all_ok = __all_sync(0xffffffffu, okt);
        if (lane == 0) votes[(k & 1) * 8 + grp * 4 + q4] = all_ok ? 0 : 1;
        const bool agreed = named_bar_any(1 + grp, 128, need || !okt);
        const int* vt = votes + (k & 1) * 8 + grp * 4;
        if (agreed) left = vt[0] | vt[1] | vt[2] | vt[3];
        if (agreed && !left) {
          // Raise: column maxima over the group's 128 positions
          tc_fence_after();
          float* cm = colmax + grp * 4 * NQC;
#pragma unroll
          for (int c = 0; c < NQC / 8; ++c) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) unpair_f32(y2[4 * c + e / 2], v[e], v[e + 1]);
            const float top = reduce_chunk(v, [](float a, float d) { return fmaxf(a, d); });
            if ((lane & 3) == 0) cm[q4 * NQC + 8 * c + (lane >> 2)] = top;
          }
          named_bar(1 + grp, 128);
          // a column's new reference, at least kRaise below its largest z (cm is relative to the old
          // one), and the factor that its sums take
          if (i < NQC) {
            const float nro = nrg[i];
            const float top = fmaxf(fmaxf(cm[i], cm[NQC + i]), fmaxf(cm[2 * NQC + i], cm[3 * NQC + i]));
            const float old = ((hollow >> i) & 1) ? kEmptyMax : -nro;
            const float now = fmaxf(old, top - nro - kRaise);
            facs[grp * NQC + i] = half_weight(old - now);
            nrg[i] = now == kEmptyMax ? 0.f : -now;
            cm[i] = now;   // (its own column: read above by this thread alone)
            cm[NQC + i] = nrg[i] - nro;   // what its logits take
          }
          named_bar(1 + grp, 128);
          // (columns with masked logits only stay without one until the next tile)
          hollow = __ballot_sync(0xffffffffu, lane < NQC && cm[lane] == kEmptyMax);
          if constexpr (NQC > 32)
            hollow |= uint64_t(__ballot_sync(0xffffffffu, lane + 32 < NQC && cm[lane + 32] == kEmptyMax))
                      << 32;
          const float4* fc = reinterpret_cast<const float4*>(facs + grp * NQC);
#pragma unroll
          for (int c = 0; c < NQC / 4; ++c) {
            const float4 v = fc[c];
            const uint64_t xy = pair_f32(v.x, v.y), zw = pair_f32(v.z, v.w);
            ls2[2 * c] = mul_f32x2(mul_f32x2(ls2[2 * c], xy), xy);
            ls2[2 * c + 1] = mul_f32x2(mul_f32x2(ls2[2 * c + 1], zw), zw);
            if constexpr (!kSmemRef) {
              const ulonglong2 r = reinterpret_cast<const ulonglong2*>(nrg)[c];
              nr2[2 * c] = r.x;
              nr2[2 * c + 1] = r.y;
            }
          }
          const ulonglong2* moved = reinterpret_cast<const ulonglong2*>(cm + NQC);
#pragma unroll
          for (int c = 0; c < NQC / 4; ++c) {
            const ulonglong2 r = moved[c];
            y2[2 * c] = add_f32x2(y2[2 * c], r.x);
            y2[2 * c + 1] = add_f32x2(y2[2 * c + 1], r.y);
          }
          if (__any_sync(0xffffffffu, deep)) {
            const float lifted = deep ? two_to(-e_v - kKv8Lift) : 0.f;
#pragma unroll
            for (int c = 0; c < NQC / 2; ++c) add_lifted(ls2[c], y2[c], lifted);
          }
          if (any) {
#pragma unroll 1
            for (int c = 0; c < NQC / 8; ++c) {
              float4 a = fc[2 * c], d = fc[2 * c + 1];
              a = make_float4(a.x * a.x, a.y * a.y, a.z * a.z, a.w * a.w);
              d = make_float4(d.x * d.x, d.y * d.y, d.z * d.z, d.w * d.w);
#pragma unroll
              for (int part = 0; part < Cfg::kParts; ++part) {
                float v8[8];
                tmem_ld8(tl + o_col + part * Cfg::PS + 8 * c, v8);
                tmem_ld_wait();
                loaded(v8);
                v8[0] *= a.x;
                v8[1] *= a.y;
                v8[2] *= a.z;
                v8[3] *= a.w;
                v8[4] *= d.x;
                v8[5] *= d.y;
                v8[6] *= d.z;
                v8[7] *= d.w;
                tmem_st8(tl + o_col + part * Cfg::PS + 8 * c, v8);
              }
            }
            tmem_st_wait();
          }
          named_bar(1 + grp, 128);   // colmax and the factors are read
        }
        if (left) {
          ok = false;
          break;
        }
        tc_fence_before();
        // the next tile's scales and the page after that, behind the vote: ahead of it they were in the way
        // of the logits (4 x 128K of 64: 207 -> 202 us)
        ekb = load_scale(k_scales, phys1);
        evb = load_scale(v_scales, phys1);
        phys1 = load_page(row, last_page, t + 4);
        mbar_arrive(sread(grp));   // S of the group's next tile may come
        if (CAPTURE && pos < Lcap) {
          srow[pos] = fmaf(fmaf(cx[2], 0x1p-8f, cx[1]), 0x1p-8f, cx[0]) * (f_k * cap_scale);
        }
        // P = 2^y in three e5m2 parts (upper bytes of f16: cut, cut, rounded), eight columns of a part in
        // eight bytes of position i's row, 16-byte chunks swizzled (columns that fill up N are never
        // read; their P may be anything)
        uint8_t* prow = smem + Cfg::kOffP + grp * Cfg::kP + i * 128;
        // (a step for all columns before the next: one column's steps are a chain of 70 clocks)
        uint32_t x[NQC / 2];
#pragma unroll
        for (int j = 0; j < NQC / 2; ++j) {
          float p0, p1;
          unpair_f32(y2[j], p0, p1);
          y2[j] = pair_f32(ex2(p0), ex2(p1));
        }
#pragma unroll
        for (int j = 0; j < NQC / 2; ++j) {
          float p0, p1;
          unpair_f32(y2[j], p0, p1);
          ls2[j] = fma_f32x2(y2[j], un2, ls2[j]);
          x[j] = pack_f16x2(p0, p1);
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          if (part == 2) {
#pragma unroll
            for (int j = 0; j < NQC / 2; ++j)
              x[j] += 0x00800080u;   // (finite, >= 0: a carry rounds up)
          }
          auto code = [&](int j) { return __byte_perm(x[j], x[j + 1], 0x7531); };
#pragma unroll
          for (int c = 0; c < NQC / 8; ++c) {
            const int byte = part * Cfg::PS + 8 * c;
            uint8_t* at16 = prow + (byte >> 7) * 16384 + ((((byte & 127) >> 4) ^ (i & 7)) << 4);
            if (Cfg::PS % 16 == 0 && c % 2 == 0 && c + 1 < NQC / 8)   // (no bank twice in a phase)
              *reinterpret_cast<uint4*>(at16) =
                  make_uint4(code(4 * c), code(4 * c + 2), code(4 * c + 4), code(4 * c + 6));
            else if (Cfg::PS % 16 != 0 || c % 2 == 0)
              *reinterpret_cast<uint2*>(at16 + (byte & 8)) = make_uint2(code(4 * c), code(4 * c + 2));
          }
          if (part < 2) {
#pragma unroll
            for (int j = 0; j < NQC / 2; ++j)
              x[j] = sub_f16x2(x[j], x[j] & 0xff00ff00u);
          }
        }
        if (pos > L + p.gamma) {
          // a cache slot behind the window: zero its V row, whose codes may be NaN
          const uint32_t vs = it % VS;
          if (mbar_wait_bounded(vfull(vs), (it / VS) & 1)) {
            uint4* vrow = reinterpret_cast<uint4*>(smem + Cfg::kOffV + vs * Cfg::kTile + i * D);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) vrow[c] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(pready(grp));
        any = true;
      }

      // ---------------------------------------------------------- the unit's end
      // row sums over the group's 128 positions
#pragma unroll
      for (int c = 0; c < NQC / 8; ++c) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) unpair_f32(ls2[4 * c + e / 2], v[e], v[e + 1]);
        const float sum = reduce_chunk(v, [](float a, float d) { return a + d; });
        if ((lane & 3) == 0) colsum[(grp * 4 + q4) * NQC + 8 * c + (lane >> 2)] = sum;
      }
      [[maybe_unused]] Place next;
      if constexpr (kAhead) {
        next = at;
        next_unit(next, tiles);
        if (next.here() > 0) request(next, it0 + uint32_t(tiles), qnext, pnext);
      }
      // The group's last PV completes its O^T.
      if (any && ok) {
        const uint32_t last = it0 + uint32_t(tiles) - 1 - ((it0 + uint32_t(tiles) - 1 - uint32_t(grp)) & 1);
        if (!mbar_wait_bounded(pvdone(grp), (last >> 1) & 1)) ok = false;
      }
      tc_fence_after();
      if (i < NQC) colmax[grp * 4 * NQC + i] = ((hollow >> i) & 1) ? kEmptyMax : -nrg[i];
      tc_fence_before();
      if (named_bar_any(kAllBar, kSoft, !ok)) {   // both groups leave together
        if (!ok && i == 0) set_error(p.err, kErrDeviceTimeout);
        break;
      }
      // the CTAs that hold tiles of the unit
      const long long tile0 = unit0 + kUnitTiles;
      const int c0 = cta_of(tile0), c1 = cta_of(tile0 + at.tiles - 1);
      // the piece's maximum and sum of a column, and the weights of the two groups' states
      if (tid < NQC) {
        const float m0 = colmax[tid], m1 = colmax[4 * NQC + tid], M = fmaxf(m0, m1);
        const float h0 = half_weight(m0 - M), h1 = half_weight(m1 - M), w0 = h0 * h0, w1 = h1 * h1;
        const float* cs = colsum + tid;
        const float sum = (cs[0] + cs[NQC] + cs[2 * NQC] + cs[3 * NQC]) * h0 * h0 +
                          (cs[4 * NQC] + cs[5 * NQC] + cs[6 * NQC] + cs[7 * NQC]) * h1 * h1;
        const float share = c0 == c1 ? 1.f / sum : 1.f;   // (a whole unit is divided by its sums here)
        wgt[tid] = w0 * share;
        wgt[NQC + tid] = w1 * share;
        colM[tid] = M;
        colL[tid] = sum;
      }
      // groups with a tile of the unit
      const bool has0 = tiles > 1 || !(it0 & 1), has1 = tiles > 1 || (it0 & 1);
      named_bar(kAllBar, kSoft);
      tc_fence_after();   // (the other group's PVs are done: its threads waited, above)
      __nv_bfloat16* ounit = out + (size_t(b) * T * p.hq + g * p.group) * D;
      // Workspace slots: 2 c for the unit that CTA c's run begins in or with, 2 c + 1 for its last one
      // where that is another; of a unit's CTAs only the first can have it as its last.  So a CTA is the
      // first of one shared unit at most, whose ticket is tickets[c0].
      const int slot0 = 2 * c0 + (run_begin(c0) >= unit0 ? 0 : 1);
      const size_t slot = cta == c0 ? slot0 : 2 * cta;
      float* part = p.part_o + (slot * p.nq + 4 * grp) * D + max(dim, 0);
      // each group finishes half of the columns, from both groups' O^T
#pragma unroll
      for (int c = grp; c < NQC / 4; c += 2) {
        float o0[Cfg::kParts][4] = {}, o1[Cfg::kParts][4] = {};
        if (has0) load_o(0, c, o0);
        if (has1) load_o(1, c, o1);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < Cfg::kParts; ++k) {
          loaded(o0[k]);
          loaded(o1[k]);
        }
        const float4 w0 = reinterpret_cast<const float4*>(wgt)[c];
        const float4 w1 = reinterpret_cast<const float4*>(wgt + NQC)[c];
        const int4 to = reinterpret_cast<const int4*>(rowat)[c];
        const float f0[4] = {w0.x, w0.y, w0.z, w0.w}, f1[4] = {w1.x, w1.y, w1.z, w1.w};
        const int row_at[4] = {to.x, to.y, to.z, to.w};
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float a = o0[0][e], d = o1[0][e];
#pragma unroll
          for (int k = 1; k < Cfg::kParts; ++k) {
            a += o0[k][e];
            d += o1[k][e];
          }
          v[e] = a * f0[e] + d * f1[e];
        }
        const int here = dim < 0 ? 0 : p.nq - 4 * c;   // columns of the four that there are
        if (c0 == c1) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < here) ounit[row_at[e] + dim] = __float2bfloat16_rn(v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < here) part[e * D] = v[e];
          part += 8 * D;
        }
      }
      tc_fence_before();
      if (c0 != c1 && tid < p.nq)
        reinterpret_cast<float2*>(p.part_ml)[slot * p.nq + tid] = make_float2(colM[tid], colL[tid]);
      if (c0 != c1) {
        named_bar(kAllBar, kSoft);
        // (released and acquired by one thread: the barriers carry that to and from the others)
        if (tid == 0) *flag = ticket_acq_rel(&p.tickets[c0]) == c1 - c0;
        named_bar(kAllBar, kSoft);
        if (*flag) {
          // Last to arrive: out = sum_c F_c o_c / sum_c F_c l_c with F_c = 2^(m_c - max m), in one pass
          // over the pieces with the running maximum.  All of a thread's elements have their loads in
          // flight together.
          const int pieces = c1 - c0 + 1;
          const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
          constexpr int E = (NQC * (D / 4) + kSoft - 1) / kSoft;
          float M[E], sum[E];
          float4 acc[E];
#pragma unroll
          for (int j = 0; j < E; ++j) {
            M[j] = kEmptyMax;
            sum[j] = 0.f;
            acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll 4
          for (int c = 0; c < pieces; ++c) {
            const size_t rows = size_t(c == 0 ? slot0 : 2 * (c0 + c)) * p.nq;
            float2 m[E];
            float4 v[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
              const int e = tid + kSoft * j, n2 = min(e / (D / 4), p.nq - 1);
              m[j] = __ldcg(ml + rows + n2);
              v[j] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (rows + n2) * D) + e % (D / 4));
            }
#pragma unroll
            for (int j = 0; j < E; ++j) {
              const float d = M[j] - m[j].x, h = half_weight(-fabsf(d));
              const bool up = d < 0.f;
              const float a = up ? h * h : 1.f, w = up ? 1.f : h * h;
              M[j] = fmaxf(M[j], m[j].x);
              sum[j] = up ? fmaf(sum[j] * h, h, m[j].y) : fmaf(m[j].y * h, h, sum[j]);
              acc[j].x = acc[j].x * a + w * v[j].x;
              acc[j].y = acc[j].y * a + w * v[j].y;
              acc[j].z = acc[j].z * a + w * v[j].z;
              acc[j].w = acc[j].w * a + w * v[j].w;
            }
          }
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const int e = tid + kSoft * j, n2 = e / (D / 4);
            if (n2 >= p.nq) continue;
            const float inv = 1.f / sum[j];
            reinterpret_cast<uint2*>(ounit + rowat[n2])[e % (D / 4)] =
                make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv),
                           pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
          }
          if (tid == 0) p.tickets[c0] = 0;
        }
      }
      named_bar(kAllBar, kSoft);   // the buffers and columns are free again
      unit0 += at.tiles + kUnitTiles;
      it0 += uint32_t(tiles);
      if constexpr (kAhead)
        at = next;
      else
        next_unit(at, tiles);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 2) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

template <int D, int NQC, bool CAP>
static cudaError_t launch_one(const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const VerifyKv8Params& p, int grid, cudaStream_t stream) {
  using Cfg = Kv8Cfg<D, NQC, CAP>;
  static std::atomic<uint32_t> configured{0};
  cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(verify_kv8_kernel<D, NQC, CAP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::kSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kv8_kernel<D, NQC, CAP>, kmap, vmap, p);
}

// The softmax's columns: nq rounded up to 8.
template <int D, bool CAP>
static cudaError_t launch_cols(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const VerifyKv8Params& p, int grid, cudaStream_t s) {
  if (!verify_kv8_supported(D, p.nq)) return cudaErrorInvalidValue;
  switch ((p.nq + 7) / 8) {
    case 1: return launch_one<D, 8, CAP>(kmap, vmap, p, grid, s);
    case 2: return launch_one<D, 16, CAP>(kmap, vmap, p, grid, s);
    case 3: return launch_one<D, 24, CAP>(kmap, vmap, p, grid, s);
    case 4: return launch_one<D, 32, CAP>(kmap, vmap, p, grid, s);
    case 5: return launch_one<D, 40, CAP>(kmap, vmap, p, grid, s);
  }
  if constexpr (D == 64) {
    switch ((p.nq + 7) / 8) {
      case 6: return launch_one<D, 48, CAP>(kmap, vmap, p, grid, s);
      case 7: return launch_one<D, 56, CAP>(kmap, vmap, p, grid, s);
      case 8: return launch_one<D, 64, CAP>(kmap, vmap, p, grid, s);
    }
  }
  return cudaErrorInvalidValue;
}

#define VEGAS_CAT2(a, b) a##b
#define VEGAS_CAT(a, b) VEGAS_CAT2(a, b)

cudaError_t VEGAS_CAT(launch_verify_kv8_d, VEGAS_KV8_D)(const CUtensorMap& kmap,
                                                       const CUtensorMap& vmap,
                                                       const VerifyKv8Params& p, bool capture,
                                                       int grid, cudaStream_t stream) {
  constexpr int D = VEGAS_KV8_D;
  return capture ? launch_cols<D, true>(kmap, vmap, p, grid, stream)
                 : launch_cols<D, false>(kmap, vmap, p, grid, stream);
}

}  // namespace vegas
