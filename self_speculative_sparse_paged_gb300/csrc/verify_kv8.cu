// Verify attention with captured scores over the 8-bit cache, on the 5th-generation tensor cores
// (compiled once per head_dim, VEGAS_KV8_D).
//
// Same work as verify_tc.cu with the roles arranged alike (three producer warps, one issuing
// warp, two softmax groups of four warps that alternate 128-position tiles and own a thread a
// position, the on-chip merge of the splits), on half the bytes:
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
//   O^T[D x N] += V'^T P^T   kind::f16, M = D: V' are V's codes as f16, exact; each thread of a
//       softmax group turns its own position's row (16 codes: one load, 8 conversions, two stores)
//       while the tensor cores still work on S of the tile.
//
// The two parts of the queries lie side by side in N (one pass over K; an MMA takes 45 clocks up
// to N = 64 and 64 at 128) up to 40 columns, else they share an accumulator.
// P <= 2^15 (f16 ends at 65504) and the largest P is 2^7 or more when r was raised, so P's grid
// reaches 2^-31 below the largest.  e_v spans 120, so that no term that weighs in a row sum is lost to
// fp32's smallest number (its P is at least 2^-121).
#include "cluster_merge.cuh"
#include "kv8.cuh"

#ifndef VEGAS_KV8_D
#error "compile with -DVEGAS_KV8_D=64 or -DVEGAS_KV8_D=128"
#endif

namespace vegas {

namespace {
constexpr float kTop = 15.f, kRaise = 7.f;   // log2 of the largest P, and of P at a raised reference
constexpr int kCapParts = 6;
constexpr int kMixed = 1000;   // (in place of the rows' common exponent) rows have their own

// Instruction descriptors, fp32 accumulator: e4m3 by e4m3, K-major (K = 32); f16 by f16,
// MN-major (K = 16).
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_mn(int m, int n) {
  return (1u << 4) | (1u << 15) | (1u << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Lane l gets op over the warp's lanes of their v[l]: in five steps a lane exchanges half of the
// columns it still holds for the other half of another lane's (31 shuffles for 32 columns).
template <class Op>
__device__ __forceinline__ float reduce_columns(float (&v)[32], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const bool upper = lane & w;
#pragma unroll
    for (int j = 0; j < w; ++j) {
      const float give = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
      v[j] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
    }
  }
  return v[0];
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
  static constexpr int NP = (NQC + 15) / 16 * 16;     // N of PV
  static constexpr int kTile = 128 * D;               // one K tile (and one V tile): 8 pages
  // Ring slots (16 KB at head_dim 128, 8 KB at 64): as many as fit beside the rest.
  static constexpr int KS = D == 64 ? 8 : 4;
  static constexpr int VS = D == 64 ? 8 : NQC <= 32 ? 4 : 3;
  static constexpr int kV16 = 128 * D * 2;            // a tile's V' [half][128][128 B], one a group
  static constexpr int kPRow = NQC <= 32 ? 64 : 128;  // bytes of a position's P row
  static constexpr int kP = 128 * kPRow;
  static constexpr int kQ = NS * D;                   // Q^T operand, one a pass
  static constexpr int kPasses = kSideS ? 1 : 2;
  static constexpr int kThreads = 384;
  static constexpr int kSCol = (NS + 31) / 32 * 32, kOCol = (NP + 31) / 32 * 32;
  static constexpr uint32_t kTmemCols =
      2 * (kSCol + kOCol) <= 128 ? 128 : 2 * (kSCol + kOCol) <= 256 ? 256 : 512;
  static_assert(2 * (kSCol + kOCol) <= 512, "tensor memory");
  static constexpr int kOffV = KS * kTile;
  static constexpr int kOffV16 = kOffV + VS * kTile;
  static constexpr int kOffP = kOffV16 + 2 * kV16;
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffBar = kOffQ + kPasses * kQ;
  static constexpr int kNumBars = 2 * KS + 2 * VS + 4 * 2 + 1;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
  // misc: tmem slot, flag, capture exponent, uniform flag; votes[2][2][4]; colmax[2][4][NQC],
  // colsum[2][4][NQC], col[NQC], nref[2][NQC]; tlim[NQC]; rowexp[NQC]
  static constexpr size_t kMisc = 16 + 64 + 4 * (16 * NQC + 3 * NQC + 2 * NQC);
  static constexpr size_t kSmem = size_t(kOffMisc) + kMisc + 1024;
  static constexpr int kMergeOff = (merge_receive_bytes<D, NQC>() + 1023) / 1024 * 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kMergeOff + kMergeWeightBytes <= kOffP, "merge areas");
  static_assert(8 * D * 4 <= kP, "partial sums of the captured query (P's buffer)");
};

template <int D, int NQC, bool CAPTURE>
__global__ void __launch_bounds__(384, 1)
    verify_kv8_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const VerifyParams p) {
  using Cfg = Kv8Cfg<D, NQC, CAPTURE>;
  constexpr int KS = Cfg::KS, VS = Cfg::VS, NS = Cfg::NS, NP = Cfg::NP;
  constexpr bool kSideS = Cfg::kSideS;
  static_assert(NQC % 8 == 0 && (D == 64 || D == 128), "columns, head_dim");

  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::kOffBar;
  // barriers: K full/free (per K slot), V full/free (per V slot); S full, S read, P and V'
  // ready, PV done (per softmax group); MMA drain
  auto kfull = [&](int s) { return bar0 + 8 * s; };
  auto kfree = [&](int s) { return bar0 + 8 * (KS + s); };
  auto vfull = [&](int s) { return bar0 + 8 * (2 * KS + s); };
  auto vfree = [&](int s) { return bar0 + 8 * (2 * KS + VS + s); };
  constexpr int B1 = 2 * KS + 2 * VS;
  auto sfull = [&](int g2) { return bar0 + 8 * (B1 + g2); };
  auto sread = [&](int g2) { return bar0 + 8 * (B1 + 2 + g2); };
  auto pready = [&](int g2) { return bar0 + 8 * (B1 + 4 + g2); };
  auto pvdone = [&](int g2) { return bar0 + 8 * (B1 + 6 + g2); };
  const uint32_t drain = bar0 + 8 * (B1 + 8);
  uint8_t* misc = smem + Cfg::kOffMisc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  int* flag = reinterpret_cast<int*>(misc + 4);
  int* capexp = reinterpret_cast<int*>(misc + 8);
  int* uniform = reinterpret_cast<int*>(misc + 12);
  int* votes = reinterpret_cast<int*>(misc + 16);                // [2][2][4]
  float* colmax = reinterpret_cast<float*>(misc + 80);           // [2][4][NQC]
  float* colsum = colmax + 8 * NQC;                              // [2][4][NQC]
  float* colfac = colsum + 8 * NQC;                              // [NQC] scale log2(e) 2^-k
  float* nrefs = colfac + NQC;                                   // [2][NQC] -reference
  int* tlim = reinterpret_cast<int*>(nrefs + 2 * NQC);           // [NQC]
  int* rowexp = tlim + NQC;                                      // [NQC]
  float* qsum = reinterpret_cast<float*>(smem + Cfg::kOffP);     // [8][D] parts of the captured sum

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int unit = b * p.hkv + g;
  const int T = p.gamma + 1;
  const int cap = p.max_pages * 16;

  if (tid == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(kfull(s), 1);
      mbar_init(kfree(s), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(vfull(s), 1);
      mbar_init(vfree(s), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull(i), 1);
      mbar_init(sread(i), 128);
      mbar_init(pready(i), 128);
      mbar_init(pvdone(i), 1);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  // Nothing above reads or writes global memory, so it overlaps the tail of
  // the previous kernel of the stream.
  griddep_wait();

  // Softmax warps (2-9) request their query rows first: row n = (warp - 2) + 8 u, lane l has
  // dims 2 l and 2 l + 1 of each half.
  constexpr int QPER = NQC / 8;
  uint32_t qreg[QPER][D / 64];
  const __nv_bfloat16* qbase = reinterpret_cast<const __nv_bfloat16*>(p.q);
  auto q_row = [&](int n) {
    const int t = n / p.group, hl = n - t * p.group;
    return qbase + ((size_t(b) * T + t) * p.hq + g * p.group + hl) * D;
  };
  const bool softmax_warp = warp >= 2 && warp <= 9;
  if (softmax_warp) {
#pragma unroll
    for (int u = 0; u < QPER; ++u) {
      const int n = warp - 2 + 8 * u;
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        qreg[u][h] = n < p.nq ? reinterpret_cast<const uint32_t*>(q_row(n))[32 * h + lane] : 0u;
    }
  }
  // Producer roles as in verify_tc.cu: warp 0 lanes 0-15 K pages 0-5, warp 10 lanes 0-15 V pages
  // 0-5 (both arm their slot's barrier), warp 11 K pages 6-7 (lanes 0-15) and V pages 6-7.
  const int half = lane >> 4, hl = lane & 15;
  const unsigned hmask = 0xFFFFu << (16 * half);
  const bool producer = warp == 0 || warp >= 10;
  const bool active = producer && (warp == 11 || half == 0);
  const bool is_k = warp == 11 ? half == 0 : warp == 0;
  const bool arms = warp != 11;
  const int pf = warp == 11 ? 6 : 0, np = warp == 11 ? 2 : 6;
  const int pbeg = p.cluster_merge ? split * p.max_pages / p.num_splits
                                   : split * p.pages_per_split;
  const int pnext = p.cluster_merge ? (split + 1) * p.max_pages / p.num_splits
                                    : pbeg + p.pages_per_split;
  const int32_t* bt_row = p.block_table + size_t(b) * p.max_pages;
  // Block-table entries four tiles ahead; lane np stands in with the tile's first page.
  auto table_entry = [&](int tt) {
    if (hl > np) return 0;
    const int page = pbeg + 8 * tt + (hl < np ? pf + hl : 0);
    return __ldg(&bt_row[min(page, p.max_pages - 1)]);
  };
  int held[4] = {0, 0, 0, 0};
  if (active) {
#pragma unroll
    for (int j = 0; j < 4; ++j) held[j] = table_entry(j);
  }
  // A softmax thread's position i of a tile is in the tile's page i / 16: the page's number is
  // requested two of the group's tiles ahead, its scale bytes one tile ahead.
  const int grp = (warp - 2) >> 2;          // 0: even tiles, 1: odd tiles
  const int q4 = warp & 3;                  // tensor-memory lane quarter of this warp
  const int i = 32 * q4 + lane;             // tile position owned
  // (volatile, here and for the scales: the compiler may not move the loads down to their uses)
  auto scale_block = [&](int t) {           // the page's block of scales, by its table entry
    const int page = min(pbeg + 8 * t + (i >> 4), p.max_pages - 1);
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(bt_row + page));
    return v;
  };
  int phys0 = 0, phys1 = 0;
  if (softmax_warp) {
    phys0 = scale_block(grp);
    phys1 = scale_block(grp + 2);
  }

  int L = p.ctx_lens[b];
  if (L < 0 || L + T > cap) {
    if (tid == 0) set_error(p.err, kErrDeviceFault);
    L = max(0, min(L, cap - T));
  }
  const int npages = (L + T + 15) / 16;
  const int pend = min(pnext, npages);
  const int ntiles = pend > pbeg ? (pend - pbeg + 7) / 8 : 0;
  const int last_valid = L + p.gamma;

  __syncthreads();   // barriers initialised before anyone waits on them
  // Producers start streaming right away; warps 1-9 build the query operand.
  uint32_t tmem = 0;
  if (warp >= 1 && warp <= 9) {
    constexpr int SN = 288;
    // Element (n, k) of a part: n * D + the 16-byte chunk k / 16 swizzled with the row.
    auto qoff = [](int n, int k) {
      const int c = k >> 4, sw = D == 128 ? n & 7 : (n >> 1) & 3;
      return n * D + ((c ^ sw) << 4) + (k & 15);
    };
    uint8_t* qs = smem + Cfg::kOffQ;
    if (softmax_warp) {
      // a row's exponent: its largest element lies in [2^n, 2^(n + 1)); rows of zeros take part
      // with the lowest
#pragma unroll
      for (int u = 0; u < QPER; ++u) {
        uint32_t most = 0;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) most = __vmaxu2(most, qreg[u][h] & 0x7fff7fffu);
        most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
        if (lane == 0) rowexp[warp - 2 + 8 * u] = most ? max(-100, int(most >> 7) - 127) : -1000;
      }
      if (CAPTURE) {
        // the captured query, summed over its rows and heads: this warp's rows
        float acc[D / 64][2] = {};
#pragma unroll
        for (int u = 0; u < QPER; ++u) {
          const int n = warp - 2 + 8 * u;
          if (n < p.nq && ((p.row_mask >> (n / p.group)) & 1u)) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              acc[h][0] += __uint_as_float(qreg[u][h] << 16);
              acc[h][1] += __uint_as_float(qreg[u][h] & 0xffff0000u);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          *reinterpret_cast<float2*>(qsum + (warp - 2) * D + 64 * h + 2 * lane) =
              make_float2(acc[h][0], acc[h][1]);
      }
    }
    for (int n = tid - 32; n < NQC; n += SN) tlim[n] = n < p.nq ? n / p.group : -1;
    named_bar(4, SN);
    // One exponent for all rows while they are within 2^4 of each other (a part's grid then
    // reaches 2^-13 of the smallest row's largest element, and 2^-17 of the unit's), else one a row.
    int most = -1000, least = 1000;
    for (int n = lane; n < NQC; n += 32) {
      const int e = rowexp[n];
      most = max(most, e);
      if (e > -1000) least = min(least, e);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    const bool one = most - least <= 4;
    if (most == -1000) most = 0;
    // The next e4m3 part of (x0, x1), |x| < 2^8, to row n of a pass; x keeps the rest.
    auto put_part = [&](int pass, int n, int k, float& x0, float& x1) {
      const uint32_t c = e4m3x2_from_f32(x0, x1);
      *reinterpret_cast<uint16_t*>(qs + pass * Cfg::kQ + qoff(n, k)) = uint16_t(c);
      uint32_t h, unused;
      f16x2_from_e4m3x4(c, h, unused);
      const float2 v = f32x2_from_f16x2(h);
      x0 -= v.x;
      x1 -= v.y;
    };
    if (softmax_warp) {
#pragma unroll
      for (int u = 0; u < QPER; ++u) {
        const int n = warp - 2 + 8 * u;
        const int e = rowexp[n], k = 7 - (one ? most : e == -1000 ? 0 : e);
        const float f = two_to(k);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          float x0 = __uint_as_float(qreg[u][h] << 16) * f;
          float x1 = __uint_as_float(qreg[u][h] & 0xffff0000u) * f;
          put_part(0, n, 64 * h + 2 * lane, x0, x1);
          put_part(kSideS ? 0 : 1, kSideS ? NQC + n : n, 64 * h + 2 * lane, x0, x1);
        }
        if (lane == 0) colfac[n] = one ? 1.f : two_to(-k);
      }
    } else {
      // warp 1: the captured query's parts, and the rows that fill up N
      int row = Cfg::kCap0;
      if constexpr (CAPTURE) {
        row += Cfg::kCap;
        float x[D / 64][2];
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          float2 v = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
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
            if (j & 1) {   // two parts leave less than 2^-8 of the largest: the next two start 2^8 lower
              x0 *= 256.f;
              x1 *= 256.f;
            }
          }
        }
        if (lane == 0) *capexp = -k;
      }
      for (int j = lane; j < (NS - row) * D / 4; j += 32)
#pragma unroll
        for (int pass = 0; pass < Cfg::kPasses; ++pass)
          reinterpret_cast<uint32_t*>(qs + pass * Cfg::kQ + row * D)[j] = 0;
      if (lane == 0) *uniform = one ? most - 7 : kMixed;
    }
    // Generic-proxy writes of Q must be visible to the tensor cores (async proxy).
    fence_proxy_async_smem();
    tc_fence_before();
    named_bar(4, SN);
    tc_fence_after();
    tmem = *tmem_slot;
  }
  bool ok = true;
  float o[NQC];   // a softmax thread's O^T row (unnormalised) at the end
  float Mg = kEmptyMax, Lg = 0.f;
  // the head dimension of a softmax thread's tensor-memory lane: M = 64 puts 16 rows in each
  // quarter of the lanes
  const int dim = !softmax_warp ? -1 : D == 128 ? i : lane < 16 ? 16 * q4 + lane : -1;
  const bool on_chip = p.cluster_merge || p.num_splits == 1;

  if (producer) {
    // ------------------------------------------------------------ producers
    const int depth = is_k ? KS : VS;
    const CUtensorMap* map = is_k ? &kmap : &vmap;
    const uint32_t ring = sbase + (is_k ? 0 : Cfg::kOffV);
    // The cache is streamed once per pass: its lines leave L2 first.
    const uint64_t stream_pol = l2_evict_first_policy();
    int issued = 0;
    if (active) {
      for (int t0 = 0; t0 < ntiles && ok; t0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = t0 + j;
          if (t >= ntiles) break;
          const int s = t % depth;
          const uint32_t full = is_k ? kfull(s) : vfull(s);
          const uint32_t freed = is_k ? kfree(s) : vfree(s);
          // the half-warp agrees on the outcome, so it leaves together
          if (t >= depth &&
              !__all_sync(hmask, mbar_wait_bounded(freed, ((t / depth) - 1) & 1))) {
            ok = false;
            break;
          }
          int phys = held[j];
          const int first = __shfl_sync(hmask, phys, np, 16);
          if (pbeg + 8 * t + pf + hl >= pend) phys = first;
          held[j] = table_entry(t + 4);
          if (hl < np && (phys < 0 || phys >= p.num_pages)) {
            set_error(p.err, kErrDeviceFault);
            phys = 0;
          }
          // one arrival per phase, with the whole tile's bytes
          if (arms && hl == 0) mbar_arrive_expect_tx(full, Cfg::kTile);
          __syncwarp(hmask);
          if (hl < np)
            tma_load_2d_hint(ring + s * Cfg::kTile + (pf + hl) * 16 * D, map, 0,
                             (phys * p.hkv + g) * 16, full, stream_pol);
          __syncwarp(hmask);
          issued = t + 1;
        }
      }
      if (!ok) {
        if (hl == 0) set_error(p.err, kErrDeviceTimeout);
        for (int t = max(0, issued - depth); t < issued; ++t)
          (void)mbar_wait_bounded(is_k ? kfull(t % depth) : vfull(t % depth), (t / depth) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idS = idesc_e4m3(128, NS);
    constexpr uint32_t idPV = idesc_f16_mn(D, NP);
    const bool leader = elect_one();
    // K and Q rows of 128 bytes with the 128-byte swizzle, or of 64 with the 64-byte one; V' and
    // P MN-major, P's rows of 128 or 64 bytes
    const uint64_t dKQ = smem_desc(0, 16, 8 * D, D == 128 ? 2 : 4);
    const uint64_t dV = smem_desc(0, 16384, 1024, 2);
    const uint64_t dP = smem_desc(0, 16384, 8 * Cfg::kPRow, Cfg::kPRow == 128 ? 2 : 4);
    auto with_addr = [](uint64_t d, uint32_t a16) { return d | uint64_t(a16 & 0x3FFFu); };
    const uint32_t qb = (sbase + Cfg::kOffQ) >> 4;
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
    };
    auto issue_pv = [&](int t) -> bool {
      const int gg = t & 1;
      if (!wait_all(pready(gg), (t >> 1) & 1)) return false;
      tc_fence_after();
      const uint32_t vb = (sbase + Cfg::kOffV16 + gg * Cfg::kV16) >> 4;
      const uint32_t pb = (sbase + Cfg::kOffP + gg * Cfg::kP) >> 4;
      if (leader) {
#pragma unroll
        for (int kp = 0; kp < 8; ++kp)
          tc_mma(tmem + 2 * Cfg::kSCol + Cfg::kOCol * gg, with_addr(dV, vb + kp * 128),
                 with_addr(dP, pb + kp * Cfg::kPRow), idPV, t >= 2 || kp > 0);
        tc_commit(pvdone(gg));
      }
      __syncwarp();
      return true;
    };
    for (int t = 0; t < ntiles && ok; ++t) {
      const int s = t % KS, gg = t & 1;
      if (!wait_all(kfull(s), (t / KS) & 1)) { ok = false; break; }
      if (t >= 2 && !wait_all(sread(gg), ((t >> 1) - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t kb = (sbase + s * Cfg::kTile) >> 4;
      if (leader) {
#pragma unroll
        for (int j = 0; j < Cfg::kPasses * (D / 32); ++j) {
          const int pass = j / (D / 32), ks = j % (D / 32);
          tc_mma_e4m3(tmem + Cfg::kSCol * gg, with_addr(dKQ, kb + 2 * ks),
                    with_addr(dKQ, qb + pass * (Cfg::kQ / 16) + 2 * ks), idS, j > 0);
        }
        tc_commit(sfull(gg));
        tc_commit(kfree(s));
      }
      __syncwarp();
      if (t >= 1 && !issue_pv(t - 1)) { ok = false; break; }
    }
    if (ok && ntiles > 0 && !issue_pv(ntiles - 1)) ok = false;
    if (!ok && leader) set_error(p.err, kErrDeviceTimeout);
    // every MMA issued has completed before tensor memory is released
    if (leader) tc_commit(drain);
    __syncwarp();
    (void)mbar_wait_bounded(drain, 0);
  } else {
    // ------------------------------------------------------------ softmax groups (warps 2-9)
    const uint32_t tl = tmem + (uint32_t(32 * q4) << 16);
    const uint32_t s_col = Cfg::kSCol * grp, o_col = 2 * Cfg::kSCol + Cfg::kOCol * grp;
    // Column references r (P = 2^(z - r)) are kept as -r, in registers up to 32 columns, else in
    // shared memory; 0 while `empty` says that the column has seen no unmasked logit.
    constexpr bool kSmemRef = NQC > 32;
    float nr[kSmemRef ? 2 : NQC];
    uint64_t ls2[NQC / 2];   // row sums, two columns each
#pragma unroll
    for (int n = 0; n < NQC; ++n) {
      if constexpr (!kSmemRef) nr[n] = 0.f;
      if (n % 2 == 0) ls2[n / 2] = 0;
    }
    float* nrg = nrefs + grp * NQC;
    if (kSmemRef) {
      if (i < NQC) nrg[i] = 0.f;
      named_bar(1 + grp, 128);
    }
    uint64_t empty = NQC == 64 ? ~0ull : (1ull << NQC) - 1;
    const int uni = *uniform;
    const bool mixed = uni == kMixed;
    const float base = mixed ? p.scale_log2 : p.scale_log2 * two_to(uni);
    const float cap_scale = CAPTURE ? p.scale * two_to(*capexp) : 0.f;
    float* srow = CAPTURE ? p.scores + size_t(unit) * p.score_stride : nullptr;
    int Lcap = L;
    if (CAPTURE && L > p.score_stride) {
      if (i == 0 && grp == 0) set_error(p.err, kErrDeviceFault);
      Lcap = p.score_stride;
    }
    // (pages past the table's or the pool's end: the producers record and clamp them)
    auto scale_at = [&](int phys) {
      return size_t(phys < 0 || phys >= p.num_pages ? 0 : phys) * p.hkv + g;
    };
    auto load_scale = [](const uint8_t* at) {
      uint32_t v;
      asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(at));
      return v;
    };
    uint32_t ekb = load_scale(p.k_scale + scale_at(phys0)), evb = load_scale(p.v_scale + scale_at(phys0));
    // S of columns 8 c .. 8 c + 7, the parts added
    auto load_chunk = [&](uint32_t at, int c, float* y) {
      float v8[8], w8[8];
      tmem_ld8(at + 8 * c, v8);
      if constexpr (kSideS) tmem_ld8(at + NQC + 8 * c, w8);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = kSideS ? v8[e] + w8[e] : v8[e];
    };
    // of all columns, up to three chunks in flight
    auto load_all = [&](uint32_t at, float* y) {
#pragma unroll
      for (int c0 = 0; c0 < NQC / 8; c0 += 3) {
        float v8[3][8], w8[3][8];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c0 + c >= NQC / 8) continue;
          tmem_ld8(at + 8 * (c0 + c), v8[c]);
          if constexpr (kSideS) tmem_ld8(at + NQC + 8 * (c0 + c), w8[c]);
        }
        if (kSideS || c0 + 3 >= NQC / 8) tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (c0 + c >= NQC / 8) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[8 * (c0 + c) + e] = kSideS ? v8[c][e] + w8[c][e] : v8[c][e];
        }
      }
    };
    int mytiles = 0;
    // A failed (timed-out) wait is carried to the group vote below, so the 128
    // threads of a group always leave the loop together.
    for (int t = grp; t < ntiles; t += 2) {
      const int k = t >> 1, s = t % VS;
      const int page = pbeg + 8 * t + (i >> 4);
      const bool live = page < pend;
      const int pos = page * 16 + (i & 15);
      // this position's scales; the next tile's are requested, and the page after that
      // (a row past the range holds the tile's first page again: its scales change nothing)
      const int e_k = kv8_exponent(uint8_t(ekb)), e_v = kv8_exponent(uint8_t(evb));
      ekb = load_scale(p.k_scale + scale_at(phys1));
      evb = load_scale(p.v_scale + scale_at(phys1));
      phys1 = scale_block(t + 4);
      // V' row i: the codes as f16 (zeros behind the window, where a code may be NaN), once PV of
      // the group's last tile has read the buffer; S of this tile follows that PV in the tensor pipe,
      // so this work hides behind it
      bool okt = ok && (k == 0 || mbar_wait_bounded(pvdone(grp), (k - 1) & 1));
      okt = okt && mbar_wait_bounded(vfull(s), (t / VS) & 1);
      {
        const int lpos = (live ? page : pbeg + 8 * t) * 16 + (i & 15);   // position loaded in row i
        const uint8_t* vrow = smem + Cfg::kOffV + s * Cfg::kTile + i * D;
        uint8_t* v16 = smem + Cfg::kOffV16 + grp * Cfg::kV16 + i * 128;
        const int sw = D == 128 ? i & 7 : (i >> 1) & 3;
        uint4 v[D / 16];   // (all loads ahead of the first store, which they might alias)
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          v[c] = *reinterpret_cast<const uint4*>(vrow + ((c ^ sw) << 4));
        if (lpos > last_valid) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint4 a, d;
          f16x2_from_e4m3x4(v[c].x, a.x, a.y);
          f16x2_from_e4m3x4(v[c].y, a.z, a.w);
          f16x2_from_e4m3x4(v[c].z, d.x, d.y);
          f16x2_from_e4m3x4(v[c].w, d.z, d.w);
          uint8_t* dst = v16 + (c >> 2) * 16384;
          const int cc = 2 * (c & 3);
          *reinterpret_cast<uint4*>(dst + ((cc ^ (i & 7)) << 4)) = a;
          *reinterpret_cast<uint4*>(dst + (((cc + 1) ^ (i & 7)) << 4)) = d;
        }
        mbar_arrive(vfree(s));
      }
      const float f_k = two_to(e_k), un = two_to(-e_v);
      const float f = live ? base * f_k : 0.f, add = live ? float(e_v) : -INFINITY;
      const uint64_t f2 = pair_f32(f, f), add2 = pair_f32(add, add), un2 = pair_f32(un, un);
      okt = okt && mbar_wait_bounded(sfull(grp), k & 1);
      tc_fence_after();
      // z of columns 8 c .. 8 c + 7 less their references; positions past the range are masked
      auto z_chunk = [&](int c, float* y) {   // (y: S in, z out)
        if (mixed) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= colfac[8 * c + e];
        }
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          float4 r4;
          if constexpr (kSmemRef)
            r4 = reinterpret_cast<const float4*>(nrg)[2 * c + e / 4];
          else
            r4 = make_float4(nr[8 * c + e], nr[8 * c + e + 1], nr[8 * c + e + 2], nr[8 * c + e + 3]);
          const uint64_t a = add_f32x2(fma_f32x2(pair_f32(y[e], y[e + 1]), f2, add2), pair_f32(r4.x, r4.y));
          const uint64_t d =
              add_f32x2(fma_f32x2(pair_f32(y[e + 2], y[e + 3]), f2, add2), pair_f32(r4.z, r4.w));
          unpair_f32(a, y[e], y[e + 1]);
          unpair_f32(d, y[e + 2], y[e + 3]);
        }
        if (pos > L) {   // window positions that a row may not see yet, and what lies behind them
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (pos > L + tlim[8 * c + e]) y[e] = -INFINITY;
        }
      };
      // P = 2^y of a chunk, eight f16 in 16 bytes of position i's row of columns, swizzled
      uint8_t* prow = smem + Cfg::kOffP + grp * Cfg::kP + i * Cfg::kPRow;
      const int psw = Cfg::kPRow == 128 ? i & 7 : (i >> 1) & 3;
      auto p_chunk = [&](int c, const float* y, bool sum) {
        uint32_t w4[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float p0 = ex2(y[e]), p1 = ex2(y[e + 1]);
          if (sum) ls2[4 * c + e / 2] = fma_f32x2(pair_f32(p0, p1), un2, ls2[4 * c + e / 2]);
          w4[e / 2] = pack_f16x2(p0, p1);
        }
        *reinterpret_cast<uint4*>(prow + ((c ^ psw) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
      };
      bool need = empty != 0;
      if (okt) {
        float y[NQC];
        float cx[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // the capture columns
        if constexpr (CAPTURE) tmem_ld8(tl + s_col + Cfg::kCap0, cx);
        load_all(tl + s_col, y);
        if (CAPTURE && pos < Lcap && live) {
          if constexpr (kSideS) {
#pragma unroll
            for (int j = 0; j < 3; ++j) cx[j] = cx[2 * j] + cx[2 * j + 1];
          }
          srow[pos] = fmaf(fmaf(cx[2], 0x1p-8f, cx[1]), 0x1p-8f, cx[0]) * (f_k * cap_scale);
        }
        float ym = -INFINITY;
#pragma unroll
        for (int c = 0; c < NQC / 8; ++c) {
          z_chunk(c, y + 8 * c);
#pragma unroll
          for (int e = 0; e < 8; e += 2) ym = fmaxf(fmaxf(ym, y[8 * c + e]), y[8 * c + e + 1]);
        }
        need = __any_sync(0xffffffffu, need || ym > kTop);
        // a warp that needs a higher reference leaves P and its sums to the raise below
        if (!need) {
#pragma unroll
          for (int c = 0; c < NQC / 8; ++c) p_chunk(c, y + 8 * c, true);
        }
      }
      // (columns that fill up N are never read; their P may be anything)
      const bool all_ok = __all_sync(0xffffffffu, okt);
      if (lane == 0) votes[(k & 1) * 8 + grp * 4 + q4] = all_ok ? 0 : 1;
      if (named_bar_any(1 + grp, 128, need || !okt)) {
        const int* vt = votes + (k & 1) * 8 + grp * 4;
        if (vt[0] | vt[1] | vt[2] | vt[3]) {
          ok = false;
          break;
        }
        // Raise: column maxima over the group's 128 positions, from S once more.  PV of the group's
        // last tile is done (above), so O^T may be rescaled.
        float* cm = colmax + grp * 4 * NQC;
#pragma unroll
        for (int c0 = 0; c0 < NQC; c0 += 32) {
          constexpr float kNone = -INFINITY;
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = kNone;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c0 + 8 * c >= NQC) continue;
            load_chunk(tl + s_col, c0 / 8 + c, y + 8 * c);
            z_chunk(c0 / 8 + c, y + 8 * c);
          }
          const float top = reduce_columns(y, [](float a, float d) { return fmaxf(a, d); });
          if (c0 + lane < NQC) cm[q4 * NQC + c0 + lane] = top;
        }
        named_bar(1 + grp, 128);
        // column n's new reference, at least kRaise below the largest z (cm is relative to the old one)
        auto raised = [&](int n, float nro, float& old) {
          const float top = fmaxf(fmaxf(cm[n], cm[NQC + n]), fmaxf(cm[2 * NQC + n], cm[3 * NQC + n]));
          old = ((empty >> n) & 1) ? kEmptyMax : -nro;
          return fmaxf(old, top - nro - kRaise);
        };
        uint64_t empty2 = empty;
        float fac[NQC];
#pragma unroll
        for (int n = 0; n < NQC; ++n) {
          const float nro = kSmemRef ? nrg[n] : nr[kSmemRef ? 0 : n];
          float old;
          const float now = raised(n, nro, old);
          const bool now_empty = now == kEmptyMax;
          fac[n] = ex2(old - now);
          if (!now_empty) empty2 &= ~(1ull << n);
          if constexpr (!kSmemRef) nr[n] = now_empty ? 0.f : -now;
        }
#pragma unroll
        for (int n = 0; n < NQC; n += 2) ls2[n / 2] = mul_f32x2(ls2[n / 2], pair_f32(fac[n], fac[n + 1]));
        if (k > 0) {
#pragma unroll
          for (int c = 0; c < NQC / 8; ++c) {
            float v8[8];
            tmem_ld8(tl + o_col + 8 * c, v8);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e) v8[e] *= fac[8 * c + e];
            tmem_st8(tl + o_col + 8 * c, v8);
          }
        }
        if (k > 0) tmem_st_wait();
        named_bar(1 + grp, 128);   // colmax (and nrg) read; colmax is rewritten at the next raise
        if constexpr (kSmemRef) {
          if (i < NQC) {
            const float nro = nrg[i];
            float old;
            const float now = raised(i, nro, old);
            nrg[i] = now == kEmptyMax ? 0.f : -now;
          }
          named_bar(1 + grp, 128);   // new references visible
        }
        empty = empty2;
        // P of this tile with the new references; the sums of a warp that has them were rescaled
#pragma unroll
        for (int c = 0; c < NQC / 8; ++c) {
          float y[8];
          load_chunk(tl + s_col, c, y);
          z_chunk(c, y);
          p_chunk(c, y, need);
        }
      }
      tc_fence_before();
      mbar_arrive(sread(grp));
      fence_proxy_async_smem();
      mbar_arrive(pready(grp));
      mytiles = k + 1;
    }
    // The group's last PV completes its O^T.
    if (mytiles > 0 && !mbar_wait_bounded(pvdone(grp), (mytiles - 1) & 1)) ok = false;
    tc_fence_after();
    if (!ok && i == 0) set_error(p.err, kErrDeviceTimeout);

    // Each group's (m, l, O^T) is a partial state of its own.  Row sums over its 128 positions:
#pragma unroll
    for (int c0 = 0; c0 < NQC; c0 += 32) {
      float v[32];
#pragma unroll
      for (int n = 0; n < 32; n += 2) {
        v[n] = v[n + 1] = 0.f;
        if (c0 + n < NQC) unpair_f32(ls2[(c0 + n) / 2], v[n], v[n + 1]);
      }
      const float sum = reduce_columns(v, [](float a, float d) { return a + d; });
      if (c0 + lane < NQC) colsum[(grp * 4 + q4) * NQC + c0 + lane] = sum;
    }
#pragma unroll
    for (int n = 0; n < NQC; ++n) o[n] = 0.f;
    if (mytiles > 0) {
#pragma unroll
      for (int c = 0; c < NQC / 8; ++c) {
        float v8[8];
        tmem_ld8(tl + o_col + 8 * c, v8);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[8 * c + e] = v8[e];
      }
      tmem_ld_wait();
    }
    if constexpr (!kSmemRef) {
#pragma unroll
      for (int n = 0; n < NQC; ++n)
        if (i == n) nrg[n] = nr[n];
    }
    named_bar(1 + grp, 128);
    if (i < NQC) {
      const float* cs = colsum + grp * 4 * NQC;
      if (mytiles > 0) Lg = cs[i] + cs[NQC + i] + cs[2 * NQC + i] + cs[3 * NQC + i];
      Mg = ((empty >> i) & 1) ? kEmptyMax : -nrg[i];
    }
    if (!on_chip) {
      // partial 2 * split + grp of the unit's 2 * num_splits
      const size_t part = (size_t(unit) * p.num_splits + split) * 2 + grp;
#pragma unroll
      for (int n = 0; n < NQC; ++n)
        if (n < p.nq && dim >= 0) p.part_o[(part * p.nq + n) * D + dim] = o[n];
      if (i < p.nq) {
        p.part_ml[(part * p.nq + i) * 2 + 0] = Mg;
        p.part_ml[(part * p.nq + i) * 2 + 1] = Lg;
      }
    }
  }

  // Every CTA of the cluster is past its last MMA and holds no load in flight,
  // so its rings and V' buffers are free from here on.
  tc_fence_before();
  if (on_chip)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out);
  auto out_row = [&](int n) {
    const int t = n / p.group, hl2 = n - t * p.group;
    return out + ((size_t(b) * T + t) * p.hq + g * p.group + hl2) * D;
  };
  if (on_chip) {
    merge_on_chip<D, NQC, Cfg::kThreads>(p, unit, split, softmax_warp ? grp : -1, dim, i, o, Mg,
                                         Lg, smem, reinterpret_cast<float*>(smem + Cfg::kMergeOff),
                                         flag, out_row);
  } else {
    SplitWorkspace ws{p.tickets, p.part_ml, p.part_o};
    finish_splits<D, Cfg::kThreads, NQC>(ws, unit, p.num_splits, 2 * p.num_splits, p.nq, out_row,
                                         reinterpret_cast<float*>(smem), flag);
  }
}

// Launch (launch = true) or, with launch = false, the number of clusters of
// p.cluster_size CTAs that can be resident at once (into *clusters).
template <int D, int NQC, bool CAP>
static cudaError_t launch_one(const CUtensorMap& kmap, const CUtensorMap& vmap,
                              const VerifyParams& p, int batch, cudaStream_t stream, bool launch,
                              int* clusters) {
  using Cfg = Kv8Cfg<D, NQC, CAP>;
  static std::atomic<uint32_t> configured{0};
  cudaError_t e = once_per_device(configured, [] {
    cudaError_t r = cudaFuncSetAttribute(verify_kv8_kernel<D, NQC, CAP>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Cfg::kSmem);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(verify_kv8_kernel<D, NQC, CAP>,
                                cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_splits, p.hkv, batch);
  cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster_merge ? p.cluster_size : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = launch ? 2 : 1;
  if (!launch)
    return cudaOccupancyMaxActiveClusters(clusters, verify_kv8_kernel<D, NQC, CAP>, &cfg);
  return cudaLaunchKernelEx(&cfg, verify_kv8_kernel<D, NQC, CAP>, kmap, vmap, p);
}

// The softmax's columns: nq rounded up to 8.
template <int D, bool CAP>
static cudaError_t launch_cols(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const VerifyParams& p, int batch, cudaStream_t s, bool launch,
                               int* clusters) {
  if (!verify_kv8_supported(D, p.nq)) return cudaErrorInvalidValue;
  switch ((p.nq + 7) / 8) {
    case 1: return launch_one<D, 8, CAP>(kmap, vmap, p, batch, s, launch, clusters);
    case 2: return launch_one<D, 16, CAP>(kmap, vmap, p, batch, s, launch, clusters);
    case 3: return launch_one<D, 24, CAP>(kmap, vmap, p, batch, s, launch, clusters);
    case 4: return launch_one<D, 32, CAP>(kmap, vmap, p, batch, s, launch, clusters);
    case 5: return launch_one<D, 40, CAP>(kmap, vmap, p, batch, s, launch, clusters);
  }
  if constexpr (D == 64) {
    switch ((p.nq + 7) / 8) {
      case 6: return launch_one<D, 48, CAP>(kmap, vmap, p, batch, s, launch, clusters);
      case 7: return launch_one<D, 56, CAP>(kmap, vmap, p, batch, s, launch, clusters);
      case 8: return launch_one<D, 64, CAP>(kmap, vmap, p, batch, s, launch, clusters);
    }
  }
  return cudaErrorInvalidValue;
}

#define VEGAS_CAT2(a, b) a##b
#define VEGAS_CAT(a, b) VEGAS_CAT2(a, b)

cudaError_t VEGAS_CAT(launch_verify_kv8_d, VEGAS_KV8_D)(const CUtensorMap& kmap,
                                                       const CUtensorMap& vmap,
                                                       const VerifyParams& p, bool capture,
                                                       int batch, cudaStream_t stream) {
  constexpr int D = VEGAS_KV8_D;
  return capture ? launch_cols<D, true>(kmap, vmap, p, batch, stream, true, nullptr)
                 : launch_cols<D, false>(kmap, vmap, p, batch, stream, true, nullptr);
}

int VEGAS_CAT(verify_kv8_max_active_clusters_d, VEGAS_KV8_D)(int nq, bool capture, int cluster) {
  constexpr int D = VEGAS_KV8_D;
  if (cluster < 1 || cluster > kMaxVerifyCluster) return 0;
  if (!verify_kv8_supported(D, nq)) return 0;
  constexpr int kDevices = 32;
  // [device][capture][column tiles of the softmax][cluster]: 0 unknown, -1 none, else the count
  static std::atomic<int> cache[kDevices][2][9][kMaxVerifyCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  std::atomic<int>& slot = cache[dev][capture ? 1 : 0][(nq + 7) / 8][cluster];
  int c = slot.load(std::memory_order_acquire);
  if (c == 0) {
    VerifyParams p{};
    p.hkv = 1;
    p.nq = nq;
    p.num_splits = cluster;
    p.cluster_size = cluster;
    p.cluster_merge = 1;
    CUtensorMap none{};
    int n = 0;
    cudaError_t e = capture ? launch_cols<D, true>(none, none, p, 1, 0, false, &n)
                            : launch_cols<D, false>(none, none, p, 1, 0, false, &n);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    c = n > 0 ? n : -1;
    slot.store(c, std::memory_order_release);
  }
  return c > 0 ? c : 0;
}

}  // namespace vegas
