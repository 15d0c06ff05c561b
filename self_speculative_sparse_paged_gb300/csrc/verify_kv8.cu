// Verify attention with captured scores over the 8-bit cache, on the 5th-generation tensor cores
// (compiled once per head_dim, VEGAS_KV8_D).
//
// The work is that of verify_tc.cu on half the bytes, laid out so that its length goes by what the
// sequences hold, not by what their tables could: the 128-position tiles of all (sequence, KV
// head) units stand in one row, and each CTA (one an SM) takes an equal run of it, whole units or
// pieces, with the K/V stream going on from one unit to the next.  Twelve warps:
//   warps 0-7   two softmax groups of four warps that alternate tiles; a thread owns a position
//               of a tile, and a head dimension of the group's O^T.  They also build the query operand
//               of a unit and finish it.
//   warps 8, 9  TMA producers: 8 pages a tile into K and V rings, block-table entries prefetched
//   warp 10     issues the MMAs
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
//
// A unit that one CTA covers is written by it; the pieces of a shared one go to the workspace
// (fp32 O, maximum and sum of each row), and the CTA that arrives last on the unit's ticket merges
// them.  No CTA waits for another.
#include "attn_core.cuh"
#include "kernels.h"
#include "kv8.cuh"

#ifndef VEGAS_KV8_D
#error "compile with -DVEGAS_KV8_D=64 or -DVEGAS_KV8_D=128"
#endif

namespace vegas {

namespace {
constexpr float kTop = 15.f, kRaise = 7.f;   // log2 of the largest P, and of P at a raised reference
constexpr int kCapParts = 6;
constexpr int kLeastTiles = 2;   // of a CTA that takes part
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
  static constexpr int kSCol = (NS + 31) / 32 * 32, kOCol = (NP + 31) / 32 * 32;
  static constexpr uint32_t kTmemCols =
      2 * (kSCol + kOCol) <= 128 ? 128 : 2 * (kSCol + kOCol) <= 256 ? 256 : 512;
  static_assert(2 * (kSCol + kOCol) <= 512, "tensor memory");
  static constexpr int kOffV = KS * kTile;
  static constexpr int kOffV16 = kOffV + VS * kTile;
  static constexpr int kOffP = kOffV16 + 2 * kV16;
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffBar = kOffQ + kPasses * kQ;
  static constexpr int kNumBars = 2 * KS + 2 * VS + 4 * 2 + 2;
  static constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
  // misc: 16 words; votes[2][2][4]; warp sums[12] (64 bits); colmax[2][4][NQC], colsum[2][4][NQC],
  // colfac[NQC], nref[2][NQC], fac[2][NQC], colM[NQC], colL[NQC]; tlim[NQC]; rowexp[NQC]
  static constexpr size_t kMisc = 64 + 64 + 96 + 4 * size_t(16 + 3 + 2 + 2 + 2) * NQC;
  static constexpr size_t kSmem = size_t(kOffMisc) + kMisc + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // a piece's merge weights (one a row and piece) in the V' and P buffers
  static_assert(NQC * 4 * kMaxKv8Ctas <= 2 * kV16 + 2 * kP, "merge weights");
  static_assert(NQC / 2 * D * 4 <= kV16, "exchange of half the columns");
  static_assert(8 * D * 4 <= kP, "partial sums of the captured query (P's buffer)");
};

// A place in the row of tiles: tile t of KV head g of sequence b.
struct Place {
  long long left;          // tiles of this CTA from here on
  int b, g, t, tiles, L;   // tiles: of each unit of sequence b; L: its context length
};

template <int D, int NQC, bool CAPTURE>
__global__ void __launch_bounds__(384, 1)
    verify_kv8_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const VerifyKv8Params p) {
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
  // ready, PV done (per softmax group); queries ready, MMA drain
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
  long long* wsum = reinterpret_cast<long long*>(misc + 128);    // [12] tiles a head of a warp's sequences
  float* colmax = reinterpret_cast<float*>(misc + 224);          // [2][4][NQC]
  float* colsum = colmax + 8 * NQC;                              // [2][4][NQC]
  float* colfac = colsum + 8 * NQC;                              // [NQC] 2^-k of rows of unlike size
  float* nrefs = colfac + NQC;                                   // [2][NQC] -reference
  float* fac = nrefs + 2 * NQC;                                  // [2][NQC] weights of the groups
  float* colM = fac + 2 * NQC;                                   // [NQC] maximum, and sum, of a piece
  float* colL = colM + NQC;
  int* tlim = reinterpret_cast<int*>(colL + NQC);                // [NQC]
  int* rowexp = tlim + NQC;                                      // [NQC]
  float* qsum = reinterpret_cast<float*>(smem + Cfg::kOffP);     // [8][D] parts of the captured sum

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
      mbar_init(vfree(s), 128);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull(i), 1);
      mbar_init(sread(i), 128);
      mbar_init(pready(i), 128);
      mbar_init(pvdone(i), 1);
    }
    mbar_init(qready, 256);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 10) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  // Nothing above reads or writes global memory, so it overlaps the tail of
  // the previous kernel of the stream.
  griddep_wait();

  // ---- this CTA's run of tiles.  A sequence's units have ceil((L + T) / 128) tiles each.
  auto length = [&](int b) {
    const int L = p.ctx_lens[b];
    return L < 0 || L + T > cap ? max(0, min(L, cap - T)) : L;   // (recorded below)
  };
  auto tiles_of = [&](int L) { return (L + T + 127) >> 7; };
  // warp w counts sequences [w * chunk, (w + 1) * chunk)
  const int chunk = (p.batch + 383) / 384 * 32;
  {
    long long sum = 0;
    for (int b = warp * chunk + lane; b < min(p.batch, (warp + 1) * chunk); b += 32) {
      const int L = p.ctx_lens[b];
      if (cta == 0 && (L < 0 || L + T > cap)) set_error(p.err, kErrDeviceFault);
      sum += tiles_of(length(b));
    }
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
    if (lane == 0) wsum[warp] = sum;
  }
  tc_fence_before();
  __syncthreads();   // (and the barriers are initialised before anyone waits on them)
  tc_fence_after();
  long long all = 0;
#pragma unroll
  for (int w = 0; w < 12; ++w) all += wsum[w];
  all *= p.hkv;
  // CTAs that take part: at least kLeastTiles each
  const int n = int(max(1ll, min((long long)gridDim.x, all / kLeastTiles)));
  // (64-bit quotients take a few hundred clocks: 32-bit ones while they do)
  const bool small = all < (1 << 24);   // (n < 2^8)
  auto quotient = [&](long long a, long long d) {
    return small ? (long long)(uint32_t(a) / uint32_t(d)) : a / d;
  };
  auto run_begin = [&](int c) { return quotient(c * all, n); };
  const long long begin = cta < n ? run_begin(cta) : 0, end = cta < n ? run_begin(cta + 1) : 0;
  // the CTA that holds tile x: the last c with run_begin(c) <= x
  auto cta_of = [&](long long x) { return int(quotient((x + 1) * n - 1, all)); };
  Place start{end - begin, 0, 0, 0, 1, 0};
  long long base = 0;   // first tile of sequence start.b
  if (begin < end) {
    int w = 0;
    while (w < 11 && base + wsum[w] * p.hkv <= begin) base += wsum[w++] * p.hkv;
    for (int b0 = w * chunk;; b0 += 32) {
      const int b = b0 + lane;
      const int L = b < p.batch ? length(b) : 0;
      const long long mine = b < p.batch ? (long long)tiles_of(L) * p.hkv : 0;
      long long upto = mine;
#pragma unroll
      for (int o2 = 1; o2 < 32; o2 <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o2);
        if (lane >= o2) upto += v;
      }
      const unsigned beyond = __ballot_sync(0xffffffffu, base + upto > begin);
      if (beyond || b0 + 32 >= p.batch) {
        const int l = beyond ? __ffs(beyond) - 1 : 31;   // (there is one: begin < end <= all)
        start.b = min(b0 + l, p.batch - 1);
        start.L = __shfl_sync(0xffffffffu, L, l);
        base += __shfl_sync(0xffffffffu, upto - mine, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
    start.tiles = tiles_of(start.L);
    start.g = int(quotient(begin - base, start.tiles));
    start.t = int((begin - base) - (long long)start.g * start.tiles);
  }
  auto next_unit = [&](Place& q) {   // (left counted down by the caller)
    q.t = 0;
    if (++q.g == p.hkv) {
      q.g = 0;
      if (q.left > 0) {
        q.L = length(++q.b);
        q.tiles = tiles_of(q.L);
      }
    }
  };
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  // 384 threads launch with 168 registers each: 2 x 128 x 216 + 128 x 72 are that.
  if (warp >= 8) {
    leave_registers<72>();
    if (warp < 10) {
      // ---------------------------------------------------------- producers: K (8), V (9)
      // Lane j < 8 loads page j of a tile; a page past the sequence's last is that one again (its
      // positions are masked).
      const bool is_k = warp == 8;
      const int depth = is_k ? KS : VS;
      const CUtensorMap* map = is_k ? &kmap : &vmap;
      const uint32_t ring = sbase + (is_k ? 0 : Cfg::kOffV);
      // The cache is streamed once per pass: its lines leave L2 first.
      const uint64_t stream_pol = l2_evict_first_policy();
      const int j8 = lane & 7;
      Place ahead = start;
      // a tile's table entry, requested four tiles before its use, and its KV head
      int held[4], head[4];
      auto request = [&](int j) {
        held[j] = head[j] = 0;
        if (ahead.left > 0) {
          const int page = min(8 * ahead.t + j8, (ahead.L + T - 1) >> 4);
          held[j] = __ldg(&p.block_table[size_t(ahead.b) * p.max_pages + page]);
          head[j] = ahead.g;
          --ahead.left;
          if (++ahead.t == ahead.tiles) next_unit(ahead);
        }
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) request(j);
      long long issued = 0;
      int s = 0, round = 0;
      for (long long it0 = 0; it0 < start.left && ok; it0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (it0 + j >= start.left) break;
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
          issued = it0 + j + 1;
          if (++s == depth) {
            s = 0;
            ++round;
          }
        }
      }
      if (!ok) {
        if (lane == 0) set_error(p.err, kErrDeviceTimeout);
        for (long long t = issued > depth ? issued - depth : 0; t < issued; ++t)
          (void)mbar_wait_bounded(is_k ? kfull(int(t % depth)) : vfull(int(t % depth)),
                                  int(t / depth) & 1);
      }
    } else if (warp == 10) {
      // ---------------------------------------------------------- MMA issuer
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
      // PV of the CTA's tile it (first: its group's first tile of the unit)
      auto issue_pv = [&](uint32_t it, bool first) -> bool {
        const int gg = it & 1;
        if (!wait_all(pready(gg), (it >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t vb = (sbase + Cfg::kOffV16 + gg * Cfg::kV16) >> 4;
        const uint32_t pb = (sbase + Cfg::kOffP + gg * Cfg::kP) >> 4;
        if (leader) {
#pragma unroll
          for (int kp = 0; kp < 8; ++kp)
            tc_mma(tmem + 2 * Cfg::kSCol + Cfg::kOCol * gg, with_addr(dV, vb + kp * 128),
                   with_addr(dP, pb + kp * Cfg::kPRow), idPV, !first || kp > 0);
          tc_commit(pvdone(gg));
        }
        __syncwarp();
        return true;
      };
      Place at = start;
      uint32_t it = 0;
      int s = 0, round = 0, seg = 0;
      while (at.left > 0 && ok) {
        const int tiles = int(min((long long)(at.tiles - at.t), at.left));
        if (!wait_all(qready, seg++ & 1)) {
          ok = false;
          break;
        }
        for (int t = 0; t < tiles && ok; ++t, ++it) {
          const int gg = it & 1;
          if (!wait_all(kfull(s), round & 1)) { ok = false; break; }
          if (it >= 2 && !wait_all(sread(gg), ((it >> 1) - 1) & 1)) { ok = false; break; }
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
          if (++s == KS) {
            s = 0;
            ++round;
          }
          if (t >= 1 && !issue_pv(it - 1, t - 1 < 2)) ok = false;
        }
        // the unit's last PV, before the next unit's queries are waited for
        if (ok && !issue_pv(it - 1, tiles - 1 < 2)) ok = false;
        at.left -= tiles;
        if (at.left > 0) next_unit(at);
      }
      if (!ok && leader) set_error(p.err, kErrDeviceTimeout);
      // every MMA issued has completed before tensor memory is released
      if (leader) tc_commit(drain);
      __syncwarp();
      (void)mbar_wait_bounded(drain, 0);
    }
  } else {
    take_registers<216>();
    // ------------------------------------------------------------ softmax groups (warps 0-7)
    const int grp = warp >> 2;                // 0: even tiles, 1: odd tiles
    const int q4 = warp & 3;                  // tensor-memory lane quarter of this warp
    const int i = 32 * q4 + lane;             // tile position owned
    // head dimension owned: M = 64 puts 16 rows in each quarter of the lanes
    const int dim = D == 128 ? i : lane < 16 ? 16 * q4 + lane : -1;
    const uint32_t tl = tmem + (uint32_t(32 * q4) << 16);
    const uint32_t s_col = Cfg::kSCol * grp, o_col = 2 * Cfg::kSCol + Cfg::kOCol * grp;
    // Column references r (P = 2^(z - r)) are kept as -r, in registers up to 32 columns, else in
    // shared memory; 0 while `empty` says that the column has seen no unmasked logit.
    constexpr bool kSmemRef = NQC > 32;
    constexpr int QPER = NQC / 8;
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
    auto load_page = [&](const Place& u, int t) {   // volatile, here and below: the compiler may not
      const int page = min(8 * t + (i >> 4), (u.L + T - 1) >> 4);   // move the loads down to their uses
      int v;
      asm volatile("ld.global.nc.s32 %0, [%1];"
                   : "=r"(v)
                   : "l"(p.block_table + size_t(u.b) * p.max_pages + page));
      return v;
    };
    auto load_scale = [&](const uint8_t* scales, int phys, int g) {
      uint32_t v;
      const size_t block = size_t(phys < 0 || phys >= p.num_pages ? 0 : phys) * p.hkv + g;
      asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(scales + block));
      return v;
    };
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

    Place at = start;
    long long unit0 = base + (long long)start.g * start.tiles;   // first tile of the unit
    uint32_t it0 = 0;             // the CTA's tile with which the unit begins
    uint32_t vs0 = 0;             // (it0 modulo the V ring, and the ring's round)
    uint32_t vround0 = 0;
    while (at.left > 0) {
      const int tiles = int(min((long long)(at.tiles - at.t), at.left));
      const int L = at.L, g = at.g, b = at.b;
      const int last_valid = L + p.gamma;
      const uint32_t first = it0 + ((it0 ^ uint32_t(grp)) & 1);   // this group's first tile

      // ---------------------------------------------------------- the unit's queries
      int phys1 = 0;
      uint32_t ekb, evb;
      {
        const int phys0 = load_page(at, at.t + int(first - it0));
        phys1 = load_page(at, at.t + int(first - it0) + 2);
        uint32_t qreg[QPER][D / 64];
#pragma unroll
        for (int u = 0; u < QPER; ++u) {
          const int n2 = warp + 8 * u, t = n2 / p.group, hl = n2 - t * p.group;
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            qreg[u][h] = n2 < p.nq ? reinterpret_cast<const uint32_t*>(
                                         qbase + ((size_t(b) * T + t) * p.hq + g * p.group + hl) * D)
                                         [32 * h + lane]
                                   : 0u;
        }
        // a row's exponent: its largest element lies in [2^n, 2^(n + 1))
#pragma unroll
        for (int u = 0; u < QPER; ++u) {
          uint32_t most = 0;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) most = __vmaxu2(most, qreg[u][h] & 0x7fff7fffu);
          most = __reduce_max_sync(0xffffffffu, max(most & 0xffffu, most >> 16));
          if (lane == 0) rowexp[warp + 8 * u] = most ? max(-100, int(most >> 7) - 127) : -1000;
        }
        ekb = load_scale(p.k_scale, phys0, g);
        evb = load_scale(p.v_scale, phys0, g);
        if (CAPTURE) {
          // the captured query, summed over its rows and heads: this warp's rows
          float acc[D / 64][2] = {};
#pragma unroll
          for (int u = 0; u < QPER; ++u) {
            const int n2 = warp + 8 * u;
            if (n2 < p.nq && ((p.row_mask >> (n2 / p.group)) & 1u)) {
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
        if (tid < NQC) tlim[tid] = tid < p.nq ? tid / p.group : -1;
        named_bar(3, 256);
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
          const int n2 = warp + 8 * u;
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
        if (kSmemRef && i < NQC) nrg[i] = 0.f;
        // Generic-proxy writes of Q must be visible to the tensor cores (async proxy).
        fence_proxy_async_smem();
        mbar_arrive(qready);
        named_bar(3, 256);   // (what was written above is read by all)
      }

      // ---------------------------------------------------------- its tiles
      float nr[kSmemRef ? 2 : NQC];
      uint64_t ls2[NQC / 2];   // row sums, two columns each
#pragma unroll
      for (int n2 = 0; n2 < NQC; ++n2) {
        if constexpr (!kSmemRef) nr[n2] = 0.f;
        if (n2 % 2 == 0) ls2[n2 / 2] = 0;
      }
      uint64_t empty = NQC == 64 ? ~0ull : (1ull << NQC) - 1;
      const int uni = *uniform;
      const bool mixed = uni == kMixed;
      const float scale0 = mixed ? p.scale_log2 : p.scale_log2 * two_to(uni);
      const float cap_scale = CAPTURE ? p.scale * two_to(*capexp) : 0.f;
      float* srow = CAPTURE ? p.scores + (size_t(b) * p.hkv + g) * p.score_stride : nullptr;
      int Lcap = L;
      if (CAPTURE && L > p.score_stride) {
        if (i == 0 && grp == 0) set_error(p.err, kErrDeviceFault);
        Lcap = p.score_stride;
      }
      uint32_t vs = vs0 + (first - it0), vround = vround0;
      if (vs >= VS) {
        vs -= VS;
        ++vround;
      }
      bool any = false;   // this group has a tile of the unit
      // A failed (timed-out) wait is carried to the group vote below, so the 128
      // threads of a group always leave the loop together.
      for (uint32_t it = first; it < it0 + uint32_t(tiles); it += 2) {
        const uint32_t k = it >> 1;
        const int t = at.t + int(it - it0);
        const int pos = 128 * t + i;
        // this position's scales; the next tile's are requested, and the page after that
        const int e_k = kv8_exponent(uint8_t(ekb)), e_v = kv8_exponent(uint8_t(evb));
        ekb = load_scale(p.k_scale, phys1, g);
        evb = load_scale(p.v_scale, phys1, g);
        phys1 = load_page(at, t + 4);
        // V' row i: the codes as f16 (zeros behind the window, where a code may be NaN), once PV of
        // the group's last tile has read the buffer; S of this tile follows that PV in the tensor
        // pipe, so this work hides behind it
        bool okt = ok && (it < 2 || mbar_wait_bounded(pvdone(grp), (k - 1) & 1));
        okt = okt && mbar_wait_bounded(vfull(vs), vround & 1);
        {
          const uint8_t* vrow = smem + Cfg::kOffV + vs * Cfg::kTile + i * D;
          uint8_t* v16 = smem + Cfg::kOffV16 + grp * Cfg::kV16 + i * 128;
          const int sw = D == 128 ? i & 7 : (i >> 1) & 3;
          uint4 v[D / 16];   // (all loads ahead of the first store, which they might alias)
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            v[c] = *reinterpret_cast<const uint4*>(vrow + ((c ^ sw) << 4));
          if (pos > last_valid) {
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
          mbar_arrive(vfree(vs));
        }
        vs += 2;
        if (vs >= VS) {
          vs -= VS;
          ++vround;
        }
        const float f_k = two_to(e_k), un = two_to(-e_v), f = scale0 * f_k, add = float(e_v);
        const uint64_t f2 = pair_f32(f, f), add2 = pair_f32(add, add), un2 = pair_f32(un, un);
        okt = okt && mbar_wait_bounded(sfull(grp), k & 1);
        tc_fence_after();
        // z of columns 8 c .. 8 c + 7 less their references (y: S in, z out)
        auto z_chunk = [&](int c, float* y) {
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
            const uint64_t a =
                add_f32x2(fma_f32x2(pair_f32(y[e], y[e + 1]), f2, add2), pair_f32(r4.x, r4.y));
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
        // (columns that fill up N are never read; their P may be anything)
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
          float cx[8] = {};   // the capture columns
          if constexpr (CAPTURE) tmem_ld8(tl + s_col + Cfg::kCap0, cx);
          load_all(tl + s_col, y);
          if (CAPTURE && pos < Lcap) {
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
        const bool all_ok = __all_sync(0xffffffffu, okt);
        if (lane == 0) votes[(k & 1) * 8 + grp * 4 + q4] = all_ok ? 0 : 1;
        if (named_bar_any(1 + grp, 128, need || !okt)) {
          const int* vt = votes + (k & 1) * 8 + grp * 4;
          if (vt[0] | vt[1] | vt[2] | vt[3]) {
            ok = false;
            break;
          }
          // Raise: column maxima over the group's 128 positions, from S once more.  PV of the
          // group's last tile is done (above), so O^T may be rescaled.
          float* cm = colmax + grp * 4 * NQC;
#pragma unroll
          for (int c0 = 0; c0 < NQC; c0 += 32) {
            float y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = -INFINITY;
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
          // column n2's new reference, at least kRaise below the largest z (cm is relative to the
          // old one)
          auto raised = [&](int n2, float nro, float& old) {
            const float top =
                fmaxf(fmaxf(cm[n2], cm[NQC + n2]), fmaxf(cm[2 * NQC + n2], cm[3 * NQC + n2]));
            old = ((empty >> n2) & 1) ? kEmptyMax : -nro;
            return fmaxf(old, top - nro - kRaise);
          };
          uint64_t empty2 = empty;
          float f1[NQC];
#pragma unroll
          for (int n2 = 0; n2 < NQC; ++n2) {
            const float nro = kSmemRef ? nrg[n2] : nr[kSmemRef ? 0 : n2];
            float old;
            const float now = raised(n2, nro, old);
            const bool now_empty = now == kEmptyMax;
            f1[n2] = ex2(old - now);
            if (!now_empty) empty2 &= ~(1ull << n2);
            if constexpr (!kSmemRef) nr[n2] = now_empty ? 0.f : -now;
          }
#pragma unroll
          for (int n2 = 0; n2 < NQC; n2 += 2)
            ls2[n2 / 2] = mul_f32x2(ls2[n2 / 2], pair_f32(f1[n2], f1[n2 + 1]));
          if (any) {
#pragma unroll
            for (int c = 0; c < NQC / 8; ++c) {
              float v8[8];
              tmem_ld8(tl + o_col + 8 * c, v8);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) v8[e] *= f1[8 * c + e];
              tmem_st8(tl + o_col + 8 * c, v8);
            }
            tmem_st_wait();
          }
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
        any = true;
      }

      // ---------------------------------------------------------- the unit's end
      // The group's last PV completes its O^T.
      if (any && ok) {
        const uint32_t last = it0 + uint32_t(tiles) - 1 - ((it0 + uint32_t(tiles) - 1 - uint32_t(grp)) & 1);
        if (!mbar_wait_bounded(pvdone(grp), (last >> 1) & 1)) ok = false;
      }
      tc_fence_after();
      // row sums over the group's 128 positions, references, O^T
#pragma unroll
      for (int c0 = 0; c0 < NQC; c0 += 32) {
        float v[32];
#pragma unroll
        for (int n2 = 0; n2 < 32; n2 += 2) {
          v[n2] = v[n2 + 1] = 0.f;
          if (c0 + n2 < NQC) unpair_f32(ls2[(c0 + n2) / 2], v[n2], v[n2 + 1]);
        }
        const float sum = reduce_columns(v, [](float a, float d) { return a + d; });
        if (c0 + lane < NQC) colsum[(grp * 4 + q4) * NQC + c0 + lane] = sum;
      }
      if (q4 == 0 && !kSmemRef) {
#pragma unroll
        for (int n2 = 0; n2 < NQC; ++n2)
          if (lane == n2) nrg[n2] = nr[kSmemRef ? 0 : n2];
      }
      // (a group without a tile: an empty reference; threads of a group agree on `empty`)
      float o[NQC];
#pragma unroll
      for (int n2 = 0; n2 < NQC; ++n2) o[n2] = 0.f;
      if (any && ok) {
#pragma unroll
        for (int c = 0; c < NQC / 8; ++c) {
          float v8[8];
          tmem_ld8(tl + o_col + 8 * c, v8);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[8 * c + e] = v8[e];
        }
        tmem_ld_wait();
      }
      tc_fence_before();
      if (named_bar_any(3, 256, !ok)) {   // both groups leave together
        if (!ok && i == 0) set_error(p.err, kErrDeviceTimeout);
        break;
      }
      // weights of the two groups' states, by the threads of a group that own a column
      if (i < NQC) {
        const float m = ((empty >> i) & 1) ? kEmptyMax : -nrg[i];
        const float* cs = colsum + grp * 4 * NQC;
        const float l = cs[i] + cs[NQC + i] + cs[2 * NQC + i] + cs[3 * NQC + i];
        fac[grp * NQC + i] = m;
        colmax[grp * 4 * NQC + i] = l;
      }
      named_bar(3, 256);
      // Group 0 finishes the first half of the columns, group 1 the second: each hands its part of
      // the other's half over in its V' buffer, weighted.
      constexpr int H = NQC / 2;
      auto weight = [&](int n2, float& M) {   // of this group's state of column n2
        const float m0 = fac[n2], m1 = fac[NQC + n2];
        M = fmaxf(m0, m1);
        return ex2((grp ? m1 : m0) - M);
      };
      float* give = reinterpret_cast<float*>(smem + Cfg::kOffV16 + grp * Cfg::kV16);
      const float* get = reinterpret_cast<const float*>(smem + Cfg::kOffV16 + (grp ^ 1) * Cfg::kV16);
      float mine[H];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        float M;
        const int other = grp ? j : H + j, own = grp ? H + j : j;
        const float w = weight(other, M);
        if (dim >= 0) give[j * D + dim] = (grp ? o[j] : o[H + j]) * w;
        mine[j] = (grp ? o[H + j] : o[j]) * weight(own, M);
      }
      if (i < H) {   // the piece's maximum and sum of the columns that this group finishes
        const int n2 = grp ? H + i : i;
        const float m0 = fac[n2], m1 = fac[NQC + n2], M = fmaxf(m0, m1);
        colM[n2] = M;
        colL[n2] = ex2(m0 - M) * colmax[n2] + ex2(m1 - M) * colmax[4 * NQC + n2];
      }
      named_bar(3, 256);
      const long long unit1 = unit0 + at.tiles;
      const int c0 = cta_of(unit0), c1 = cta_of(unit1 - 1);
      const size_t unit = size_t(b) * p.hkv + g;
      auto out_row = [&](int n2) {
        const int t = n2 / p.group, hl = n2 - t * p.group;
        return out + ((size_t(b) * T + t) * p.hq + g * p.group + hl) * D;
      };
      // Workspace slots: 2 c for the unit that CTA c's run begins in or with, 2 c + 1 for its last one
      // where that is another; of a unit's CTAs only the first can have it as its last.
      const int slot0 = 2 * c0 + (run_begin(c0) >= unit0 ? 0 : 1);
      const size_t slot = cta == c0 ? slot0 : 2 * cta;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const int n2 = grp ? H + j : j;
        if (dim < 0 || n2 >= p.nq) continue;
        const float v = mine[j] + get[j * D + dim];
        if (c0 == c1)
          out_row(n2)[dim] = __float2bfloat16_rn(v / colL[n2]);
        else
          p.part_o[(slot * p.nq + n2) * D + dim] = v;
      }
      if (c0 != c1) {
        if (tid < p.nq) {
          p.part_ml[2 * (slot * p.nq + tid)] = colM[tid];
          p.part_ml[2 * (slot * p.nq + tid) + 1] = colL[tid];
        }
        __threadfence();
        named_bar(3, 256);
        if (tid == 0) *flag = atomicAdd(&p.tickets[unit], 1) == c1 - c0;
        named_bar(3, 256);
        if (*flag) {
          // Last to arrive: out = sum_c F_c o_c / sum_c F_c l_c with F_c = 2^(m_c - max m).
          __threadfence();
          const int pieces = c1 - c0 + 1;
          auto slot_of = [&](int c) { return size_t(c == 0 ? slot0 : 2 * (c0 + c)); };
          float* wts = reinterpret_cast<float*>(smem + Cfg::kOffV16);   // [nq][pieces]
          for (int n2 = warp; n2 < p.nq; n2 += 8) {
            float M = kEmptyMax;
            for (int c = lane; c < pieces; c += 32)
              M = fmaxf(M, __ldcg(&p.part_ml[2 * (slot_of(c) * p.nq + n2)]));
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
            float sum = 0.f;
            for (int c = lane; c < pieces; c += 32) {
              const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) +
                                       slot_of(c) * p.nq + n2);
              const float F = ex2(ml.x - M);
              wts[n2 * pieces + c] = F;
              sum += F * ml.y;
            }
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
            const float inv = 1.f / sum;
            for (int c = lane; c < pieces; c += 32) wts[n2 * pieces + c] *= inv;
          }
          named_bar(3, 256);
          for (int e = tid; e < p.nq * (D / 4); e += 256) {
            const int n2 = e / (D / 4), d = 4 * (e - n2 * (D / 4));
            const float* w = wts + n2 * pieces;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int c = 0; c < pieces; ++c) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(
                  p.part_o + (slot_of(c) * p.nq + n2) * D + d));
              acc.x += w[c] * v.x;
              acc.y += w[c] * v.y;
              acc.z += w[c] * v.z;
              acc.w += w[c] * v.w;
            }
            const uint2 pk = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
            *reinterpret_cast<uint2*>(out_row(n2) + d) = pk;
          }
          if (tid == 0) p.tickets[unit] = 0;
        }
      }
      named_bar(3, 256);   // the exchange buffers and columns are free again
      unit0 = unit1;
      it0 += uint32_t(tiles);
      vs0 += uint32_t(tiles) % VS;
      vround0 += uint32_t(tiles) / VS;
      if (vs0 >= VS) {
        vs0 -= VS;
        ++vround0;
      }
      at.left -= tiles;
      if (at.left > 0) next_unit(at);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
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
  cfg.blockDim = dim3(384, 1, 1);
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
