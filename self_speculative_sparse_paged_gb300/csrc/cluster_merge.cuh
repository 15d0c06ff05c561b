// The on-chip end of the tcgen05 verify kernels: the partial softmax states of a unit's splits,
// one for each softmax group of each CTA, meet in the CTAs of the unit's cluster.
#pragma once

#include <cooperative_groups.h>

#include "kernels.h"
#include "split_merge.cuh"

namespace vegas {

namespace cg = cooperative_groups;

// Cluster-wide barrier of every thread (release / acquire): shared-memory
// writes before it, local or remote, are visible to every CTA after it.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Bytes of merge_on_chip's two areas.
template <int D, int NQC>
__host__ __device__ constexpr int merge_receive_bytes() {
  return 2 * (NQC + kMaxVerifyCluster) * (D + 4) * 4;
}
constexpr int kMergeWeightBytes = (64 * 2 * kMaxVerifyCluster + 2 * 64 + 64 * 32) * 4;

// Split-KV merge on chip (one split: a cluster of one CTA).  Row n of the
// output belongs to cluster rank n % S, which receives in `area`, at
// slot n / S, the 2S partial states of the row (state 2 * rank + group of
// each sender, O[D] then m and l), pushed with distributed-shared-memory
// stores; one cluster barrier publishes them and each rank merges its rows
// from local shared memory: O = sum_q 2^(m_q - M) O_q / sum_q 2^(m_q - M) l_q
// with M = max_q m_q.  Nothing reads another CTA's shared memory, so no
// barrier precedes the exit.
//
// Called by all NTH threads of every CTA of the cluster once no CTA uses `area` or `wts` any more
// (a cluster barrier before this call).  grp: the thread's softmax group, or -1; dim: the head
// dimension whose O^T row it holds in o, or -1; Mg, Lg: maximum and row sum of column `col` where
// col < nq.  area, wts: merge_receive_bytes and kMergeWeightBytes of shared memory, the same
// addresses in every CTA.
template <int D, int NQC, int NTH, class OutRow>
__device__ __forceinline__ void merge_on_chip(const VerifyParams& p, int unit, int split, int grp,
                                              int dim, int col, const float (&o)[NQC], float Mg,
                                              float Lg, uint8_t* area, float* wts, int* flag,
                                              OutRow out_row) {
  constexpr int RS = D + 4;   // one received state: O[D], m, l, padding to 16 bytes
  static_assert(2 * kMaxVerifyCluster <= 32, "one lane per state in the weight pass");
  cg::cluster_group cluster = cg::this_cluster();
  const int S = p.cluster_merge ? p.cluster_size : 1, r = (int)cluster.block_rank();
  const int C = p.num_splits / S, c = split / S;   // clusters of the unit, this one's index
  const float* recv = reinterpret_cast<const float*>(area);
  const uint32_t area_s = smem_u32(area);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (grp >= 0) {
    const int q = 2 * r + grp;
    int owner = 0, slot = 0;
#pragma unroll
    for (int n = 0; n < NQC; ++n) {
      if (n < p.nq && dim >= 0)
        st_cluster_f32(cluster_map(area_s + 4 * ((slot * 2 * S + q) * RS + dim), owner), o[n]);
      if (++owner == S) {
        owner = 0;
        ++slot;
      }
    }
    if (col < p.nq) {
      const uint32_t dst =
          cluster_map(area_s + 4 * (((col / S) * 2 * S + q) * RS + D), col % S);
      st_cluster_f32(dst, Mg);
      st_cluster_f32(dst + 4, Lg);
    }
  }
  cluster_sync_all();
  const int nown = r < p.nq ? (p.nq - r + S - 1) / S : 0;
  // Weights 2^(m_q - M) / sum_q' 2^(m_q' - M) l_q' of the 2S states of each
  // owned row (one warp per row, lane q), into `wts` [nown][2S], with the
  // row's cluster-level maximum M and sum (used when C > 1) ...
  // (nown <= NQC <= 64 rows, 2S <= 32 states, C <= 32 clusters)
  float* rowml = wts + 64 * 2 * kMaxVerifyCluster;           // [nown][2]
  for (int k = warp; k < nown; k += NTH / 32) {
    const float* st = recv + k * 2 * S * RS;
    const bool has = lane < 2 * S;
    const float m = has ? st[lane * RS + D] : kEmptyMax;
    const float l = has ? st[lane * RS + D + 1] : 0.f;
    float M = m;
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
    const float f = has ? ex2(m - M) : 0.f;
    float Lsum = f * l;
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) Lsum += __shfl_xor_sync(0xffffffffu, Lsum, o2);
    if (has) wts[k * 2 * S + lane] = Lsum > 0.f ? f / Lsum : 0.f;
    if (lane == 0) {
      rowml[2 * k] = M;
      rowml[2 * k + 1] = Lsum;
    }
  }
  __syncthreads();
  // ... then four output elements per thread: sum_q w_q O_q[d .. d + 3]
  for (int e = tid; e < nown * (D / 4); e += NTH) {
    const int k = e / (D / 4), d = 4 * (e - k * (D / 4));
    const float* st = recv + k * 2 * S * RS + d;
    const float* wk = wts + k * 2 * S;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int q = 0; q < 2 * S; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(st + q * RS);
      const float wq = wk[q];
      acc.x += wq * v.x;
      acc.y += wq * v.y;
      acc.z += wq * v.z;
      acc.w += wq * v.w;
    }
    if (C == 1) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
      uint2 pk;
      pk.x = *reinterpret_cast<const uint32_t*>(&lo);
      pk.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(out_row(r + k * S) + d) = pk;
    } else {
      // this cluster's normalised row, merged across the unit's clusters below
      const size_t row = (size_t(unit) * C + c) * p.nq + (r + k * S);
      *reinterpret_cast<float4*>(p.part_o + row * D + d) = acc;
    }
  }
  if (C > 1) {
    // Cross-cluster merge through the workspace, per owner rank: rank r of
    // every cluster of the unit writes its rows' (o_c, M_c, L_c), takes the
    // ticket of (unit, r), and the last to arrive combines them:
    // out = sum_c F_c o_c / sum_c F_c with F_c = 2^(M_c - max M) L_c.
    for (int k = tid; k < nown; k += NTH) {
      const size_t row = (size_t(unit) * C + c) * p.nq + (r + k * S);
      p.part_ml[2 * row] = rowml[2 * k];
      p.part_ml[2 * row + 1] = rowml[2 * k + 1];
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) *flag = atomicAdd(&p.tickets[unit * S + r], 1) == C - 1;
    __syncthreads();
    if (*flag) {
      __threadfence();
      float* w2 = rowml + 2 * 64;   // [nown][C]
      for (int k = warp; k < nown; k += NTH / 32) {
        const bool has = lane < C;
        const size_t row = (size_t(unit) * C + lane) * p.nq + (r + k * S);
        const float m = has ? __ldcg(&p.part_ml[2 * row]) : kEmptyMax;
        const float l = has ? __ldcg(&p.part_ml[2 * row + 1]) : 0.f;
        float M = m;
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o2));
        const float F = has ? ex2(m - M) * l : 0.f;
        float Fs = F;
#pragma unroll
        for (int o2 = 16; o2 > 0; o2 >>= 1) Fs += __shfl_xor_sync(0xffffffffu, Fs, o2);
        if (has) w2[k * C + lane] = Fs > 0.f ? F / Fs : 0.f;
      }
      __syncthreads();
      for (int e = tid; e < nown * (D / 4); e += NTH) {
        const int k = e / (D / 4), d = 4 * (e - k * (D / 4));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < C; ++q) {
          const size_t row = (size_t(unit) * C + q) * p.nq + (r + k * S);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part_o + row * D + d));
          const float wq = w2[k * C + q];
          acc.x += wq * v.x;
          acc.y += wq * v.y;
          acc.z += wq * v.z;
          acc.w += wq * v.w;
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z, acc.w);
        uint2 pk;
        pk.x = *reinterpret_cast<const uint32_t*>(&lo);
        pk.y = *reinterpret_cast<const uint32_t*>(&hi);
        *reinterpret_cast<uint2*>(out_row(r + k * S) + d) = pk;
      }
      if (tid == 0) p.tickets[unit * S + r] = 0;
    }
  }
}

}  // namespace vegas
