// What the draft kernels of both caches share: the CTAs of a list (one thread-block cluster) joining their
// softmax states, the launch of such a kernel, and how many of its clusters can be resident at once.
//
// CTA r owns the output elements [r * per, (r + 1) * per) of the G x D (per a multiple of four).  Every CTA
// pushes the slices of its state to their owners' receive areas with asynchronous distributed-shared-memory
// stores, 16 bytes each (four elements of one owner), and its G row maxima and sums to every CTA, one (CTA,
// row) pair a thread; each store counts against the owner's receive barrier, and an owner merges as soon as
// that barrier has counted every byte it expects:
//   M = max_r m_r, O = sum_r 2^(m_r - M) O_r / sum_r 2^(m_r - M) l_r.
// Spreading the pushes over the threads (rather than one thread a row looping over the CTAs, four bytes a
// store) took the batch-1 step over the bf16 cache from 5.75 to 5.3 us.
#pragma once

#include <cooperative_groups.h>

#include "kernels.h"
#include "vegas_common.cuh"

namespace vegas {

// NPAD: rows of the state, the G query heads rounded up to 8.
template <int D, int NPAD>
struct DraftCluster {
  int rank, ctas;    // this CTA, of how many
  int nel, per;      // output elements of the unit (G x D), and of each CTA
  int group;
  uint64_t* bar;     // completes when every peer's state has landed
  float *m, *l, *o;  // this CTA's state: [NPAD], [NPAD], [NPAD][D]
  // received: [ctas][per] output slices (16-byte aligned: they arrive in 16-byte stores; ctas * per <=
  // G * D + 4 * ctas - 1), [ctas][NPAD] maxima and row sums
  float *all_o, *all_m, *all_l;

  // Shared memory behind `at` that set_areas takes.
  static constexpr size_t kBytes = size_t(NPAD) * (D + 2) * 4                          // CTA partial
                                   + (size_t(NPAD) * D + 4 * kMaxSparseCluster) * 4 + 16   // slices
                                   + size_t(kMaxSparseCluster) * NPAD * 2 * 4;         // m, l

  // At entry: sets up the receive barrier, and begins the cluster barrier's phase (its shared memory may
  // receive other CTAs' stores once every CTA has arrived).
  __device__ __forceinline__ void begin(uint64_t* receive, int heads) {
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    rank = (int)cluster.block_rank();
    ctas = (int)cluster.num_blocks();
    group = heads;
    nel = heads * D;
    per = ((nel + ctas - 1) / ctas + 3) & ~3;
    bar = receive;
    if (threadIdx.x == 0) {
      // Every CTA sends this one its slice of the partial output and its G row
      // maxima and sums: 4 * ctas * (slice + 2G) bytes, counted by st.async.
      mbar_init(smem_u32(bar), 1);
      const int mine = max(0, min(per, nel - rank * per));
      mbar_arrive_expect_tx(smem_u32(bar), uint32_t(4 * ctas * (mine + 2 * group)));
      fence_mbar_init();
    }
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
  __device__ __forceinline__ void set_areas(void* at) {
    m = reinterpret_cast<float*>(at);
    l = m + NPAD;
    o = l + NPAD;
    all_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(o + NPAD * D) + 15) & ~uintptr_t(15));
    all_m = all_o + NPAD * D + 4 * kMaxSparseCluster;
    all_l = all_m + kMaxSparseCluster * NPAD;
  }

  // Called by all NTH threads when the CTA's state is in m, l, o.  out: the unit's first row (rows of D).
  // FarSums: a row sum may weigh although 2^(m - M) is below fp32's smallest (the 8-bit cache's, kv8.cuh).
  template <int NTH, bool FarSums>
  __device__ __forceinline__ void merge(__nv_bfloat16* out, int* err) const {
    const int tid = threadIdx.x;
    // The receive areas are used by nothing else, so only the barrier phase begun at entry (every CTA has
    // started, its receive barrier is ready) precedes the stores, and no cluster barrier follows them.
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    {
      const uint32_t o_s = smem_u32(all_o), m_s = smem_u32(all_m), l_s = smem_u32(all_l);
      const uint32_t rb = smem_u32(bar);
      for (int e = 4 * tid; e < nel; e += 4 * NTH) {   // 4 | nel (D is 64 or 128)
        const int owner = e / per;                      // e .. e + 3 share it
        st_async_f32x4(cluster_map(o_s + 4 * (rank * per + e - owner * per), owner), o[e], o[e + 1],
                       o[e + 2], o[e + 3], cluster_map(rb, owner));
      }
      static_assert(kMaxSparseCluster * 16 <= NTH, "one (CTA, row) pair a thread");
      const int t = NTH - 1 - tid;   // the last threads, which carry fewer elements
      if (t < ctas * group) {        // ctas * G <= 256 <= NTH
        const int r = t / group, n = t - r * group;
        st_async_f32(cluster_map(m_s + 4 * (rank * NPAD + n), r), m[n], cluster_map(rb, r));
        st_async_f32(cluster_map(l_s + 4 * (rank * NPAD + n), r), l[n], cluster_map(rb, r));
      }
    }
    if (!mbar_wait_cluster_bounded(smem_u32(bar), 0)) {
      if (tid == 0) set_error(err, kErrDeviceTimeout);
      return;
    }
    constexpr int R = kMaxSparseCluster;
    const int e0 = rank * per, e1 = min(nel, e0 + per);
    for (int e = e0 + tid; e < e1; e += NTH) {
      const int n = e / D;
      float mr[R], lr[R], v[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        mr[r] = -INFINITY;
        lr[r] = v[r] = 0.f;
        if (r < ctas) {
          mr[r] = all_m[r * NPAD + n];
          lr[r] = all_l[r * NPAD + n];
          v[r] = all_o[r * per + e - e0];
        }
      }
      float M = -INFINITY;
#pragma unroll
      for (int r = 0; r < R; ++r) M = fmaxf(M, mr[r]);
      float L = 0.f, a = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (FarSums) {
          const float h = r < ctas ? half_weight(mr[r] - M) : 0.f;
          L += lr[r] * h * h;
          a += h * h * v[r];
        } else {
          const float f = r < ctas ? ex2(mr[r] - M) : 0.f;
          L += f * lr[r];
          a += f * v[r];
        }
      }
      out[size_t(n) * D + (e % D)] = __float2bfloat16_rn(L > 0.f ? a / L : 0.f);
    }
  }
};

// Launches Kernel with clusters of p.num_splits CTAs, or with `clusters` set, reports how many of them can be
// resident at once.
template <auto Kernel, class Params>
cudaError_t launch_draft_cluster(const Params& p, size_t smem, int threads, int batch, cudaStream_t stream,
                                 int* clusters) {
  static std::atomic<uint32_t> configured{0};
  cudaError_t e = once_per_device(configured, [&] {
    cudaError_t r = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_splits, p.hkv, batch);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.num_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = clusters ? 1 : 2;
  if (clusters) return cudaOccupancyMaxActiveClusters(clusters, Kernel, &cfg);
  return cudaLaunchKernelEx(&cfg, Kernel, p);
}

// How many clusters of `cluster` CTAs of a draft kernel can be resident at once, asked once per device and
// shape.  Launch(p, head_dim, ntiles, batch, stream, clusters): the kernel's launch, as above.
template <class Params, auto Launch>
int resident_draft_clusters(int head_dim, int ntiles, int cluster) {
  if (cluster < 1 || cluster > kMaxSparseCluster || ntiles < 1 || ntiles > 2) return 0;
  constexpr int kDevices = 32;
  // [device][head_dim 64/128][ntiles][cluster]: 0 unknown, -1 none, else the count
  static std::atomic<int> cache[kDevices][2][3][kMaxSparseCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  std::atomic<int>& slot = cache[dev][head_dim == 128 ? 1 : 0][ntiles][cluster];
  int c = slot.load(std::memory_order_acquire);
  if (c == 0) {
    Params p{};
    p.hkv = 1;
    p.num_splits = cluster;
    int n = 0;
    if (Launch(p, head_dim, ntiles, 1, 0, &n) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    c = n > 0 ? n : -1;
    slot.store(c, std::memory_order_release);
  }
  return c > 0 ? c : 0;
}

}  // namespace vegas
