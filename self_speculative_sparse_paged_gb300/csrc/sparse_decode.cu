// Sparse draft-decode attention: one draft step over the selected positions.
//
// "Vegas: Self-Speculative Decoding with Verification-Guided Sparse
// Attention", gist.science technical summary: §2 "Core mechanism" (the draft
// phase attends only to the critical KV entries selected from the previous
// verification) and §3 "Implementation" (PagedAttention with a page size of
// one token, the selected token indices passed as page indices).
//
// Here the selected positions stay logical token positions: each is mapped
// through the block table of the 16-token paged cache, so the same cache
// serves verify and draft.  One thread-block cluster of CL CTAs per
// (KV head, sequence); CTA r owns a contiguous range of the unit's list
// "T then tail".  It first resolves every entry of its range to a cache row
// (position -> page -> row) in shared memory, then each warp gathers 16-entry
// groups with one 1-D bulk copy per K row and per V row (lanes 0-15 K, 16-31
// V) into padded rows and runs the same warp core as the verify kernel with
// the G query heads of the group as the tile's columns.  The CTAs' softmax
// states meet in distributed shared memory: each CTA pushes the slices of its
// state to the CTAs that own them, then merges and writes the slice it owns,
// with no global scratch and no second pass.
#include "draft_cluster.cuh"
#include "kernels.h"
#include "split_merge.cuh"

namespace vegas {

template <int D, int NT>
struct SparseCfg {
  // Warps, each with two 16-row groups in flight: sixteen at head_dim 64 (a
  // group is half the bytes of a head_dim-128 one; 3% faster than eight warps
  // with four groups), twelve at head_dim 128 with one column tile (3% faster
  // than eight with three), eight with two column tiles (the shared memory
  // holds no more there).  More warps keep the same bytes in flight with more
  // groups computed at once.
  static constexpr int kWarps = D == 64 ? 16 : (NT == 1 ? 12 : kAttnWarps);
  static constexpr int kStages = 2;
  static constexpr int kRow = D * 2 + 16;           // padded row stride
  static constexpr int kTile = 16 * kRow;
  static constexpr int kStage = 2 * kTile;
  static constexpr int kMaxRows = kMaxSparseRowsPerCta;
  static constexpr size_t kStageBytes = size_t(kWarps) * kStages * kStage;
};

template <int D, int NT>
constexpr size_t sparse_smem_layout_bytes() {
  using Cfg = SparseCfg<D, NT>;
  return Cfg::kStageBytes                                          // stages
         + size_t(NT) * 8 * (2 * D + 16)                           // Q tile
         + (size_t(Cfg::kWarps) * Cfg::kStages + 1) * 8            // mbarriers (+ receive)
         + size_t(Cfg::kMaxRows) * 4                               // row table
         + DraftCluster<D, NT * 8>::kBytes                         // states of this CTA and of its peers
         + 1024;
}
static_assert(sparse_smem_layout_bytes<128, 1>() <= 227 * 1024 &&
                  sparse_smem_layout_bytes<128, 2>() <= 227 * 1024 &&
                  sparse_smem_layout_bytes<64, 1>() <= 227 * 1024 &&
                  sparse_smem_layout_bytes<64, 2>() <= 227 * 1024,
              "shared memory of a draft CTA");

template <int D, int NT>
__global__ void __launch_bounds__(SparseCfg<D, NT>::kWarps * 32, 1)
    sparse_decode_kernel(const SparseParams p) {
  constexpr int W = SparseCfg<D, NT>::kWarps;
  constexpr int NTH = W * 32;
  constexpr int NPAD = NT * 8;
  constexpr int STAGES = SparseCfg<D, NT>::kStages;
  constexpr int ROW = SparseCfg<D, NT>::kRow;
  constexpr int TILE = SparseCfg<D, NT>::kTile;
  constexpr int STAGE = SparseCfg<D, NT>::kStage;
  constexpr int QROW = 2 * D + 16;
  using Tile = PaddedTile<D>;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* stage_area = smem;
  uint8_t* qs = smem + SparseCfg<D, NT>::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(qs + NPAD * QROW);
  uint64_t* recv_bar = bars + W * STAGES;   // the cluster's receive barrier
  int32_t* rows = reinterpret_cast<int32_t*>(recv_bar + 1);
  DraftCluster<D, NPAD> peers;
  peers.begin(recv_bar, p.group);
  griddep_begin();
  peers.set_areas(rows + SparseCfg<D, NT>::kMaxRows);
  const int rank = peers.rank;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int unit = b * p.hkv + g;
  const int cap = p.max_pages * 16;

  // The selected positions of this CTA's range are requested together with
  // k_b and the tail (entries past k_b are replaced below), so the index and
  // length loads take one round trip.
  constexpr int kPer = (SparseCfg<D, NT>::kMaxRows + NTH - 1) / NTH;   // entries a thread
  const int rbeg = rank * p.rows_per_split;
  int pos[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * NTH, e = rbeg + i;
    pos[u] = (i < p.rows_per_split && e < p.k_max) ? __ldcg(&p.idx[size_t(unit) * p.k_max + e]) : 0;
  }
  int kb = p.k_per_seq[b];
  if (kb < 0 || kb > p.k_max) {
    if (tid == 0 && g == 0 && rank == 0) set_error(p.err, kErrDeviceFault);
    kb = max(0, min(kb, p.k_max));
  }
  const int tstart = p.tail_start[b];
  const int tlen = max(0, p.tail_len[b]);
  const int total = kb + tlen;
  const int rend = min(rbeg + p.rows_per_split, total);
  const int nrows = max(0, rend - rbeg);

  // The draft queries are requested with the indices and lengths, so their
  // load overlaps the block-table loads below (one 16-byte chunk per thread).
  constexpr int QCH = NPAD * (D / 8);
  static_assert(QCH <= NTH, "one Q chunk per thread");
  uint4 qchunk = make_uint4(0, 0, 0, 0);
  if (tid < QCH && tid / (D / 8) < p.group)
    qchunk = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p.q) +
                                            (size_t(b) * p.hq + g * p.group + tid / (D / 8)) * D)
        [tid % (D / 8)];

  if (tid == 0) {
    // one arrival per lane per stage use: each lane's cp.async copies signal it
    for (int i = 0; i < W * STAGES; ++i) mbar_init(smem_u32(&bars[i]), 32);
    fence_mbar_init();
  }
  // Entry e of the list: T[e] for e < k_b, else tail_start + (e - k_b).
  // Resolved in batches: every index of a thread (loaded above), then every
  // page load.
  {
    int phys[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = tid + u * NTH;
      const int e = rbeg + i;
      if (i >= nrows) pos[u] = 0;
      else if (e >= kb) pos[u] = tstart + (e - kb);
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (pos[u] < 0 || pos[u] >= cap) {
        set_error(p.err, kErrDeviceFault);
        pos[u] = 0;
      }
      phys[u] = tid + u * NTH < nrows ? __ldg(&p.block_table[size_t(b) * p.max_pages + (pos[u] >> 4)]) : 0;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = tid + u * NTH;
      if (i < nrows) {
        if (phys[u] < 0 || phys[u] >= p.num_pages) {
          set_error(p.err, kErrDeviceFault);
          phys[u] = 0;
        }
        rows[i] = (phys[u] * p.hkv + g) * 16 + (pos[u] & 15);
      }
    }
  }
  if (tid < QCH)
    *reinterpret_cast<uint4*>(qs + (tid / (D / 8)) * QROW + (tid % (D / 8)) * 16) = qchunk;
  __syncthreads();

  const int ngroups = (nrows + 15) / 16;
  const int nmy = warp < ngroups ? (ngroups - warp + W - 1) / W : 0;
  const uint32_t stage0 = smem_u32(stage_area + warp * STAGES * STAGE);
  const uint32_t bar0 = smem_u32(&bars[warp * STAGES]);
  const __nv_bfloat16* kc = reinterpret_cast<const __nv_bfloat16*>(p.k_cache);
  const __nv_bfloat16* vc = reinterpret_cast<const __nv_bfloat16*>(p.v_cache);

  // The warp copies the group's 16 K rows and 16 V rows with 16-byte cp.async
  // (consecutive lanes cover consecutive 16-byte chunks of a row); rows past
  // the range repeat the group's first row (masked later).  Each lane then
  // arrives on the stage barrier when its own copies have landed.
  constexpr int CPR = D / 8;                       // 16-byte chunks per row
  auto issue = [&](int i) {
    const int grp = warp + i * W;
    const int s = i % STAGES;
#pragma unroll
    for (int j = 0; j < (32 * CPR) / 32; ++j) {
      const int c = lane + 32 * j;                 // chunk of the 32 rows (K rows, then V rows)
      const int r32 = c / CPR, cc = c % CPR;
      const int r = r32 & 15;
      const int li = grp * 16 + r;
      const int row = rows[li < nrows ? li : grp * 16];
      const __nv_bfloat16* src = (r32 < 16 ? kc : vc) + size_t(row) * D + cc * 8;
      cp_async16(stage0 + s * STAGE + (r32 < 16 ? 0 : TILE) + r * ROW + cc * 16, src);
    }
    cp_async_arrive_noinc(bar0 + s * 8);
  };
  for (int i = 0; i < min(STAGES, nmy); ++i) issue(i);

  uint32_t qf[D / 16][NT][2];
  load_q_frags<D, NT>(smem_u32(qs), qf);
  WarpState<D, NT> st;
  st.init();

  int done = 0;
  bool ok = true;
  for (; done < nmy; ++done) {
    const int i = done;
    const int s = i % STAGES;
    if (!mbar_wait_bounded(bar0 + s * 8, (i / STAGES) & 1)) {
      ok = false;
      break;
    }
    const int grp = warp + i * W;
    const uint32_t kb_s[1] = {stage0 + s * STAGE};
    const uint32_t vb_s[1] = {stage0 + s * STAGE + TILE};
    float sc[1][NT][4];
    tile_scores<D, NT, 1, Tile>(kb_s, qf, sc);
    float x[1][NT][4];
    const int valid = nrows - grp * 16;   // rows of this group inside the range
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = (lane >> 2) + 8 * (k >> 1);
        const int n = nt * 8 + 2 * (lane & 3) + (k & 1);
        x[0][nt][k] = (r < valid && n < p.group) ? sc[0][nt][k] * p.scale_log2 : -INFINITY;
      }
    tile_softmax_pv<D, NT, 1, Tile>(st, x, vb_s);
    __syncwarp();
    if (i + STAGES < nmy) {
      fence_proxy_async_smem();
      issue(i + STAGES);
    }
  }
  if (!ok) {
    if (lane == 0) set_error(p.err, kErrDeviceTimeout);
    for (int j = done; j < min(done + STAGES, nmy); ++j)
      (void)mbar_wait_bounded(bar0 + (j % STAGES) * 8, (j / STAGES) & 1);
  }
  reduce_row_sums<D, NT>(st);
  __syncthreads();
  cta_merge_to_smem<D, NT, W>(st, stage_area, SparseCfg<D, NT>::kStageBytes, p.group, peers.m, peers.l,
                              peers.o);
  __syncthreads();   // the pushes below read elements other threads merged

  peers.template merge<NTH, false>(
      reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t(b) * p.hq + g * p.group) * D, p.err);
}

template <int D, int NT>
static cudaError_t launch_sparse_one(const SparseParams& p, int batch, cudaStream_t stream,
                                     int* clusters) {
  return launch_draft_cluster<sparse_decode_kernel<D, NT>>(p, sparse_smem_layout_bytes<D, NT>(),
                                                           SparseCfg<D, NT>::kWarps * 32, batch, stream,
                                                           clusters);
}

static cudaError_t launch_sparse_any(const SparseParams& p, int head_dim, int ntiles, int batch,
                                     cudaStream_t stream, int* clusters) {
  if (p.num_splits < 1 || p.num_splits > kMaxSparseCluster) return cudaErrorInvalidValue;
  if (head_dim == 128) {
    if (ntiles == 1) return launch_sparse_one<128, 1>(p, batch, stream, clusters);
    if (ntiles == 2) return launch_sparse_one<128, 2>(p, batch, stream, clusters);
  } else if (head_dim == 64) {
    if (ntiles == 1) return launch_sparse_one<64, 1>(p, batch, stream, clusters);
    if (ntiles == 2) return launch_sparse_one<64, 2>(p, batch, stream, clusters);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_sparse(const SparseParams& p, int head_dim, int ntiles, int batch,
                          cudaStream_t stream) {
  return launch_sparse_any(p, head_dim, ntiles, batch, stream, nullptr);
}

int sparse_max_active_clusters(int head_dim, int ntiles, int cluster) {
  return resident_draft_clusters<SparseParams, launch_sparse_any>(head_dim, ntiles, cluster);
}

}  // namespace vegas
