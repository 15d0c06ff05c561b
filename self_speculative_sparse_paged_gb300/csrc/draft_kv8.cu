// Draft attention over the paged cache in 8 bits: one draft step over the selected positions.
//
// The list "T then tail" of a (sequence, KV head) is split over one thread-block cluster, as in the
// bf16 draft kernel; here every CTA resolves its entries to cache rows and to the two scale
// exponents of their blocks, each warp gathers 16 rows of K and V at a time with 16-byte copies
// (D bytes a row), and the warp core of kv8_core.cuh turns them into logits and weighted sums.  The
// CTAs' softmax states meet in distributed shared memory, with no global scratch and no second pass.
//
// What bounds it: rows at random places come at 4.7 TB/s where they have 128 bytes and at 2.3 where
// they have 64 (a plain gather of 4 million of them), and short lists at the length of the chain
// index -> page -> row -> merge.  5.8 us at 1,645 entries x 8 heads of 128; 4 lists of 3,933
// entries x 8 heads of 64: 11.3; 8 of 2,908 x 8 of 128: 17.0; 4 of 10,008 x 8 of 128: 22.6.
#include "draft_cluster.cuh"
#include "kernels.h"
#include "kv8_core.cuh"
#include "split_merge.cuh"

namespace vegas {

// W warps, each with two 16-row groups in flight.  Long lists: sixteen, twelve where two column tiles
// of head_dim 128 leave no registers for more (8 -> 16: 26.8 -> 22.4 us for 4 lists of 10,008
// entries).  Up to kFewRows entries a CTA eight have them all in flight too, and merge fewer states
// (16 -> 8: 5.9 -> 5.6 us at 1,645 entries; at head_dim 64, with half the state, 4.9 -> 5.3).
constexpr int kFewWarps = 8, kFewRows = 2 * 16 * kFewWarps;
template <int D, int NT>
constexpr int draft_kv8_warps(bool few) { return D == 64 ? 16 : few ? kFewWarps : NT == 2 ? 12 : 16; }

template <int D, int NT, int W>
struct DraftKv8Cfg {
  static constexpr int kWarps = W;
  static constexpr int kStages = 2;
  static constexpr int kTile = 16 * D;
  static constexpr int kStage = 2 * kTile;
  static constexpr int kMaxRows = kMaxDraftKv8Rows;
  static constexpr size_t kStageBytes = size_t(kWarps) * kStages * kStage;
};

template <int D, int NT, int W>
constexpr size_t draft_kv8_smem_bytes() {
  using Cfg = DraftKv8Cfg<D, NT, W>;
  return Cfg::kStageBytes                                          // stages
         + (size_t(Cfg::kWarps) * Cfg::kStages + 1) * 8            // mbarriers (+ receive)
         + size_t(Cfg::kMaxRows) * 6                               // row table, scale exponents
         + DraftCluster<D, NT * 8>::kBytes                         // states of this CTA and of its peers
         + 1024;
}
static_assert(draft_kv8_smem_bytes<128, 1, 16>() <= 227 * 1024 &&
                  draft_kv8_smem_bytes<128, 2, 12>() <= 227 * 1024 &&
                  draft_kv8_smem_bytes<64, 1, 16>() <= 227 * 1024 &&
                  draft_kv8_smem_bytes<64, 2, 16>() <= 227 * 1024,
              "shared memory of a draft CTA");

template <int D, int NT, int W>
__global__ void __launch_bounds__(DraftKv8Cfg<D, NT, W>::kWarps * 32, 1)
    draft_kv8_kernel(const DraftKv8Params p) {
  constexpr int NTH = W * 32;
  constexpr int NPAD = NT * 8;
  constexpr int STAGES = DraftKv8Cfg<D, NT, W>::kStages;
  constexpr int TILE = DraftKv8Cfg<D, NT, W>::kTile;
  constexpr int STAGE = DraftKv8Cfg<D, NT, W>::kStage;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* stage_area = smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + DraftKv8Cfg<D, NT, W>::kStageBytes);
  uint64_t* recv_bar = bars + W * STAGES;   // the cluster's receive barrier
  int32_t* rows = reinterpret_cast<int32_t*>(recv_bar + 1);
  // entry i's exponents, K's in the low byte and V's in the high one
  uint16_t* exps = reinterpret_cast<uint16_t*>(rows + DraftKv8Cfg<D, NT, W>::kMaxRows);
  DraftCluster<D, NPAD> peers;
  peers.begin(recv_bar, p.group);
  griddep_begin();
  peers.set_areas(exps + DraftKv8Cfg<D, NT, W>::kMaxRows);
  const int rank = peers.rank;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y, b = blockIdx.z;
  const int unit = b * p.hkv + g;
  const int cap = p.max_pages * 16;

  // The selected positions of this CTA's range are requested together with
  // k_b and the tail (entries past k_b are replaced below), so the index and
  // length loads take one round trip.
  constexpr int kPer = (DraftKv8Cfg<D, NT, W>::kMaxRows + NTH - 1) / NTH;   // entries a thread
  // (a split's own length ends the walks over the table early: 6.3 -> 5.9 us at 1,645 entries)
  auto past = [&](int u) { return u * NTH >= p.rows_per_split; };
  const int rbeg = rank * p.rows_per_split;
  int pos[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    if (past(u)) break;
    const int i = tid + u * NTH, e = rbeg + i;
    pos[u] = (i < p.rows_per_split && e < p.k_max) ? __ldcg(&p.idx[size_t(unit) * p.k_max + e]) : 0;
  }
  int kb = p.k_per_seq[b];
  if (kb < 0 || kb > p.k_max) {
    if (tid == 0 && g == 0 && rank == 0) set_error(p.err, kErrDeviceFault);
    kb = max(0, min(kb, p.k_max));
  }
  const int tstart = p.tail_start[b];
  int tlen = max(0, p.tail_len[b]);
  if (tlen > p.max_tail) {   // (before it is added to anything: it may be as large as an int)
    if (tid == 0 && g == 0 && rank == 0) set_error(p.err, kErrDeviceFault);
    tlen = p.max_tail;
  }
  const int total = kb + tlen;
  const int rend = min(rbeg + p.rows_per_split, total);
  const int nrows = max(0, rend - rbeg);

  if (tid == 0) {
    // one arrival per lane per stage use: each lane's cp.async copies signal it
    for (int i = 0; i < W * STAGES; ++i) mbar_init(smem_u32(&bars[i]), 32);
    fence_mbar_init();
  }
  // Entry e of the list: T[e] for e < k_b, else tail_start + (e - k_b).
  // Resolved in batches: every index of a thread (loaded above), then every
  // page load.
  uint8_t ek[kPer], ev[kPer];   // the entries' scale bytes
  {
    int phys[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (past(u)) break;
      const int i = tid + u * NTH;
      const int e = rbeg + i;
      if (i >= nrows) pos[u] = 0;
      else if (e >= kb) pos[u] = tstart + (e - kb);
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (past(u)) break;
      if (pos[u] < 0 || pos[u] >= cap) {
        set_error(p.err, kErrDeviceFault);
        pos[u] = 0;
      }
      phys[u] = tid + u * NTH < nrows ? __ldg(&p.block_table[size_t(b) * p.max_pages + (pos[u] >> 4)]) : 0;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (past(u)) break;
      const int i = tid + u * NTH;
      if (i < nrows) {
        if (phys[u] < 0 || phys[u] >= p.num_pages) {
          set_error(p.err, kErrDeviceFault);
          phys[u] = 0;
        }
        rows[i] = (phys[u] * p.hkv + g) * 16 + (pos[u] & 15);
      }
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (past(u)) break;
      if (tid + u * NTH >= nrows) continue;
      const size_t block = size_t(phys[u]) * p.hkv + g;
      ek[u] = __ldg(&p.k_scale[block]);
      ev[u] = __ldg(&p.v_scale[block]);
    }
  }
  __syncthreads();

  const int ngroups = (nrows + 15) / 16;
  const int nmy = warp < ngroups ? (ngroups - warp + W - 1) / W : 0;
  const uint32_t stage0 = smem_u32(stage_area + warp * STAGES * STAGE);
  const uint32_t bar0 = smem_u32(&bars[warp * STAGES]);
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(p.k_cache);
  const uint8_t* vc = reinterpret_cast<const uint8_t*>(p.v_cache);

  // The warp copies the group's 16 K rows and 16 V rows with 16-byte cp.async
  // (consecutive lanes cover consecutive 16-byte chunks of a row); rows past
  // the range repeat the group's first row (masked later).  Each lane then
  // arrives on the stage barrier when its own copies have landed.
  constexpr int CPR = D / 16;                      // 16-byte chunks per row
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
      const uint8_t* src = (r32 < 16 ? kc : vc) + size_t(row) * D + cc * 16;
      cp_async16(stage0 + s * STAGE +
                     (r32 < 16 ? Kv8Rows<D>::k(r, cc) : TILE + Kv8Rows<D>::v(r, cc)),
                 src);
    }
    cp_async_arrive_noinc(bar0 + s * 8);
  };
  for (int i = 0; i < min(STAGES, nmy); ++i) issue(i);

  uint32_t qf[D / 16][NT][2];
  float col[NT][2];   // logit units of column 2 (lane % 4) + e, log2
  // the scale bytes were requested before the first rows; every warp reads its entries' below
  bool deep = false;   // the CTA's range has blocks far below the others
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    if (past(u)) break;
    const int i = tid + u * NTH;
    if (i < nrows) {
      exps[i] = uint16_t(uint8_t(kv8_exponent(ek[u]))) | uint16_t(uint8_t(kv8_exponent(ev[u]))) << 8;
      deep |= kv8_exponent(ev[u]) < kKv8Deep;
    }
  }
  kv8_load_q<D, NT>(reinterpret_cast<const __nv_bfloat16*>(p.q) + (size_t(b) * p.hq + g * p.group) * D,
                    p.group, qf, col);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) col[nt][e] *= p.scale_log2;
  deep = __syncthreads_or(deep);
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
    const int valid = nrows - grp * 16;   // rows of this group inside the range
    float z[NT][4];
    kv8_scores<D, NT>(stage0 + s * STAGE, qf, z);
    float unscale[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (lane >> 2) + 8 * j;
      const uint16_t ex = exps[grp * 16 + (r < valid ? r : 0)];
      const int e_v = int8_t(ex >> 8);
      const float f = two_to(int8_t(ex)), zv = r < valid ? float(e_v) : -INFINITY;
      unscale[j] = two_to(-e_v);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)   // (columns past the group have zero queries)
          z[nt][2 * j + e] = fmaf(z[nt][2 * j + e], col[nt][e] * f, zv);
    }
    kv8_softmax_pv<D, NT>(st, z, unscale, deep, stage0 + s * STAGE + TILE);
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
  cta_merge_to_smem<D, NT, W, Kv8Dims<D>, true>(st, stage_area, DraftKv8Cfg<D, NT, W>::kStageBytes,
                                                p.group, peers.m, peers.l, peers.o);
  __syncthreads();   // the pushes below read elements other threads merged

  peers.template merge<NTH, true>(
      reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t(b) * p.hq + g * p.group) * D, p.err);
}

template <int D, int NT, int W>
static cudaError_t launch_draft_kv8_w(const DraftKv8Params& p, int batch, cudaStream_t stream,
                                      int* clusters) {
  return launch_draft_cluster<draft_kv8_kernel<D, NT, W>>(p, draft_kv8_smem_bytes<D, NT, W>(), W * 32, batch,
                                                          stream, clusters);
}

template <int D, int NT>
static cudaError_t launch_draft_kv8_one(const DraftKv8Params& p, int batch, cudaStream_t stream,
                                        int* clusters) {
  // (the count of resident clusters is the larger kernel's)
  return !clusters && p.rows_per_split <= kFewRows
             ? launch_draft_kv8_w<D, NT, draft_kv8_warps<D, NT>(true)>(p, batch, stream, nullptr)
             : launch_draft_kv8_w<D, NT, draft_kv8_warps<D, NT>(false)>(p, batch, stream, clusters);
}

static cudaError_t launch_draft_kv8_any(const DraftKv8Params& p, int head_dim, int ntiles, int batch,
                                        cudaStream_t stream, int* clusters) {
  if (p.num_splits < 1 || p.num_splits > kMaxSparseCluster) return cudaErrorInvalidValue;
  if (head_dim == 128) {
    if (ntiles == 1) return launch_draft_kv8_one<128, 1>(p, batch, stream, clusters);
    if (ntiles == 2) return launch_draft_kv8_one<128, 2>(p, batch, stream, clusters);
  } else if (head_dim == 64) {
    if (ntiles == 1) return launch_draft_kv8_one<64, 1>(p, batch, stream, clusters);
    if (ntiles == 2) return launch_draft_kv8_one<64, 2>(p, batch, stream, clusters);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_draft_kv8(const DraftKv8Params& p, int head_dim, int ntiles, int batch,
                             cudaStream_t stream) {
  return launch_draft_kv8_any(p, head_dim, ntiles, batch, stream, nullptr);
}

int draft_kv8_max_active_clusters(int head_dim, int ntiles, int cluster) {
  return resident_draft_clusters<DraftKv8Params, launch_draft_kv8_any>(head_dim, ntiles, cluster);
}

}  // namespace vegas
