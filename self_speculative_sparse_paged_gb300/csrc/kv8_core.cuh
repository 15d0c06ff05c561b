// Warp-level attention over 16-position groups of 8-bit rows, the counterpart of attn_core.cuh's
// tile_scores and tile_softmax_pv for the draft kernel's 8-bit variant.
//
// Codes become f16 fragments in registers (exact): S^T = K Q^T and O^T += V^T P^T run on
// m16n8k16 f16 with fp32 sums.  What a fragment's k and m indices mean is free as long as both
// operands (and the output) agree, which makes every load a whole chunk of a row:
//   K: lane (r, c) = (lane / 4, lane % 4) reads the 16 codes of dims 64 h + 16 c .. + 15 of
//      positions r and r + 8; word w of them is the k-step (h, w), dims 64 h + 16 c + 4 w + {0..3}.
//   V: lane (r, c) reads the D / 8 codes of dims (D / 8) r .. of positions 2c, 2c + 1, 2c + 8,
//      2c + 9; bytes of two positions are interleaved into pairs, and m-tile mt holds dims
//      (D / 8) r + 2 mt (row r) and + 2 mt + 1 (row r + 8).
//
// Scales: with x the logit in log2 units and V's exponent e_v, z = x + e_v and P = 2^(z - m)
// multiplies V's codes, while the row sum takes P 2^-e_v = 2^(x - m) in fp32 (of a deep block from
// 2^(z - m + kKv8Lift): kv8.cuh).  m is a reference with P <= 2^15 (f16 ends at 65504), at least 7
// below the largest z when it is raised, so that P's f16 grid reaches 2^-31 below the largest and
// its roundings are 2^-11 of each.
#pragma once

#include "attn_core.cuh"
#include "kv8.cuh"

namespace vegas {

constexpr float kKv8Top = 15.f;      // log2 of the largest P
constexpr float kKv8Raise = 7.f;     // log2 of the largest P when the reference is raised

// Where the 16-byte chunk `cc` of row r of a 16-row group lies: no padding, chunks exchanged so
// that the reads above touch every bank once a phase.
template <int D>
struct Kv8Rows {
  __device__ __forceinline__ static uint32_t k(int r, int cc) {
    return D == 128 ? r * 128 + ((cc ^ ((r & 1) << 2)) << 4) : r * 64 + cc * 16;
  }
  __device__ __forceinline__ static uint32_t v(int r, int cc) {
    return D == 128 ? r * 128 + ((cc ^ (r & 6)) << 4)
                    : (r >> 1) * 128 + ((((r & 1) * 4 + cc) ^ (r & 6)) << 4);
  }
};

// The dim of o[mt][.][2 * hi + .] of lane row r (stage_warp_o's map).
template <int D>
struct Kv8Dims {
  __device__ __forceinline__ static int dim(int mt, int r, int hi) {
    return (D / 8) * r + 2 * mt + hi;
  }
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32"
      " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// The group's query heads as f16 fragments, each head scaled by a power of two to a largest
// element in [2^14, 2^15): a bf16 element is then exact in f16 unless it is below 2^-31 of its
// head's largest, and off by at most 2^-39 of that there.  q: the unit's first head (rows of D bf16);
// back[nt][e]: 1 / scale of column 8 nt + 2 (lane % 4) + e.
template <int D, int NT>
__device__ __forceinline__ void kv8_load_q(const __nv_bfloat16* q, int group,
                                           uint32_t (&qf)[D / 16][NT][2], float (&back)[NT][2]) {
  const int lane = threadIdx.x & 31, n = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t w[D / 64][8];
    uint32_t most = 0;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (8 * nt + n < group) {
        const uint4* src = reinterpret_cast<const uint4*>(q + size_t(8 * nt + n) * D + 64 * h + 16 * c);
        lo = src[0];
        hi = src[1];
      }
      const uint32_t all[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[h][i] = all[i];
        most = __vmaxu2(most, all[i] & 0x7fff7fffu);
      }
    }
    most = max(most & 0xffffu, most >> 16);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
    // 2^(14 - n) for a largest element in [2^n, 2^(n + 1))
    const int up = max(-120, min(120, 14 - (int(most >> 7) - 127)));
    const float f = two_to(up), b = two_to(-up);
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        qf[4 * h + i / 2][nt][i & 1] = pack_f16x2(__uint_as_float(w[h][i] << 16) * f,
                                                  __uint_as_float(w[h][i] & 0xffff0000u) * f);
#pragma unroll
    for (int e = 0; e < 2; ++e) back[nt][e] = __shfl_sync(0xffffffffu, b, 4 * (2 * c + e));
  }
}

// S^T of one group.
template <int D, int NT>
__device__ __forceinline__ void kv8_scores(uint32_t k_base, const uint32_t (&qf)[D / 16][NT][2],
                                           float (&s)[NT][4]) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    const uint4 k0 = lds128(k_base + Kv8Rows<D>::k(r, 4 * h + c));
    const uint4 k1 = lds128(k_base + Kv8Rows<D>::k(r + 8, 4 * h + c));
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0, a1, a2, a3;
      f16x2_from_e4m3x4(w0[w], a0, a2);
      f16x2_from_e4m3x4(w1[w], a1, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_f16_16816(s[nt], a0, a1, a2, a3, qf[4 * h + w][nt][0], qf[4 * h + w][nt][1]);
    }
  }
}

// Online softmax with the group's z (masked entries -inf) and O^T += V^T P^T.  unscale[0], [1]:
// 2^-e_v of positions r and r + 8 (changed here).  deep: some of the CTA's blocks lie below 2^kKv8Deep.
template <int D, int NT>
__device__ __forceinline__ void kv8_softmax_pv(WarpState<D, NT>& st, const float (&z)[NT][4],
                                               float (&unscale)[2], bool deep, uint32_t v_base) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  bool need = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) need |= fmaxf(z[nt][e], z[nt][2 + e]) > st.m[nt][e] + kKv8Top;
  if (__any_sync(0xffffffffu, need)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(z[nt][e], z[nt][2 + e]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mnew = fmaxf(st.m[nt][e], mx - kKv8Raise);
        const float h = half_weight(st.m[nt][e] - mnew), alpha = h * h;
        st.m[nt][e] = mnew;
        st.l[nt][e] = st.l[nt][e] * h * h;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          st.o[mt][nt][e] *= alpha;
          st.o[mt][nt][2 + e] *= alpha;
        }
      }
  }
  if (deep) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (unscale[j] <= two_to(-kKv8Deep)) continue;
      const float lifted = unscale[j] * two_to(-kKv8Lift);
      unscale[j] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          st.l[nt][e] = fmaf(ex2(z[nt][2 * j + e] - st.m[nt][e] + float(kKv8Lift)), lifted, st.l[nt][e]);
    }
  }
  uint32_t pb[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = ex2(z[nt][i] - st.m[nt][i & 1]);
      st.l[nt][i & 1] = fmaf(p[i], unscale[i >> 1], st.l[nt][i & 1]);
    }
    pb[nt][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
    pb[nt][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
  }
  uint32_t v[4][D / 32];   // words of positions 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = 2 * c + (i & 1) + 8 * (i >> 1);
    if constexpr (D == 128) {
      const uint4 x = lds128(v_base + Kv8Rows<D>::v(pos, r));
      v[i][0] = x.x;
      v[i][1] = x.y;
      v[i][2] = x.z;
      v[i][3] = x.w;
    } else {
      const uint2 x = lds64(v_base + Kv8Rows<D>::v(pos, r >> 1) + 8 * (r & 1));
      v[i][0] = x.x;
      v[i][1] = x.y;
    }
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t sel = b ? 0x7362u : 0x5140u;
      uint32_t a0, a1, a2, a3;
      f16x2_from_e4m3x4(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
      f16x2_from_e4m3x4(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_f16_16816(st.o[2 * w + b][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
    }
}

}  // namespace vegas
