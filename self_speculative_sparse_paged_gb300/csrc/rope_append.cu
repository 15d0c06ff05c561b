// Rotary positions on queries and keys, and the append of the rotated keys and
// of the values to the paged cache, in one pass over the projections' output.
//
// Row t of sequence b sits at cache position c_b + t.  Pair j < rot / 2 of
// every query and key head turns by the angle p_a * f_j, where p_a is the
// row's position on the pair's axis a (time, height, width of an image or
// video token; one axis, the cache position, for text):
//   (x, y) -> s * (x cos - y sin, y cos + x sin),
// the pair being elements (j, j + rot / 2) or, interleaved, (2j, 2j + 1).
//
// A far position times a frequency needs more than fp32's 24 bits before the
// whole turns are dropped (position 10^5 would leave 0.004 rad), so the
// product and the reduction to [-1/2, 1/2] turn are done in fp64, once per
// (row, pair) and shared by all heads through shared memory; the remainder
// goes to sine and cosine in fp32.  The rotation is fp32, rounded once to bf16.
//
// Memory bounds the call.  A warp takes a row, or with few rows a fourth of one:
// lane i turns unit i % (rot / 16) (8 pairs) of head i / (rot / 16) and the heads
// a fixed stride on, so its cosines and sines stay in registers and a head costs
// two 16-byte loads, 32 multiply-adds and two 16-byte stores, with no barrier
// between warps; the first heads, the frequencies and the given positions are loaded
// before the row's sequence and page are looked up.  32768 rows of 32 + 8 + 8 heads of
// 128: 127 us, 6.35 TB/s of bytes read and written once (0.93 of the measured copy); 32
// rows: 3.2 us, launch and three dependent lookups.
#include "kernels.h"
#include "vegas_common.cuh"

namespace vegas {

namespace {
constexpr int kRopeWarps = 4;   // warps of a block

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
}  // namespace

// Split: warps that share a row (1, 2 or kRopeWarps); Batch: heads a lane has in flight.
template <int Split, int Batch>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs_all[kRopeWarps][64];   // scaled (cos, sin) of each pair
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kRopeWarps / Split) + warp / Split, part = warp % Split;
  float2* cs = cs_all[warp];
  griddep_begin();
  if (row >= p.total_rows) return;

  const uint16_t* qrow = reinterpret_cast<const uint16_t*>(p.q) + size_t(row) * p.q_stride;
  const uint16_t* krow = reinterpret_cast<const uint16_t*>(p.k) + size_t(row) * p.k_stride;
  const uint16_t* vrow = reinterpret_cast<const uint16_t*>(p.v) + size_t(row) * p.v_stride;
  const int D = p.head_dim, half = p.rot >> 1;
  auto source = [&](int h) { return h < p.hq ? qrow + h * D : krow + (h - p.hq) * D; };
  // the lane's unit, its two chunks of a head, its first head and the step to the next
  const int units = p.rot >> 4, per_pass = units ? 32 / units : 0, hl = units ? lane / units : 0;
  const int u = lane - hl * units, o0 = p.interleaved ? 16 * u : 8 * u;
  const int o1 = p.interleaved ? o0 + 8 : o0 + half;
  const int all_heads = p.hq + p.hkv, stride = per_pass * Split;
  const int h0 = hl < per_pass ? hl + part * per_pass : all_heads;
  uint4 A[Batch], B[Batch];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < Batch; ++i) {
      const int hh = h + i * stride;
      if (hh >= all_heads) continue;
      const uint16_t* src = source(hh);
      A[i] = *reinterpret_cast<const uint4*>(src + o0);
      B[i] = *reinterpret_cast<const uint4*>(src + o1);
    }
  };
  if (units) load(h0);   // the first heads are on their way under the lookups below
  // the frequencies, and the positions where they are given, of the lane's two pairs
  float freq[2] = {0.f, 0.f};
  int given[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j >= half) continue;
    freq[i] = p.inv_freq[j];
    if (p.positions) {
      int axis = p.pair_axis ? p.pair_axis[j] : 0;
      if (axis < 0 || axis >= p.num_axes) {
        set_error(p.err, kErrDeviceFault);
        axis = 0;
      }
      given[i] = p.positions[size_t(axis) * p.total_rows + row];
    }
  }

  // The row's sequence: the last one that begins at or before it, found 32 at a time.
  int s = 0;
  for (int n = p.batch; n > 0;) {
    const int step = (n + 31) >> 5, at = s + lane * step;
    const bool before = lane * step < n && p.row_start[at] <= row;
    const unsigned m = __ballot_sync(0xffffffffu, before);
    if (!m) return;                  // (no sequence begins that early)
    const int l = 31 - __clz(m);
    n = min(step, n - l * step);
    s += l * step;
    if (step == 1) break;
  }
  const int beg = p.row_start[s], end = p.row_start[s + 1], ctx = p.ctx_lens[s];
  if (end < beg) {
    if (lane == 0) set_error(p.err, kErrDeviceFault);
    return;
  }
  if (row >= end) return;            // a row behind the last sequence
  if (beg < 0 || end > p.total_rows || ctx < 0 ||
      (long long)ctx + (end - beg) > (long long)p.max_pages * 16) {
    if (lane == 0) set_error(p.err, kErrDeviceFault);
    return;
  }
  const int pos = ctx + (row - beg);
  const int page = p.block_table[size_t(s) * p.max_pages + (pos >> 4)];
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (!page_ok && lane == 0) set_error(p.err, kErrDeviceFault);

#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = lane + 32 * i;
    if (j >= half) continue;
    const int at = p.positions ? given[i] : pos;
    double turns = double(at) * double(freq[i]) * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cn;
    sincospif(2.f * float(turns), &sn, &cn);
    cs[j] = make_float2(cn * p.scale, sn * p.scale);
  }
  __syncwarp();

  uint16_t* qout = reinterpret_cast<uint16_t*>(p.q_out) + size_t(row) * p.hq * D;
  const size_t slot = (size_t(page_ok ? page : 0) * p.hkv * 16 + (pos & 15)) * D;
  uint16_t* kslot = reinterpret_cast<uint16_t*>(p.k_cache) + slot;
  uint16_t* vslot = reinterpret_cast<uint16_t*>(p.v_cache) + slot;
  const int heads = page_ok ? all_heads : p.hq;   // (a key without a page goes nowhere)
  auto target = [&](int h) { return h < p.hq ? qout + h * D : kslot + (h - p.hq) * 16 * D; };

  if (p.rot > 0) {
    float2 c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = cs[8 * u + e];
    for (int h = h0; h < heads; h += Batch * stride) {
      if (h != h0) load(h);
#pragma unroll
      for (int i = 0; i < Batch; ++i) {
        const int hh = h + i * stride;
        if (hh >= heads) continue;
        uint32_t a[4] = {A[i].x, A[i].y, A[i].z, A[i].w}, b[4] = {B[i].x, B[i].y, B[i].z, B[i].w};
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack_bf16x2(a[e]), y = unpack_bf16x2(b[e]);
            a[e] = pack_bf16x2(x.x * c[e].x - x.y * c[e].y, x.y * c[e].x + x.x * c[e].y);
            b[e] = pack_bf16x2(y.x * c[4 + e].x - y.y * c[4 + e].y,
                               y.y * c[4 + e].x + y.x * c[4 + e].y);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack_bf16x2(a[e]), y = unpack_bf16x2(b[e]);
            const float2 p0 = c[2 * e], p1 = c[2 * e + 1];
            a[e] = pack_bf16x2(x.x * p0.x - y.x * p0.y, x.y * p1.x - y.y * p1.y);
            b[e] = pack_bf16x2(y.x * p0.x + x.x * p0.y, y.y * p1.x + x.y * p1.y);
          }
        }
        uint16_t* dst = target(hh);
        *reinterpret_cast<uint4*>(dst + o0) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(dst + o1) = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  }
  const int first = lane + 32 * part, step = 32 * Split;
  const int rest = (D - p.rot) >> 3;   // 16-byte chunks of a head that pass through
  for (int i = first; i < heads * rest; i += step) {
    const int h = i / rest, o = p.rot + 8 * (i - h * rest);
    *reinterpret_cast<uint4*>(target(h) + o) = *reinterpret_cast<const uint4*>(source(h) + o);
  }
  if (page_ok) {
    const int shift = D == 128 ? 4 : 3;   // chunks of a value head
#pragma unroll 4
    for (int i = first; i < p.hkv << shift; i += step) {
      const int g = i >> shift, o = 8 * (i - (g << shift));
      *reinterpret_cast<uint4*>(vslot + g * 16 * D + o) =
          *reinterpret_cast<const uint4*>(vrow + g * D + o);
    }
  }
}

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t stream) {
  // Warps a row: one when the rows alone keep the SMs busy, else two, else four (32 query and
  // 8 KV heads of 128: 1000 rows 14.1 / 10.3 / 9.0 us, 2000 rows 14.8 / 13.2 / 15.2 us, 4000 rows
  // 21.0 / 22.0 / 24.9 us with one / two / four; no other shape of heads was measured).
  const int split = p.total_rows >= 3000 ? 1 : p.total_rows >= 1500 ? 2 : kRopeWarps;
  const int rows = kRopeWarps / split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.total_rows + rows - 1) / rows, 1, 1);
  cfg.blockDim = dim3(32 * kRopeWarps, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Heads in flight: four of 64, two of 128 (3021 rows of 64: 14.7 us against 17.2 with two;
  // 32768 rows of 128: 131 us against 128 with four).
  if (split == 1)
    return p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, rope_append_kernel<1, 4>, p)
                            : cudaLaunchKernelEx(&cfg, rope_append_kernel<1, 2>, p);
  if (split == 2) return cudaLaunchKernelEx(&cfg, rope_append_kernel<2, 2>, p);
  return cudaLaunchKernelEx(&cfg, rope_append_kernel<kRopeWarps, 3>, p);
}

}  // namespace vegas
