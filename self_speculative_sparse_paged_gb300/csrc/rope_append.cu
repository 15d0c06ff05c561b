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
#include "kernels.h"
#include "vegas_common.cuh"

namespace vegas {

namespace {
constexpr int kRopeThreads = 256;

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
}  // namespace

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  __shared__ float2 cs[64];          // (cos, sin) of each pair
  __shared__ int where[2];           // sequence, cache position
  griddep_begin();
  const int row = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) where[0] = -1;
  __syncthreads();
  for (int s = tid; s < p.batch; s += kRopeThreads) {
    const int beg = p.row_start[s], end = p.row_start[s + 1];
    if (end < beg) set_error(p.err, kErrDeviceFault);
    if (row >= beg && row < end) {
      const int ctx = p.ctx_lens[s];
      if (beg < 0 || end > p.total_rows || ctx < 0 ||
          (long long)ctx + (end - beg) > (long long)p.max_pages * 16) {
        set_error(p.err, kErrDeviceFault);
      } else {
        where[0] = s;
        where[1] = ctx + (row - beg);
      }
    }
  }
  __syncthreads();
  const int seq = where[0], pos = where[1];
  if (seq < 0) return;               // a row behind the last sequence
  const int page = p.block_table[size_t(seq) * p.max_pages + (pos >> 4)];
  const bool page_ok = page >= 0 && page < p.num_pages;
  if (!page_ok && tid == 0) set_error(p.err, kErrDeviceFault);
  const int half = p.rot >> 1;
  if (tid < half) {
    int at = pos;
    if (p.positions) {
      int a = p.pair_axis ? p.pair_axis[tid] : 0;
      if (a < 0 || a >= p.num_axes) {
        set_error(p.err, kErrDeviceFault);
        a = 0;
      }
      at = p.positions[size_t(a) * p.total_rows + row];
    }
    double turns = double(at) * double(p.inv_freq[tid]) * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= rint(turns);
    float sn, cn;
    sincospif(2.f * float(turns), &sn, &cn);
    cs[tid] = make_float2(cn * p.scale, sn * p.scale);
  }
  __syncthreads();

  const int D = p.head_dim, hr = p.hq + p.hkv;
  const int pc = half >> 3;                 // units of 8 pairs per head
  const int rest = (D - p.rot) >> 3;        // 16-byte chunks per head that pass through
  const int n_rot = hr * pc, n_pass = hr * rest, n_v = p.hkv * (D >> 3);
  const uint16_t* qrow = reinterpret_cast<const uint16_t*>(p.q) + size_t(row) * p.q_stride;
  const uint16_t* krow = reinterpret_cast<const uint16_t*>(p.k) + size_t(row) * p.k_stride;
  const uint16_t* vrow = reinterpret_cast<const uint16_t*>(p.v) + size_t(row) * p.v_stride;
  uint16_t* qout = reinterpret_cast<uint16_t*>(p.q_out) + size_t(row) * p.hq * D;
  auto cache_row = [&](void* cache, int g) {
    return reinterpret_cast<uint16_t*>(cache) +
           ((size_t(page) * p.hkv + g) * 16 + (pos & 15)) * D;
  };
  for (int i = tid; i < n_rot + n_pass + n_v; i += kRopeThreads) {
    if (i < n_rot) {
      const int h = i / pc, u = i - h * pc;
      const bool is_q = h < p.hq;
      if (!is_q && !page_ok) continue;
      const uint16_t* src = is_q ? qrow + h * D : krow + (h - p.hq) * D;
      uint16_t* dst = is_q ? qout + h * D : cache_row(p.k_cache, h - p.hq);
      const int o0 = p.interleaved ? 16 * u : 8 * u, o1 = p.interleaved ? o0 + 8 : o0 + half;
      const uint4 A = *reinterpret_cast<const uint4*>(src + o0);
      const uint4 B = *reinterpret_cast<const uint4*>(src + o1);
      const uint32_t a[4] = {A.x, A.y, A.z, A.w}, b[4] = {B.x, B.y, B.z, B.w};
      uint32_t ra[4], rb[4];
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack_bf16x2(a[e]), y = unpack_bf16x2(b[e]);
          const float2 c0 = cs[8 * u + e], c1 = cs[8 * u + 4 + e];
          ra[e] = pack_bf16x2(x.x * c0.x - x.y * c0.y, x.y * c0.x + x.x * c0.y);
          rb[e] = pack_bf16x2(y.x * c1.x - y.y * c1.y, y.y * c1.x + y.x * c1.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack_bf16x2(a[e]), y = unpack_bf16x2(b[e]);
          const float2 c0 = cs[8 * u + 2 * e], c1 = cs[8 * u + 2 * e + 1];
          ra[e] = pack_bf16x2(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
          rb[e] = pack_bf16x2(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
        }
      }
      *reinterpret_cast<uint4*>(dst + o0) = make_uint4(ra[0], ra[1], ra[2], ra[3]);
      *reinterpret_cast<uint4*>(dst + o1) = make_uint4(rb[0], rb[1], rb[2], rb[3]);
    } else if (i < n_rot + n_pass) {
      const int k = i - n_rot, h = k / rest, c = p.rot + 8 * (k - h * rest);
      const bool is_q = h < p.hq;
      if (!is_q && !page_ok) continue;
      const uint16_t* src = is_q ? qrow + h * D : krow + (h - p.hq) * D;
      uint16_t* dst = is_q ? qout + h * D : cache_row(p.k_cache, h - p.hq);
      *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(src + c);
    } else if (page_ok) {
      const int k = i - n_rot - n_pass, per = D >> 3, g = k / per, c = 8 * (k - g * per);
      *reinterpret_cast<uint4*>(cache_row(p.v_cache, g) + c) =
          *reinterpret_cast<const uint4*>(vrow + g * D + c);
    }
  }
}

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.total_rows, 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_append_kernel, p);
}

}  // namespace vegas
