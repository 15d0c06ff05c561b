// Rotary positions on queries and keys, and the append of keys and values to the cache in 8 bits,
// in one pass over the projections' output.
//
// The turning is that of rope_append.cu: y = bf16(s * R(p f) x).  Then, for every (page, KV head)
// that gets rows, with a the largest finite |y| of the page's new rows (all of its 16 x d elements
// that are new),
//   e_new = min { e : a <= 448 * 2^e },      c = e4m3(y * 2^-e),
// with e = e_new where the page begins with this call's rows, and e = max(e_new, e_old) where it
// holds rows of earlier calls (positions before ctx), whose codes become e4m3(c * 2^(e_old - e))
// when e is larger.  An exponent never falls while its page holds rows.
//
// A block's maximum needs all of its rows, so the unit of work is a page: two CTAs take the (at
// most 16) new rows of a page, each every other (KV head, K or V) and half of the query heads.  A warp
// holds one KV head's rows of the page in registers: lane l has unit l % (d / 16) (two chunks of 8
// elements: the two halves of 8 pairs) of every (32 / (d / 16))-th row, so the maximum is a warp
// reduction and no row is read twice.  The queries of the page's rows are then turned by all warps, an
// item a unit.  Each CTA makes the cosines and sines once per (row, pair), for all of its heads.  The
// angle in turns is taken modulo 1 by 64-bit integers: a pair's frequency over 2 pi, from fp64, as a
// fraction F of 2^64, and p F wraps by itself.  (In fp64, of which an SM does two operations a clock, the
// angles of 16K rows took 10 us of 70, and as much again for every part that the heads were divided
// into.)
//
// Pages are dealt out by slots: sequence b owns the slots from floor(row_start[b] / 16) + 2 b on,
// at least floor(n / 16) + 2 of them, and n rows touch at most that many pages; a slot without a
// page leaves at once.  Memory bounds large calls, the chain of dependent loads small ones: 16384
// rows of 32 + 8 + 8 heads of 128 58.0 us (0.94 of the copy peak), 48 windows of 5 rows of 64 + 8 + 8
// heads of 64 4.7 us, 32 single rows 4.0 us.
#include "kernels.h"
#include "kv8.cuh"

namespace vegas {

namespace {
constexpr int kQueryBatch = 4;   // query units a thread has in flight

__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// The larger of two pairs of bf16 magnitudes, infinities and NaN left out.
__device__ __forceinline__ uint32_t max_finite(uint32_t most, uint32_t v) {
  v &= 0x7fff7fffu;
  v &= __vcmpltu2(v, 0x7f807f80u);
  return __vmaxu2(most, v);
}

// Turns 8 pairs: chunks a and b (8 bf16 each) by (cos, sin) pairs cs[j][8 units], j = two pairs.
__device__ __forceinline__ void turn_unit(uint4& A, uint4& B, const float4* cs, int stride,
                                          bool interleaved) {
  uint32_t a[4] = {A.x, A.y, A.z, A.w}, b[4] = {B.x, B.y, B.z, B.w};
  float2 c[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = cs[j * stride];
    c[2 * j] = make_float2(v.x, v.y);
    c[2 * j + 1] = make_float2(v.z, v.w);
  }
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpack2(a[e]), y = unpack2(b[e]);
      a[e] = pack_bf16x2(x.x * c[e].x - x.y * c[e].y, x.y * c[e].x + x.x * c[e].y);
      b[e] = pack_bf16x2(y.x * c[4 + e].x - y.y * c[4 + e].y, y.y * c[4 + e].x + y.x * c[4 + e].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpack2(a[e]), y = unpack2(b[e]);
      const float2 p0 = c[2 * e], p1 = c[2 * e + 1];
      a[e] = pack_bf16x2(x.x * p0.x - y.x * p0.y, x.y * p1.x - y.y * p1.y);
      b[e] = pack_bf16x2(y.x * p0.x + x.x * p0.y, y.y * p1.x + x.y * p1.y);
    }
  }
  A = make_uint4(a[0], a[1], a[2], a[3]);
  B = make_uint4(b[0], b[1], b[2], b[3]);
}

__device__ __forceinline__ uint32_t max_of_chunk(uint32_t most, const uint4& v) {
  return max_finite(max_finite(max_finite(max_finite(most, v.x), v.y), v.z), v.w);
}

// Eight bf16 times 2^-e as codes.
__device__ __forceinline__ uint2 codes_of(const uint4& v, float inv) {
  auto two = [&](uint32_t w) {
    const float2 f = unpack2(w);
    return e4m3x2_from_f32(f.x * inv, f.y * inv);
  };
  return make_uint2(two(v.x) | two(v.y) << 16, two(v.z) | two(v.w) << 16);
}

__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float f) {
  uint32_t lo, hi;
  f16x2_from_e4m3x4(w, lo, hi);
  const float2 a = f32x2_from_f16x2(lo), b = f32x2_from_f16x2(hi);
  return e4m3x2_from_f32(a.x * f, a.y * f) | e4m3x2_from_f32(b.x * f, b.y * f) << 16;
}
}  // namespace

template <int D, int Threads>
__global__ void __launch_bounds__(Threads, Threads == 256 ? 3 : 1)
    kv8_append_kernel(const RopeKv8Params p) {
  constexpr int U = D / 16;              // units of a head
  constexpr int RowsPerPass = 32 / U, Passes = 16 / RowsPerPass;
  // (cos, sin) of pairs 2j, 2j + 1 of unit u of a row at [row][j][u]: eight lanes with
  // consecutive units read consecutive 16 bytes
  __shared__ float4 cs_all[16 * 4 * U];
  __shared__ unsigned long long turn_all[D / 2];   // F of a pair
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_begin();
  if (tid < (p.rot >> 1)) {
    const double c = double(p.inv_freq[tid]) * 0.15915494309189533577;   // 1 / (2 pi)
    turn_all[tid] = __double2ull_rn((c - floor(c)) * 18446744073709551616.0);
  }

  // The slot's sequence: the last b with floor(row_start[b] / 16) + 2 b <= slot, 32 at a time; the
  // last step brings the sequence's rows and context along.
  const int slot = blockIdx.x;
  int s = 0, beg = 0, end = 0, ctx = 0;
  for (int n = p.batch; n > 0;) {
    const int step = (n + 31) >> 5, at = s + lane * step;
    const bool there = lane * step < n;
    const int first = there ? p.row_start[at] : 0;
    int next = 0, held_rows = 0;
    if (step == 1 && there) {
      next = p.row_start[at + 1];
      held_rows = p.ctx_lens[at];
    }
    const unsigned m = __ballot_sync(0xffffffffu, there && (first >> 4) + 2 * at <= slot);
    if (!m) return;
    const int l = 31 - __clz(m);
    n = min(step, n - l * step);
    s += l * step;
    if (step == 1) {
      beg = __shfl_sync(0xffffffffu, first, l);
      end = __shfl_sync(0xffffffffu, next, l);
      ctx = __shfl_sync(0xffffffffu, held_rows, l);
      break;
    }
  }
  const int j = slot - ((beg >> 4) + 2 * s);
  if (end == beg) return;                // (without rows ctx may be anything)
  if (end < beg || beg < 0 || end > p.total_rows || ctx < 0 ||
      (long long)ctx + (end - beg) > (long long)p.max_pages * 16) {
    if (tid == 0) set_error(p.err, kErrDeviceFault);
    return;
  }
  // the page, and its new rows: t0 .. t0 + R - 1 of the sequence, at slots o .. o + R - 1
  const int page = (ctx >> 4) + j;
  const int t0 = max(0, page * 16 - ctx), R = min(end - beg, page * 16 + 16 - ctx) - t0;
  if (R <= 0) return;
  const int o = ctx + t0 - page * 16, row0 = beg + t0;
  const int phys = p.block_table[size_t(s) * p.max_pages + page];
  const bool held = j == 0 && o > 0;     // slots 0 .. o - 1 hold rows of earlier calls

  const int u = lane % U, half = p.rot >> 1;
  const bool turned = u < (p.rot >> 4);
  const int o0 = !turned || p.interleaved ? 16 * u : 8 * u;
  const int o1 = !turned || p.interleaved ? o0 + 8 : o0 + half;

  // this CTA's share of the heads: every gridDim.y-th (KV head, K or V), a run of query heads
  const int part = blockIdx.y, parts = gridDim.y;
  const int tasks = 2 * p.hkv, task0 = part + parts * warp;
  const int q0 = p.hq * part / parts, hq = p.hq * (part + 1) / parts - q0;
  uint4 A[Passes], B[Passes];
  auto load_task = [&](int t) {
    const bool is_v = t >= p.hkv;
    const int g = is_v ? t - p.hkv : t;
    const uint16_t* src = is_v ? reinterpret_cast<const uint16_t*>(p.v) + size_t(row0) * p.v_stride
                               : reinterpret_cast<const uint16_t*>(p.k) + size_t(row0) * p.k_stride;
    const size_t stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
    for (int i = 0; i < Passes; ++i) {
      const int r = lane / U + i * RowsPerPass;
      A[i] = B[i] = make_uint4(0, 0, 0, 0);
      if (r < R) {
        const uint16_t* at = src + r * stride + g * D;
        // values keep their place in the row; keys are turned in pairs of chunks
        A[i] = *reinterpret_cast<const uint4*>(at + (is_v ? 16 * u : o0));
        B[i] = *reinterpret_cast<const uint4*>(at + (is_v ? 16 * u + 8 : o1));
      }
    }
  };
  // The warp's first (KV head, K or V): its rows are on their way under the sines below.
  if (task0 < tasks) load_task(task0);

  // Queries: item i is unit i % U of head q0 + (i / U) % hq of row i / (U hq).
  const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + size_t(row0) * p.q_stride + q0 * D;
  uint16_t* qo = reinterpret_cast<uint16_t*>(p.q_out) + (size_t(row0) * p.hq + q0) * D;
  constexpr int Step = Threads / U;   // heads from one item of a thread to its next
  const int step_r = hq ? Step / hq : 0, step_h = Step - step_r * hq;
  int r = hq ? (tid / U) / hq : R, h = tid / U - r * hq;
  uint4 a[kQueryBatch], b[kQueryBatch];
  int rr[kQueryBatch], hh[kQueryBatch];
  auto load_queries = [&]() {
#pragma unroll
    for (int i = 0; i < kQueryBatch; ++i) {
      rr[i] = r;
      hh[i] = h;
      if (r < R) {
        const uint16_t* at = q + r * size_t(p.q_stride) + h * D;
        a[i] = *reinterpret_cast<const uint4*>(at + o0);
        b[i] = *reinterpret_cast<const uint4*>(at + o1);
      }
      h += step_h;
      r += step_r;
      if (h >= hq) {
        h -= hq;
        ++r;
      }
    }
  };
  // few threads a page (many pages): other CTAs hide the latency, and registers are short
  constexpr bool kEarly = Threads > 256;
  if (kEarly) load_queries();

  __syncthreads();
  float2* cs2 = reinterpret_cast<float2*>(cs_all);
  for (int i = tid; i < R * half; i += Threads) {
    const int r = i / half, pair = i - r * half;
    int at = ctx + t0 + r;
    if (p.positions) {
      int axis = p.pair_axis ? p.pair_axis[pair] : 0;
      if (axis < 0 || axis >= p.num_axes) {
        set_error(p.err, kErrDeviceFault);
        axis = 0;
      }
      at = p.positions[size_t(axis) * p.total_rows + row0 + r];
    }
    const float turns = __ll2float_rn((long long)((unsigned long long)at * turn_all[pair])) * 0x1p-64f;
    float sn, cn;
    sincospif(2.f * turns, &sn, &cn);
    const int unit = pair >> 3, e = pair & 7;
    cs2[((r * 4 + (e >> 1)) * U + unit) * 2 + (e & 1)] = make_float2(cn * p.scale, sn * p.scale);
  }
  const bool page_ok = phys >= 0 && phys < p.num_pages;
  if (!page_ok && tid == 0) set_error(p.err, kErrDeviceFault);
  __syncthreads();

  for (int t = page_ok ? task0 : tasks; t < tasks; t += parts * (Threads / 32)) {
    if (t != task0) load_task(t);
    const bool is_v = t >= p.hkv;
    const int g = is_v ? t - p.hkv : t;
    const size_t block = size_t(phys) * p.hkv + g;
    uint8_t* codes = reinterpret_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + block * 16 * D;
    uint8_t* scale = (is_v ? p.v_scale : p.k_scale) + block;
    const int e_old = held ? kv8_exponent(*scale) : kKv8MinExp;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < Passes; ++i) {
      const int r = lane / U + i * RowsPerPass;
      if (!is_v && turned && r < R) turn_unit(A[i], B[i], cs_all + r * 4 * U + u, U, p.interleaved);
      most = max_of_chunk(max_of_chunk(most, A[i]), B[i]);
    }
    most = max(most & 0xffffu, most >> 16);
    const int e = max(e_old, kv8_exponent_for(__reduce_max_sync(0xffffffffu, most)));
    const float inv = two_to(-e);
    const int w0 = is_v ? 16 * u : o0, w1 = is_v ? 16 * u + 8 : o1;
#pragma unroll
    for (int i = 0; i < Passes; ++i) {
      const int r = lane / U + i * RowsPerPass;
      if (r < R) {
        *reinterpret_cast<uint2*>(codes + (o + r) * D + w0) = codes_of(A[i], inv);
        *reinterpret_cast<uint2*>(codes + (o + r) * D + w1) = codes_of(B[i], inv);
      }
    }
    if (held && e > e_old) {
      const float f = two_to(e_old - e);
      for (int c = lane; c < o * U; c += 32) {
        uint4* at = reinterpret_cast<uint4*>(codes) + c;
        const uint4 v = *at;
        *at = make_uint4(rescale_codes(v.x, f), rescale_codes(v.y, f), rescale_codes(v.z, f),
                         rescale_codes(v.w, f));
      }
    }
    if (lane == 0) *scale = uint8_t(e + kKv8Bias);
  }

  bool loaded = kEarly;
  while (true) {
    if (!loaded) load_queries();
    loaded = false;
#pragma unroll
    for (int i = 0; i < kQueryBatch; ++i) {
      if (rr[i] >= R) continue;
      if (turned) turn_unit(a[i], b[i], cs_all + rr[i] * 4 * U + u, U, p.interleaved);
      uint16_t* at = qo + (size_t(rr[i]) * p.hq + hh[i]) * D;
      *reinterpret_cast<uint4*>(at + o0) = a[i];
      *reinterpret_cast<uint4*>(at + o1) = b[i];
    }
    if (rr[kQueryBatch - 1] >= R) break;
  }
}

template <int Threads>
static cudaError_t launch_threads(const RopeKv8Params& p, int parts, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.total_rows / 16 + 2 * p.batch, parts, 1);
  cfg.blockDim = dim3(Threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, kv8_append_kernel<64, Threads>, p)
                          : cudaLaunchKernelEx(&cfg, kv8_append_kernel<128, Threads>, p);
}

cudaError_t launch_kv8_append(const RopeKv8Params& p, int sms, cudaStream_t stream) {
  // Two CTAs a page, each half of the heads.  While they are about one wave of SMs, 512 threads
  // each; from there on 256, three on an SM, so that one's lookups run under another's stream
  // (32 query and 8 KV heads of 128; 512 / 256 threads: 32 pages of a row 4.0 / 4.8 us, 63 pages 6.0 /
  // 11.4, 126 pages 15.1 / 12.8, 500 pages 46.8 / 31.3, 1024 pages 87 / 58; with one CTA a page and
  // 256 threads 60, with four 68, as each makes the page's sines anew).
  const long long pages = p.total_rows / 16 + (long long)p.batch;
  return 2 * pages <= sms ? launch_threads<512>(p, 2, stream) : launch_threads<256>(p, 2, stream);
}

}  // namespace vegas
