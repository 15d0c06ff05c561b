// Positions of the 8-bit cache back into a bf16 one: out = bf16(c * 2^e), which is exact.
//
// The unit of work is a page of a sequence.  While the tables hold few pages a CTA stands ready for each of
// them; beyond that a bounded grid takes turns on the pages that the sequences have, so that a call's length
// goes by those and not by what its tables could hold.  A thread takes eight codes of one row (an 8-byte load,
// a 16-byte store, both contiguous across the warp) at the same place of every head's block, K and V, a few
// heads in flight; a block's exponent is one byte that all of its threads read.  Memory bounds it, at 6 d
// bytes a position and head: 90,000 positions of 8 heads of 128 in 85.7 us, 0.95 of the copy peak; 700 of 2
// heads of 64 1.7 us, a launch and two dependent loads.
#include <algorithm>

#include "kernels.h"
#include "kv8.cuh"

namespace vegas {

namespace {
constexpr int kReadThreads = 256;
// Pages of the tables up to which each has a CTA (of 16 x 4000, 32 x 500 and 1 x 64K, 8 heads of 128, 61.0, 13.3
// and 62.5 us; in turns 61.7, 15.0 and 63.5; one of 700 1.8 and 2.1), and the CTAs that take turns beyond: every
// one of them counts the pages of all sequences, 256 at a time, so they are fewer for a batch of more
// than that (kReadCtas 2432, 4864, 8192: eight up to 31,000 77.9, 75.9, 76.3 us, one of 20,000 among 63 of 30
// 6.6, 9.4, 13.2; kReadFew 1216, 2432, 8192: 8192 x 20 83, 119, 291, one of 32K among 1023 of 100 140, 133, 132).
// A CTA for every page of the tables, however many, took 317 us for 1024 x 100 in tables of 64K (99 in
// turns), 107 for one of 64K among 63 of 500 (92).
constexpr int kReadPages = 8192, kReadCtas = 4864, kReadFew = 2432;
constexpr int kReadBatch = 4;   // blocks (each K and V) a thread has in flight

__device__ __forceinline__ uint4 bf16_of(uint2 c, float f) {
  uint32_t h[4], w[4];
  f16x2_from_e4m3x4(c.x, h[0], h[1]);
  f16x2_from_e4m3x4(c.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f32x2_from_f16x2(h[i]);
    w[i] = pack_bf16x2(v.x * f, v.y * f);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A chunk of the batch: 256 sequences, their ranges, and how many pages they have up to each.
struct ReadChunk {
  int first[kReadThreads], upto[kReadThreads], ends[kReadThreads];
  int warp_pages[kReadThreads / 32];
};

// Whether sequence b has positions to read; its range.
__device__ __forceinline__ bool read_range(const Kv8ReadParams& p, int b, bool record, int& first, int& upto) {
  first = p.first ? p.first[b] : 0;
  upto = p.upto[b];
  if (upto <= first) return false;
  const bool fits = first >= 0 && upto <= 16 * min(p.max_pages, p.to_max_pages);
  if (!fits && record) set_error(p.err, kErrDeviceFault);
  return fits;
}

// The positions of [first, upto) in a page of sequence b, by the whole CTA.
template <int D>
__device__ __forceinline__ void read_page(const Kv8ReadParams& p, size_t b, int page, int first, int upto) {
  constexpr int C = D / 8, Block = 16 * C;         // 8-code chunks of a row and of a block
  constexpr int Together = kReadThreads / Block;   // blocks that the CTA takes at once
  const int tid = threadIdx.x, chunk = tid % Block;
  const int from = p.block_table[b * p.max_pages + page];
  const int to = p.to_block_table[b * p.to_max_pages + page];
  if (from < 0 || from >= p.num_pages || to < 0 || to >= p.to_num_pages) {
    if (tid == 0) set_error(p.err, kErrDeviceFault);
    return;
  }
  const int pos = page * 16 + chunk / C;
  if (pos < first || pos >= upto) return;
  for (int g0 = tid / Block; g0 < p.hkv; g0 += Together * kReadBatch) {
    uint2 k[kReadBatch], v[kReadBatch];
    uint8_t ek[kReadBatch], ev[kReadBatch];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int g = g0 + i * Together;
      if (g >= p.hkv) continue;
      const size_t block = size_t(from) * p.hkv + g;
      k[i] = reinterpret_cast<const uint2*>(p.k_cache)[block * Block + chunk];
      v[i] = reinterpret_cast<const uint2*>(p.v_cache)[block * Block + chunk];
      ek[i] = p.k_scale[block];
      ev[i] = p.v_scale[block];
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int g = g0 + i * Together;
      if (g >= p.hkv) continue;
      const size_t at = (size_t(to) * p.hkv + g) * Block + chunk;
      reinterpret_cast<uint4*>(p.to_k)[at] = bf16_of(k[i], two_to(kv8_exponent(ek[i])));
      reinterpret_cast<uint4*>(p.to_v)[at] = bf16_of(v[i], two_to(kv8_exponent(ev[i])));
    }
  }
}
}  // namespace

// Grid (pages of the tables, batch).  (With a loop, although every CTA has one page at most: its loads are
// kept together then, 32 x 500 14.3 -> 13.3 us.)
template <int D>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const Kv8ReadParams p) {
  const int b = blockIdx.y;
  griddep_begin();
  int first, upto;
  if (!read_range(p, b, threadIdx.x == 0 && blockIdx.x == 0, first, upto)) return;
  for (int page = (first >> 4) + blockIdx.x; page * 16 < upto; page += gridDim.x)
    read_page<D>(p, b, page, first, upto);
}

// A bounded grid takes turns on the pages that the sequences have, standing in one row.
template <int D>
__global__ void __launch_bounds__(kReadThreads) kv8_read_turns_kernel(const Kv8ReadParams p) {
  __shared__ ReadChunk ch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_begin();
  long long next = blockIdx.x;   // the CTA's next page, counted from the chunk's first
  for (int b0 = 0; b0 < p.batch; b0 += kReadThreads) {
    int first = 0, upto = 0, pages = 0;
    if (b0 + tid < p.batch && read_range(p, b0 + tid, blockIdx.x == 0, first, upto))
      pages = ((upto + 15) >> 4) - (first >> 4);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pages, o);
      if (lane >= o) pages += v;
    }
    if (b0) __syncthreads();     // (the chunk before has been read)
    if (lane == 31) ch.warp_pages[warp] = pages;
    ch.first[tid] = first;
    ch.upto[tid] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kReadThreads / 32; ++w) {
      const int v = ch.warp_pages[w];
      if (w < warp) pages += v;
      total += v;
    }
    ch.ends[tid] = pages;
    __syncthreads();
    for (; next < total; next += gridDim.x) {
      // its sequence: the first whose pages end behind it
      const int i = int(next);
      const int s8 = 8 * __popc(__ballot_sync(0xffffffffu, ch.ends[8 * lane + 7] <= i));
      const int s = s8 + __popc(__ballot_sync(0xffffffffu, lane < 8 && ch.ends[s8 + (lane & 7)] <= i));
      const int page = (ch.first[s] >> 4) + i - (s ? ch.ends[s - 1] : 0);
      read_page<D>(p, size_t(b0 + s), page, ch.first[s], ch.upto[s]);
      __syncwarp();
    }
    next -= total;
  }
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int pages = std::min(p.max_pages, p.to_max_pages);
  const bool turns = (long long)pages * p.batch > kReadPages;
  cfg.gridDim = turns ? dim3(p.batch <= kReadThreads ? kReadCtas : kReadFew, 1, 1) : dim3(pages, p.batch, 1);
  cfg.blockDim = dim3(kReadThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.head_dim == 64)
    return cudaLaunchKernelEx(&cfg, turns ? kv8_read_turns_kernel<64> : kv8_read_kernel<64>, p);
  return cudaLaunchKernelEx(&cfg, turns ? kv8_read_turns_kernel<128> : kv8_read_kernel<128>, p);
}

}  // namespace vegas
