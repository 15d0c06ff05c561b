// Positions of the 8-bit cache back into a bf16 one: out = bf16(c * 2^e), which is exact.
//
// One CTA a (sequence, page); sequences of many take turns on fewer CTAs, so that a call's length does
// not go by what its tables could hold.  A thread takes eight codes of one row (an 8-byte load, a 16-byte
// store, both contiguous across the warp) at the same place of every head's block, K and V, a few
// heads in flight; a block's exponent is one byte that all of its threads read.  Memory bounds
// it, at 6 d bytes a position and head: 90,000 positions of 8 heads of 128 in 85.3 us, 0.95 of the copy
// peak; 700 of 2 heads of 64 1.7 us, a launch and two dependent loads.
#include <algorithm>

#include "kernels.h"
#include "kv8.cuh"

namespace vegas {

namespace {
constexpr int kReadThreads = 256;
// CTAs of a call, and of a sequence at least (a CTA a page of the tables / these / 8192 and 152: one
// of 64K among 63 of 500, 8 heads of 128, 317 / 107 / 136 us; one of 20,000 among 63 of 30, 2 heads of
// 64, 83 / 22 / 11 us; eight up to 31,000 86 / 85 / 85 us).
constexpr int kReadCtas = 8192, kReadLeast = 304;
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
}  // namespace

template <int D>
__global__ void __launch_bounds__(kReadThreads) kv8_read_kernel(const Kv8ReadParams p) {
  constexpr int C = D / 8, Block = 16 * C;         // 8-code chunks of a row and of a block
  constexpr int Together = kReadThreads / Block;   // blocks that the CTA takes at once
  const int b = blockIdx.y, tid = threadIdx.x;
  griddep_begin();
  const int first = p.first ? p.first[b] : 0, upto = p.upto[b];
  if (upto <= first) return;                       // (nothing to read)
  if (first < 0 || upto > 16 * min(p.max_pages, p.to_max_pages)) {
    if (tid == 0 && blockIdx.x == 0) set_error(p.err, kErrDeviceFault);
    return;
  }
  const int chunk = tid % Block;
  for (int page = (first >> 4) + blockIdx.x; page * 16 < upto; page += gridDim.x) {
    const int from = p.block_table[size_t(b) * p.max_pages + page];
    const int to = p.to_block_table[size_t(b) * p.to_max_pages + page];
    if (from < 0 || from >= p.num_pages || to < 0 || to >= p.to_num_pages) {
      if (tid == 0) set_error(p.err, kErrDeviceFault);
      continue;
    }
    const int pos = page * 16 + chunk / C;
    if (pos < first || pos >= upto) continue;
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
}

cudaError_t launch_kv8_read(const Kv8ReadParams& p, int batch, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  // CTAs a sequence: its table's pages, but about kReadCtas in all
  const int pages = std::min(p.max_pages, p.to_max_pages);
  cfg.gridDim = dim3(std::min(pages, std::max(kReadLeast, kReadCtas / batch)), batch, 1);
  cfg.blockDim = dim3(kReadThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, kv8_read_kernel<64>, p)
                          : cudaLaunchKernelEx(&cfg, kv8_read_kernel<128>, p);
}

}  // namespace vegas
